"""What the paged-cache calls promise beside their formulas: lengths past the table, values that are
not finite, a sequence's bits, rows that are to give nothing, weights under a window, calls from
several host threads, and sizes past the tests of the formulas (GPU).  Tolerances are those of
test_gpu_paged.py."""
import ctypes
import math
import threading

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_paged import BF16, F16, Batch, check_mass, pp_, run_evict, turned  # noqa: E402


# ---- lengths past the table ---------------------------------------------------------------------

def full(type, D, chunks, over, window=0, page=16, width=20, seed=1):
    """Sequences that fill their table row (width * page entries), and one that does not; kv_len
    says `over` entries more for the first ones.  `lens` are the entries that there are."""
    cap = width * page
    lens = [cap] * (len(chunks) - 1) + [cap // 2 + 3]
    b = Batch(type, D, 2, 2, page, chunks, lens, window=window, seed=seed)
    b.told = [cap + over] * (len(chunks) - 1) + lens[-1:]
    b.len = torch.tensor(b.told, dtype=torch.int32, device="cuda")

    def sees(s):
        p = torch.arange(b.told[s] - b.chunks[s], b.told[s], device="cuda")[:, None]
        j = torch.arange(b.lens[s], device="cuda")[None]
        m = j <= p
        return m & (j > p - b.window) if b.window else m
    b.sees = sees
    return b


OVER = [(over, window) for over in (1, 3, 70) for window in (0, 50)] + [(70, 325)]


@pytest.mark.parametrize("type,D", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("over,window", OVER)
@pytest.mark.parametrize("chunks", [[1, 1], [5, 2], [200, 9]])
def test_rows_keep_their_places_when_the_table_is_full(chunks, over, window, type, D):
    """Row i sits at entry kv_len - n + i whether or not that entry has a place; the entries that
    have none take no part, and the status says so."""
    b = full(type, D, chunks, over, window)
    kv = b.kv()
    out, lse = kv.attention(b.q, b.cu, b.len, max_q=max(chunks), window=window, with_lse=True)
    assert kv.read_status() == pp_().PP_S_INDEX
    b.check(out, lse)
    before = b.mass.clone()
    kv.attention_mass(b.q, lse, b.cu, b.len, max_q=max(chunks), window=window, decay=0.5)
    assert kv.read_status() == pp_().PP_S_INDEX
    for s in range(len(chunks)):
        check_mass(b, s, before, b.mass, lse, 0.5)
    # a stored infinity in the last tile reaches the rows that see it and no other
    p, r = b.where(0)
    j = b.lens[0] - 2
    v = b.v.clone()
    v[p[j], :, r[j], 3] = math.inf
    got, gl = pp_().PagedKV(b.k, v, b.table).attention(b.q, b.cu, b.len, max_q=max(chunks),
                                                       window=window, with_lse=True)
    see = torch.zeros(b.T, dtype=torch.bool, device="cuda")
    see[b.at[0]:b.at[1]] = b.sees(0)[:, j]
    ok = torch.ones_like(got, dtype=torch.bool)
    ok[see, :, 3] = False
    assert torch.equal(got[ok], out[ok]) and torch.equal(gl, lse)
    assert (got[see][:, :, 3] == math.inf).all()


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("chunk,over", [(1, 1), (5, 2), (5, 40), (40, 1)])
def test_append_past_the_table_leaves_the_entries_that_are_there(chunk, over, far):
    b = full(BF16, 128, [chunk, 3], over)
    x = torch.randn((b.T, 4 + 2 + 2, 128), generator=b.g, device="cuda").to(BF16)
    K, V, M = b.k.clone(), b.v.clone(), b.mass.clone()
    kv = pp_().PagedKV(K, V, b.table, mass=M)
    entry = torch.cat([torch.arange(b.told[s] - b.chunks[s], b.told[s]) for s in range(2)]).int().cuda()
    pos = entry + 1000 if far else entry
    out = kv.append(x[:, :4], x[:, 4:6], x[:, 6:], b.cu, b.len, positions=pos if far else None)
    assert kv.read_status() == pp_().PP_S_INDEX
    want, tol = turned(x[:, :4], None, pos, 128, False)
    half = torch.finfo(BF16).eps / 2
    assert ((out.double() - want).abs() <= tol + half * want.abs()).all()
    kw, ktol = turned(x[:, 4:6], None, pos, 128, False)
    touched = torch.zeros(b.n_pages, b.page, dtype=torch.bool, device="cuda")
    for s in range(2):
        p, r = b.where(s)
        for i in range(b.chunks[s]):
            j, t = b.told[s] - b.chunks[s] + i, b.at[s] + i
            if j >= b.lens[s]:
                continue
            touched[p[j], r[j]] = True
            assert torch.equal(V[p[j], :, r[j]], x[t, 6:])
            assert ((K[p[j], :, r[j]].double() - kw[t]).abs() <= ktol[t] + half * kw[t].abs()).all()
            assert (M[p[j], :, r[j]] == 0).all()
    for new, old in ((K, b.k), (V, b.v), (M, b.mass)):
        assert torch.equal(new.transpose(1, 2)[~touched], old.transpose(1, 2)[~touched])


def test_lengths_of_any_size_are_taken():
    """The largest int32 (taken as 2^30) and the lowest: the first sees its whole row, the other
    nothing."""
    b = full(BF16, 64, [2, 2], 2 ** 31 - 1 - 320)
    b.told[0], b.told[1], b.lens[1] = 2 ** 30, 0, 0
    b.len[1] = -(2 ** 31)
    for max_q in (2, 300):
        kv = b.kv()
        out, lse = kv.attention(b.q, b.cu, b.len, max_q=max_q, with_lse=True)
        b.check(out, lse)
        assert kv.read_status() == pp_().PP_S_INDEX
        assert (out[2:] == 0).all() and (lse[2:] == -math.inf).all()
        got, gl = kv.attention(b.q, b.cu, b.len, max_q=max_q, window=100, with_lse=True)
        assert (got == 0).all() and (gl == -math.inf).all()
        kv.read_status()
        before = b.mass.clone()
        kv.attention_mass(b.q, lse, b.cu, b.len, max_q=max_q)
        check_mass(b, 0, before, b.mass, lse, 1.0)
        assert kv.read_status() == pp_().PP_S_INDEX
        K, V, M = b.k.clone(), b.v.clone(), b.mass.clone()
        kv2 = pp_().PagedKV(K, V, b.table, mass=M)
        kv2.append(b.q, b.q[:, :2], b.q[:, :2], b.cu, b.len)
        assert kv2.read_status() == pp_().PP_S_INDEX
        assert torch.equal(K, b.k) and torch.equal(V, b.v) and torch.equal(M, b.mass)


def test_evict_reports_a_length_past_the_table():
    b = Batch(BF16, 64, 2, 1, 16, [0, 0], [320, 100])
    want = b.kv().evict(b.len, 50, 7, other(b, 50))
    b.len[0] = 333
    kv = b.kv()
    got = kv.evict(b.len, 50, 7, other(b, 50))
    assert kv.read_status() == pp_().PP_S_INDEX
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def other(b, budget):
    need = -(-budget // b.page)
    n = need * len(b.lens)
    K = torch.zeros((n, b.Hk, b.page, b.D), dtype=b.type, device="cuda")
    table = torch.arange(n, dtype=torch.int32, device="cuda").view(len(b.lens), need)
    return pp_().PagedKV(K, K.clone(), table, mass=torch.zeros(K.shape[:3], device="cuda"))


# ---- values that are not finite -----------------------------------------------------------------

@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("n,max_q", [(1, 1), (3, 3), (40, 40), (200, 200)])
@pytest.mark.parametrize("entry", [5, 2000])
def test_a_value_that_a_row_sees_is_not_lost_by_its_small_weight(entry, n, max_q, bad):
    """A key whose score lies 2^-1000 below the others', in another split of the keys than theirs or
    in the same one: its weight is 0 in fp32, its value all the same not finite."""
    b = Batch(BF16, 128, 2, 1, 64, [n], [3000])
    b.k.mul_(0.01)
    b.q.fill_(1.0)
    p, r = b.where(0)
    near = slice(max(0, entry - 600), entry + 600)     # its split: as unlikely all of it
    b.k[p[near], :, r[near]] = -64.0                   # a score of -64 sqrt(128)
    want, _ = b.kv().attention(b.q, b.cu, b.len, max_q=max_q, with_lse=True)
    assert torch.isfinite(want).all()
    v = b.v.clone()
    v[p[entry], :, r[entry], 3] = bad
    got, _ = pp_().PagedKV(b.k, v, b.table).attention(b.q, b.cu, b.len, max_q=max_q, with_lse=True)
    assert not torch.isfinite(got[..., 3]).any()
    ok = torch.ones_like(got, dtype=torch.bool)
    ok[..., 3] = False
    assert torch.equal(got[ok], want[ok])


# ---- a sequence's bits ---------------------------------------------------------------------------

def alone(b, s, max_q, window=0):
    a, e = b.at[s], b.at[s + 1]
    kv = pp_().PagedKV(b.k, b.v, b.table[s:s + 1].contiguous())
    return kv.attention(b.q[a:e], b.cu[s:s + 2] - a, b.len[s:s + 1], max_q=max_q, window=window,
                        with_lse=True)


@pytest.mark.parametrize("type,D,Hk,G,window", [(BF16, 128, 8, 1, 0), (F16, 64, 16, 2, 0),
                                                (BF16, 64, 8, 4, 700)])
def test_bits_do_not_depend_on_what_an_sm_has_done_before(type, D, Hk, G, window):
    """Many short units to a CTA, most with an odd number of tiles."""
    n = 64
    lens = [1 + (s * 389) % 1900 for s in range(n)]
    b = Batch(type, D, Hk, G, 64, [1] * n, lens, window=window)
    out, lse = b.kv().attention(b.q, b.cu, b.len, max_q=1, window=window, with_lse=True)
    b.check(out, lse)
    for s in range(n):
        one, l = alone(b, s, 1, window)
        assert torch.equal(one, out[s:s + 1]) and torch.equal(l, lse[s:s + 1]), s


def test_the_same_call_gives_the_same_bits():
    x = Batch(BF16, 128, 8, 1, 64, [1] * 40, [3000 - 61 * i for i in range(40)])
    y = Batch(F16, 128, 2, 4, 16, [5, 1, 8, 3], [9000, 20000, 700, 5000])
    z = Batch(BF16, 64, 2, 3, 32, [700, 1, 90, 300], [5000, 3000, 90, 2000], window=1000)
    noise = torch.randn((4096, 4096), device="cuda")
    for b in (x, y, z):
        kv, n = b.kv(), max(b.chunks)
        got = []
        for i in range(6):
            if i & 1:
                noise = noise @ noise / 64
            o, l = kv.attention(b.q, b.cu, b.len, max_q=n, window=b.window, with_lse=True)
            m = torch.ones_like(b.mass)
            kv.attention_mass(b.q, l, b.cu, b.len, max_q=n, window=b.window, mass=m)
            got.append((o, l, m))
        for g in got[1:]:
            assert all(torch.equal(p, q) for p, q in zip(g, got[0]))


# ---- the caller's max_q ----------------------------------------------------------------------------

@pytest.mark.parametrize("G,max_q,chunks,window", [
    (4, 8, [4, 1, 8, 2, 1], 0), (4, 8, [4, 1, 8, 2, 1], 300), (8, 5, [1, 5, 1, 3, 1], 0),
    (1, 40, [1, 3, 40, 16, 33], 0), (2, 7, [7, 1, 1, 1, 5], 129)])
def test_bits_follow_the_callers_max_q(G, max_q, chunks, window):
    """The wrapper hands on the max_q that it is given, however few rows the call has.  (Chunks of
    more than 32 rows to a key head: compared one sequence to a call, in which nothing else sets
    the splits.)"""
    lens = [900, 77, 3000, 300, 1500]
    b = Batch(BF16, 128, 2, G, 64, chunks, lens, window=window)
    out, lse = b.kv().attention(b.q, b.cu, b.len, max_q=max_q, window=window, with_lse=True)
    b.check(out, lse)
    for s in range(len(chunks)):
        one, l = alone(b, s, max_q, window)
        if max_q * G <= 32:
            assert torch.equal(one, out[b.at[s]:b.at[s + 1]]), s
            assert torch.equal(l, lse[b.at[s]:b.at[s + 1]]), s
        # the same through the C call, which knows nothing of the wrapper
        a, e = b.at[s], b.at[s + 1]
        pp, T = pp_(), e - a
        kv = pp.PagedKV(b.k, b.v, b.table[s:s + 1].contiguous())
        size = pp.pp_paged_attention_scratch_bytes(kv.c, b.H, T, max_q, window)
        scratch = torch.empty(size, dtype=torch.uint8, device="cuda")
        o2, l2 = torch.empty_like(one), torch.empty_like(l)
        cu = (b.cu[s:s + 2] - a).contiguous()
        pp.pp_paged_attention(kv.c, b.q[a:e].data_ptr(), b.H * b.D, cu.data_ptr(),
                              b.len[s:s + 1].data_ptr(), T, max_q, b.H, b.scale, window,
                              o2.data_ptr(), l2.data_ptr(), kv.status.data_ptr(), scratch.data_ptr(),
                              size, torch.cuda.current_stream().cuda_stream)
        assert torch.equal(one, o2) and torch.equal(l, l2), s


# ---- rows that give nothing ----------------------------------------------------------------------

@pytest.mark.parametrize("type,D,G,chunks,lens", [
    (BF16, 128, 1, [1, 1], [700, 130]), (F16, 64, 4, [32, 5], [900, 300]),
    (BF16, 128, 2, [64, 200], [1500, 700]), (BF16, 64, 3, [300, 40], [400, 2000])])
@pytest.mark.parametrize("window", [0, 200])
def test_a_row_without_a_sum_gives_nothing_whatever_it_holds(type, D, G, chunks, lens, window):
    """Rows with an lse of -infinity, as a caller marks rows of padding, whose queries may be
    anything."""
    b = Batch(type, D, 2, G, 32, chunks, lens, window=window)
    kv = b.kv()
    _, lse = kv.attention(b.q, b.cu, b.len, window=window, with_lse=True)
    dead = torch.rand(b.T, generator=b.g, device="cuda") < 0.4
    dead[0] = True
    lse[dead] = -math.inf
    want = torch.zeros_like(b.mass)
    kv.attention_mass(b.q, lse, b.cu, b.len, window=window, mass=want)
    for s in range(2):
        check_mass(b, s, torch.zeros_like(want), want, lse, 1.0)
    for bad in (math.nan, math.inf, -math.inf, torch.finfo(type).max):
        q = b.q.clone()
        q[dead] = bad
        got = torch.zeros_like(b.mass)
        kv.attention_mass(q, lse, b.cu, b.len, window=window, mass=got)
        assert torch.equal(got, want), bad


@pytest.mark.parametrize("G,max_q", [(1, 8), (4, 40)])
def test_the_entries_of_padding_rows_stay_empty(G, max_q):
    """The last rows of a chunk are padding: neither their queries nor their keys are finite, and
    they alone see these keys."""
    b = Batch(BF16, 128, 2, G, 32, [40, 5], [500, 300])
    kv, live = b.kv(), 30
    _, lse = kv.attention(b.q, b.cu, b.len, max_q=40, with_lse=True)
    lse[live:40] = -math.inf
    want = torch.zeros_like(b.mass)
    kv.attention_mass(b.q, lse, b.cu, b.len, max_q=max_q, mass=want)
    p, r = (t[-10:] for t in b.where(0))
    assert (want[p, :, r] == 0).all()
    b.q[live:40] = math.nan
    b.k[p, :, r] = math.nan
    got = torch.zeros_like(b.mass)
    kv.attention_mass(b.q, lse, b.cu, b.len, max_q=max_q, mass=got)
    assert torch.equal(got, want)


# ---- weights under a window ---------------------------------------------------------------------

@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0])
@pytest.mark.parametrize("G,chunks,lens,window", [
    (1, [1, 1, 0], [9000, 100, 600], 300), (4, [70, 5], [20000, 700], 500),
    (2, [600, 0, 200], [5000, 300, 200], 257), (8, [33], [3000], 1)])
def test_weights_under_a_window_over_a_long_cache(G, chunks, lens, window, decay):
    """Most entries are seen by no row: they decay and nothing else."""
    b = Batch(BF16, 64, 3, G, 64, chunks, lens, window=window)
    kv = b.kv()
    _, lse = kv.attention(b.q, b.cu, b.len, max_q=max(chunks), window=window, with_lse=True)
    before = b.mass.clone()
    kv.attention_mass(b.q, lse, b.cu, b.len, max_q=max(chunks), window=window, decay=decay)
    for s, n in enumerate(lens):
        check_mass(b, s, before, b.mass, lse, decay)
        old = max(0, n - chunks[s] - window + 1) if chunks[s] else n
        p, r = (t[:old] for t in b.where(s))
        assert torch.equal(b.mass[p, :, r], before[p, :, r] * decay)


def test_the_weights_cost_what_the_window_sees():
    """The same rows and window over a short cache and over a long one: without a decay the older
    entries are no work, and the rest spreads over the SMs alike (a ratio of 10 when the units that
    no row sees counted as much as the others)."""
    times = []
    for n in (5120, 65000):
        b = Batch(BF16, 128, 8, 4, 64, [4096], [n], window=1000)
        kv = b.kv()
        lse = torch.full((4096, 32), 8.0, device="cuda")
        best = math.inf
        for _ in range(5):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            for _ in range(20):
                kv.attention_mass(b.q, lse, b.cu, b.len, max_q=4096, window=1000)
            end.record()
            torch.cuda.synchronize()
            best = min(best, start.elapsed_time(end))
        times.append(best)
    assert times[1] < 3 * times[0], times


# ---- several host threads --------------------------------------------------------------------------

def test_host_threads_do_not_disturb_each_other():
    """Two threads, each with its own stream and caches; the shared memory that their launches ask
    for differs with the number of sequences, the rows of a step and the width of the table."""
    pp = pp_()
    L, rounds = pp.lib(), 3000

    def calls(n, entries, heads, max_q):
        k = torch.randn((n + 1, 1, 64, 128), device="cuda").to(BF16)
        width = entries // 64
        table = torch.zeros((n, width), dtype=torch.int32, device="cuda")
        table[:, 0] = torch.arange(n, device="cuda")
        kv = pp.PagedKV(k, k.clone(), table, mass=torch.zeros((n + 1, 1, 64), device="cuda"))
        to = pp.PagedKV(k.clone(), k.clone(), table, mass=torch.zeros((n + 1, 1, 64), device="cuda"))
        cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
        length = torch.full((n,), 9, dtype=torch.int32, device="cuda")
        q = torch.randn((n, heads, 128), device="cuda").to(BF16)
        out, lse = torch.empty_like(q), torch.zeros((n, heads), device="cuda")
        size = pp.pp_paged_attention_scratch_bytes(kv.c, heads, n, max_q, 0)
        scratch = torch.empty(size, dtype=torch.uint8, device="cuda")
        to_len = torch.empty(n, dtype=torch.int32, device="cuda")
        kept = torch.empty((n, 1, 8), dtype=torch.int32, device="cuda")
        stream = torch.cuda.Stream()
        ref, tref, s = ctypes.byref(kv.c), ctypes.byref(to.c), stream.cuda_stream
        keep = (kv, to, cu, length, q, out, lse, scratch, to_len, kept, stream)

        def go():
            st = kv.status.data_ptr()
            return (L.pp_paged_attention(ref, q.data_ptr(), heads * 128, cu.data_ptr(),
                                         length.data_ptr(), n, max_q, heads, 0.1, 0, out.data_ptr(),
                                         lse.data_ptr(), st, scratch.data_ptr(), size, s),
                    L.pp_paged_mass(ref, q.data_ptr(), heads * 128, lse.data_ptr(), cu.data_ptr(),
                                    length.data_ptr(), n, max_q, heads, 0.1, 0, 0.5, st, s),
                    L.pp_paged_evict(ref, length.data_ptr(), 8, 2, tref, to_len.data_ptr(),
                                     kept.data_ptr(), st, s))
        return go, keep

    # (the tables' unused entries are never looked at: nine entries to a sequence)
    sides = [calls(1, 64, 1, 1), calls(48, 1 << 19, 2, 1)]
    torch.cuda.synchronize()
    wrong = [[], []]

    def work(i):
        torch.cuda.set_device(0)
        for _ in range(rounds):
            rc = sides[i][0]()
            if any(rc):
                wrong[i].append(rc)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong[0] and not wrong[1], (len(wrong[0]), wrong[0][:3], len(wrong[1]), wrong[1][:3])
    for _, keep in sides:
        assert keep[0].read_status() == 0


# ---- sizes that no other test reaches -----------------------------------------------------------------

@pytest.mark.parametrize("lens,budget,recent", [([400000], 150000, 1000), ([400000, 5], 3, 0)])
def test_evict_of_rows_too_long_for_shared_memory(lens, budget, recent):
    """More than 8 x 45056 entries to a key head: each round reads the weights again."""
    b = Batch(BF16, 64, 1, 1, 256, [0] * len(lens), lens)
    b.mass.mul_(500).round_()                    # ties, at the threshold too
    run_evict(b, budget, recent, 256)


def test_long_chunks_of_very_different_lengths():
    """More units than SMs: one of 20000 entries beside chunks of 33 to 64 tokens."""
    chunks = [33 + (i * 7) % 32 for i in range(100)]
    lens = [c + (i * 13) % 50 for i, c in enumerate(chunks)]
    lens[40] = 20000
    lens[99] = 9000
    b = Batch(BF16, 64, 4, 1, 64, chunks, lens)
    out, lse = b.kv().attention(b.q, b.cu, b.len, max_q=64, with_lse=True)
    b.check(out, lse)


@pytest.mark.parametrize("type,D,chunks,lens", [(BF16, 128, [1], [60000]), (F16, 64, [1, 2], [30000, 900]),
                                                (BF16, 128, [3, 1], [500, 20000])])
def test_many_query_heads_over_a_long_cache(type, D, chunks, lens):
    b = Batch(type, D, 1, 64, 64, chunks, lens)
    kv = b.kv()
    out, lse = kv.attention(b.q, b.cu, b.len, max_q=max(chunks), with_lse=True)
    b.check(out, lse)
    before = b.mass.clone()
    kv.attention_mass(b.q, lse, b.cu, b.len, max_q=max(chunks))
    for s in range(len(lens)):
        check_mass(b, s, before, b.mass, lse, 1.0)
