"""The paged-cache operators (pp_paged_append, pp_paged_attention, pp_paged_mass,
pp_paged_evict) against plain 64-bit arithmetic on the same inputs (GPU).

Tolerances count roundings.  A result rounded to type t is off by at most eps_t / 2 of its
value.  In the attention each softmax weight is rounded once to the cache's type before the
second product: eps_t / 2 of sum_j w_j |v_j|.  Scores are sums of D exact products in fp32: off by
at most D 2^-23 scale sum|q k|, which the exponential turns into a relative error of the
weights; the sums over n entries add n 2^-23.  fp16 weights below their normal range are off by
2^-25 absolutely, on weights scaled up by 2^7.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def pp_():
    import full_duplex_speech_lockstep_gb300 as pp
    return pp


class Batch:
    """A seeded cache with shuffled pages, new rows, and plain 64-bit results."""

    def __init__(self, type, D, Hk, G, page, chunks, lens, seed=1, window=0, pad=0, lead=0,
                 width=0, joint=False, spare=1, stride_pages=1):
        self.type, self.D, self.Hk, self.G, self.page = type, D, Hk, G, page
        self.H, self.window = Hk * G, window
        self.chunks, self.lens = chunks, lens
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g = g
        need = [-(-n // page) for n in lens]
        self.n_pages = sum(need) + spare
        order = torch.randperm(self.n_pages, generator=g, device="cuda").int()
        self.table = torch.full((len(lens), max(1, max(need), width)), -7, dtype=torch.int32,
                                device="cuda")
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        shape = (self.n_pages, stride_pages, Hk, page, D)
        self.k = torch.randn(shape, generator=g, device="cuda").to(type)[:, 0]
        self.v = torch.randn(shape, generator=g, device="cuda").to(type)[:, 0]
        self.mass = torch.rand((self.n_pages, Hk, page), generator=g, device="cuda")
        cu = [lead]
        for c in chunks:
            cu.append(cu[-1] + c)
        self.at, self.T = cu, cu[-1] + pad
        self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        rows = torch.randn((self.T, self.H + (5 if joint else 0), D), generator=g,
                           device="cuda").to(type)
        self.q = rows[:, :self.H]
        self.scale = D ** -0.5

    def kv(self, **kw):
        return pp_().PagedKV(self.k, self.v, self.table, mass=self.mass, **kw)

    def where(self, b, table=None, n=None, page=None):
        page = page or self.page
        j = torch.arange(self.lens[b] if n is None else n, device="cuda")
        return (self.table if table is None else table)[b].long()[j // page], j % page

    def entries(self, pool, b):
        p, r = self.where(b)
        return pool[p, :, r].double().transpose(0, 1)           # [Hk, len, ...]

    def sees(self, b):
        n, total = self.chunks[b], self.lens[b]
        p = torch.arange(total - n, total, device="cuda")[:, None]
        j = torch.arange(total, device="cuda")[None]
        m = j <= p
        return m & (j > p - self.window) if self.window else m

    def scores(self, b):
        a, n = self.at[b], self.chunks[b]
        q = self.q[a:a + n].double().transpose(0, 1).unflatten(0, (self.Hk, self.G))
        k = self.entries(self.k, b)[:, None]
        s = (q @ k.transpose(-1, -2)) * self.scale
        size = (q.abs() @ k.abs().transpose(-1, -2)) * self.scale
        see = self.sees(b)
        return s.masked_fill(~see, -math.inf), size.masked_fill(~see, 0)

    def attention(self, b):
        """out, lse and their error bounds for sequence b: [n, H, D] and [n, H]."""
        s, size = self.scores(b)
        v = self.entries(self.v, b)[:, None]
        empty = ~self.sees(b).any(-1)
        lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full(s.shape[:-1], -math.inf,
                                                                   device="cuda").double()
        w = torch.exp(s - lse.masked_fill(empty, 0)[..., None]).masked_fill(
            ~self.sees(b), 0)
        out = w @ v
        half = torch.finfo(self.type).eps / 2
        n = max(1, s.shape[-1])
        ds = self.D * 2.0 ** -23 * (size.amax(-1) if s.shape[-1] else 0) + n * 2.0 ** -23 + 2.0 ** -21
        mass = w @ v.abs()
        tol = half * out.abs() + (half + 2 * ds[..., None] if torch.is_tensor(ds) else half) * mass
        if self.type == F16 and s.shape[-1]:
            tol = tol + n * 2.0 ** -31 * v.abs().amax()
        back = lambda t: t.flatten(0, 1).transpose(0, 1)
        ltol = ds + 2.0 ** -22 * (1 + lse.abs().masked_fill(empty, 0))
        return back(out), back(lse), back(tol + 1e-30), back(ltol.expand(lse.shape))

    def check(self, out, lse):
        for b in range(len(self.lens)):
            if self.chunks[b] == 0:
                continue
            a, n = self.at[b], self.chunks[b]
            o, l, tol, ltol = self.attention(b)
            err = (out[a:a + n].double() - o).abs()
            assert not torch.isnan(out[a:a + n]).any(), b
            assert (err <= tol).all(), (b, float((err / tol).max()))
            got = lse[a:a + n].double()
            dead = l == -math.inf
            assert (got[dead] == -math.inf).all() and (out[a:a + n][dead] == 0).all()
            assert ((got - l).abs()[~dead] <= ltol[~dead]).all(), b


SHAPES = [  # type, D, Hk, G, page, chunks, lens, window
    (BF16, 128, 2, 1, 64, [1, 1, 1], [3000, 1, 129], 0),
    (BF16, 128, 3, 4, 16, [1, 1, 0, 1], [777, 16, 50, 5000], 0),
    (F16, 128, 1, 8, 32, [1, 2, 5], [100, 2, 1500], 0),
    (BF16, 64, 2, 3, 128, [4, 1, 7, 2], [4, 300, 1025, 128], 0),
    (F16, 64, 5, 7, 256, [1, 9], [513, 2600], 0),
    (BF16, 128, 1, 16, 64, [1, 1], [257, 40000], 0),
    (BF16, 64, 1, 64, 16, [1, 3], [90, 400], 0),
    (BF16, 128, 2, 4, 64, [37, 200, 0, 1], [37, 1000, 10, 128], 0),
    (F16, 128, 1, 2, 16, [333, 1], [700, 260], 0),
    (BF16, 64, 3, 5, 32, [129, 64, 65], [129, 64, 2000], 0),
    (F16, 64, 1, 1, 256, [1000], [1000], 0),
    (BF16, 128, 1, 3, 64, [600, 3], [1400, 2500], 0),
    # windows, also of one entry and next to a tile's end
    (BF16, 128, 2, 2, 64, [1, 1, 4], [3000, 100, 1200], 1),
    (BF16, 128, 2, 2, 64, [1, 1, 4], [3000, 100, 1200], 127),
    (F16, 64, 2, 1, 16, [50, 3, 1], [900, 700, 130], 129),
    (BF16, 128, 1, 4, 32, [300, 1], [2000, 1999], 500),
    (BF16, 64, 1, 2, 128, [300, 257], [300, 3000], 64),
    # rows without an entry: more new rows than entries, and no entry at all
    (BF16, 128, 2, 2, 64, [5, 3, 1], [2, 0, 0], 0),
    (F16, 64, 1, 4, 16, [200, 150], [40, 0], 0),
]


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "-".join(str(x) for x in c[1:]))
def test_attention(case):
    type, D, Hk, G, page, chunks, lens, window = case
    b = Batch(type, D, Hk, G, page, chunks, lens, window=window)
    kv = b.kv()
    for max_q in (max(chunks), None):
        out, lse = kv.attention(b.q, b.cu, b.len, max_q=max_q, window=window, with_lse=True)
        b.check(out, lse)
    # a hint that is too small changes speed only
    out, lse = kv.attention(b.q, b.cu, b.len, max_q=1, window=window, with_lse=True)
    b.check(out, lse)
    assert kv.read_status() == 0


def test_attention_of_large_scores_and_scales():
    b = Batch(BF16, 128, 2, 2, 64, [70, 1], [500, 3000], seed=5)
    b.q.mul_(12)
    b.scale = 0.3
    out, lse = b.kv().attention(b.q, b.cu, b.len, scale=0.3, with_lse=True)
    b.check(out, lse)


@pytest.mark.parametrize("chunks,lens", [([1, 1], [130, 3000]), ([9, 300], [200, 1000])])
def test_padding_rows_are_left_alone(chunks, lens):
    b = Batch(BF16, 128, 2, 4, 64, chunks, lens, pad=7, lead=3)
    out = torch.full((b.T, b.H, b.D), 7.0, dtype=b.type, device="cuda")
    _, lse = b.kv().attention(b.q, b.cu, b.len, with_lse=True, out=out)
    b.check(out, lse)
    assert (out[:3] == 7).all() and (out[-7:] == 7).all()


@pytest.mark.parametrize("D,type", [(128, BF16), (64, F16)])
@pytest.mark.parametrize("chunks,lens,window", [([1, 1], [130, 3000], 0), ([1, 4], [260, 700], 100),
                                                ([200, 3], [600, 300], 0),
                                                ([150, 300], [150, 900], 60)])
def test_what_a_row_does_not_see_never_reaches_it(D, type, chunks, lens, window):
    """Stale rows, unused pages and later or older entries may hold anything."""
    b = Batch(type, D, 2, 2, 32, chunks, lens, window=window)
    want, wl = b.kv().attention(b.q, b.cu, b.len, window=window, with_lse=True)
    live = torch.zeros(b.k.shape[0], b.page, dtype=torch.bool, device="cuda")
    for s in range(len(lens)):
        p, r = b.where(s)
        live[p, r] = True
        if window:      # entries that even the first row no longer sees
            old = max(0, lens[s] - chunks[s] - window + 1)
            live[p[:old], r[:old]] = False
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(type).max):
        k, v = b.k.clone(), b.v.clone()
        k.transpose(1, 2)[~live] = bad
        v.transpose(1, 2)[~live] = bad
        got, gl = pp_().PagedKV(k, v, b.table).attention(b.q, b.cu, b.len, window=window,
                                                         with_lse=True)
        assert torch.equal(got, want) and torch.equal(gl, wl), bad
    # one entry inside a chunk: only the rows that see it change, and they get what the sum gives
    for s in range(len(lens)):
        if chunks[s] < 3:
            continue
        i = chunks[s] // 2
        j = lens[s] - chunks[s] + i
        p, r = b.where(s)
        for bad in (float("nan"), float("inf"), -float("inf")):
            v = b.v.clone()
            v[p[j], :, r[j], 3] = bad
            got, gl = pp_().PagedKV(b.k, v, b.table).attention(b.q, b.cu, b.len, window=window,
                                                               with_lse=True)
            see = torch.zeros(b.T, dtype=torch.bool, device="cuda")
            last = chunks[s] if not window else min(chunks[s], i + window)
            see[b.at[s] + i:b.at[s] + last] = True
            ok = torch.ones_like(got, dtype=torch.bool)
            ok[see, :, 3] = False
            assert torch.equal(got[ok], want[ok]) and torch.equal(gl, wl)
            hit = got[see][:, :, 3]
            assert torch.isnan(hit).all() if bad != bad else (hit == bad).all()
            k = b.k.clone()
            k[p[j], :, r[j]] = float("nan")
            got, gl = pp_().PagedKV(k, b.v, b.table).attention(b.q, b.cu, b.len, window=window,
                                                               with_lse=True)
            assert torch.equal(got[~see], want[~see]) and torch.equal(gl[~see], wl[~see])
            assert torch.isnan(got[see]).all() and torch.isnan(gl[see]).all()


@pytest.mark.parametrize("chunk", [1, 200])
def test_pages_outside_the_pool_take_no_part(chunk):
    b = Batch(BF16, 128, 1, 2, 32, [chunk, chunk], [700, 300])
    b.table[0, 3] = b.n_pages
    b.table[1, 0] = -1
    kv = b.kv()
    out, lse = kv.attention(b.q, b.cu, b.len, with_lse=True)
    kv.attention_mass(b.q, lse, b.cu, b.len, decay=0.0)
    assert kv.read_status() == pp_().PP_S_INDEX and kv.read_status() == 0
    whole = b.sees
    hide = {0: slice(96, 128), 1: slice(0, 32)}

    def sees(s):
        m = whole(s)
        m[:, hide[s]] = False
        return m
    b.sees = sees
    b.table[0, 3] = b.table[1, 0] = 0
    b.check(out, lse)


def test_attention_reads_strided_rows_and_pages():
    b = Batch(BF16, 128, 2, 3, 64, [1, 40], [500, 300], joint=True, stride_pages=2)
    assert b.q.stride(0) > b.H * b.D and b.k.stride(0) > b.Hk * b.page * b.D
    out, lse = b.kv().attention(b.q, b.cu, b.len, with_lse=True)
    b.check(out, lse)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements, its last pages in use."""
    n = 40
    page, D = 256, 128
    stride = (1 << 32) // n + 4096
    stride -= stride % 8
    big = torch.empty((n - 1) * stride + page * D, dtype=BF16, device="cuda")
    b = Batch(BF16, D, 1, 2, page, [3, 150], [600, 800], spare=0)
    k = big.as_strided((n, 1, page, D), (stride, page * D, D, 1))
    v = torch.empty_like(big).as_strided(k.size(), k.stride())
    table = torch.where(b.table >= 0, n - 1 - b.table, b.table)
    for s in range(2):
        old, new = b.table[s][b.table[s] >= 0].long(), table[s][table[s] >= 0].long()
        k[new], v[new] = b.k[old], b.v[old]
    kv = pp_().PagedKV(k, v, table)
    out, lse = kv.attention(b.q, b.cu, b.len, with_lse=True)
    b.check(out, lse)
    x = torch.randn((153, 4, D), device="cuda", dtype=BF16)
    kv.append(x[:, :2], x[:, 2:3], x[:, 3:], b.cu, b.len, rot_dim=0)
    p, r = b.where(1, table)
    assert torch.equal(v[p[-150:], 0, r[-150:]], x[3:, 3])
    assert torch.equal(k[p[-150:], 0, r[-150:]], x[3:, 2])


def test_a_sequence_does_not_depend_on_its_neighbours():
    chunks, lens = [1, 1, 4, 2], [3000, 77, 20000, 300]
    b = Batch(BF16, 128, 2, 4, 64, chunks, lens)
    out, lse = b.kv().attention(b.q, b.cu, b.len, max_q=4, with_lse=True)
    for s in range(4):
        a, e = b.at[s], b.at[s + 1]
        kv = pp_().PagedKV(b.k, b.v, b.table[s:s + 1].contiguous())
        one, l = kv.attention(b.q[a:e], b.cu[s:s + 2] - a, b.len[s:s + 1], max_q=4, with_lse=True)
        assert torch.equal(one, out[a:e]) and torch.equal(l, lse[a:e])


def test_many_sequences():
    n = 2048
    chunks = [i % 3 for i in range(n)]
    lens = [(i * 7) % 41 + chunks[i] for i in range(n)]
    b = Batch(BF16, 64, 1, 2, 16, chunks, lens)
    kv = b.kv()
    out, lse = kv.attention(b.q, b.cu, b.len, max_q=2, with_lse=True)
    before = b.mass.clone()
    kv.attention_mass(b.q, lse, b.cu, b.len, max_q=2)
    for s in list(range(0, n, 97)) + [n - 1]:
        if chunks[s]:
            o, l, tol, ltol = b.attention(s)
            a = b.at[s]
            assert ((out[a:a + chunks[s]].double() - o).abs() <= tol).all()
        check_mass(b, s, before, b.mass, lse, 1.0)


@pytest.mark.parametrize("chunk", [1, 300])
def test_graphs_replay_with_new_lengths_and_share_nothing(chunk):
    b = Batch(BF16, 128, 2, 2, 64, [chunk, chunk], [2000, 900])
    kv = b.kv()
    kv.attention(b.q, b.cu, b.len, max_q=chunk)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, l = kv.attention(b.q, b.cu, b.len, max_q=chunk, with_lse=True)
            kv.attention_mass(b.q, l, b.cu, b.len, max_q=chunk, decay=0.0)
        graphs.append(g)
        outs.append((o, l))
    for lens in ([2000, 900], [chunk, 900], [1500, chunk]):
        b.lens = lens
        b.len.copy_(torch.tensor(lens, dtype=torch.int32))
        streams = [torch.cuda.Stream() for _ in graphs]
        torch.cuda.synchronize()
        # replayed one after the other (both write one mass), each on its own stream
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
            s.synchronize()
        for o, l in outs:
            b.check(o, l)


@pytest.mark.parametrize("G,n", [(1, 1), (2, 40)])
def test_sequences_share_the_pages_of_a_common_prompt(G, n):
    b = Batch(BF16, 128, 2, G, 64, [n, n, n], [700, 900, 600])
    b.table[1:, :8] = b.table[0, :8]
    out, lse = b.kv().attention(b.q, b.cu, b.len, with_lse=True)
    b.check(out, lse)


def guarded(shape, type, fill):
    """A tensor with a guard behind it, and a check that the guard is untouched."""
    n = math.prod(shape)
    whole = torch.full((n + (1 << 20),), fill, dtype=type, device="cuda")

    def intact():
        return bool((whole[n:] == fill).all())
    return whole[:n].view(shape), intact


@pytest.mark.parametrize("T,page,n", [(6, 16, 1500), (2560, 64, 1500)])
def test_row_offsets_that_fall_touch_nothing_else(T, page, n):
    """Sequences 0, 2 and 4 are all given every row, so the call holds more units than T rows
    make: outputs and scratch keep to their bounds, and what has no part in it stays."""
    pp = pp_()
    b = Batch(BF16, 128, 1, 1, page, [T], [n] * 6, pad=2)
    cu = torch.tensor([0, T, 0, T, 0, T, 0], dtype=torch.int32, device="cuda")
    kv = b.kv()
    rows = b.T
    stream = torch.cuda.current_stream().cuda_stream
    size = pp.pp_paged_attention_scratch_bytes(kv.c, 1, rows, T, 0)
    scratch, scratch_ok = guarded((size,), torch.uint8, 77)
    out, out_ok = guarded((rows, 1, 128), BF16, 3.0)
    lse, lse_ok = guarded((rows, 1), F32, 3.0)
    k0, v0, mass0 = b.k.clone(), b.v.clone(), b.mass.clone()
    pp.pp_paged_attention(kv.c, b.q.data_ptr(), 128, cu.data_ptr(), b.len.data_ptr(), rows, T,
                          1, b.scale, 0, out.data_ptr(), lse.data_ptr(), 0, scratch.data_ptr(), size,
                          stream)
    torch.cuda.synchronize()
    assert scratch_ok() and out_ok() and lse_ok()
    assert (out[T:] == 3).all() and (lse[T:] == 3).all()
    assert torch.equal(b.k, k0) and torch.equal(b.v, v0) and torch.equal(b.mass, mass0)

    pp.pp_paged_mass(kv.c, b.q.data_ptr(), 128, lse.data_ptr(), cu.data_ptr(),
                     b.len.data_ptr(), rows, T, 1, b.scale, 0, 1.0, 0, stream)
    x, x_ok = guarded((rows, 1, 128), BF16, 3.0)
    pp.pp_paged_append(kv.c, b.q.data_ptr(), 128, b.q.data_ptr(), 128, b.q.data_ptr(), 128,
                       pp.PP_BF16, 0, 0, 1e-5, 1e4, 128, 0, 0, cu.data_ptr(), b.len.data_ptr(),
                       rows, 1, x.data_ptr(), 0, stream)
    torch.cuda.synchronize()
    assert x_ok() and (x[T:] == 3).all()
    for s in (1, 3, 5):                      # no rows: nothing of theirs has changed
        p, r = b.where(s)
        for new, old in ((b.k, k0), (b.v, v0)):
            assert torch.equal(new[p, :, r], old[p, :, r])
        assert torch.equal(b.mass[p, :, r], mass0[p, :, r])


def test_calls_on_two_streams_at_once():
    x = Batch(BF16, 128, 4, 1, 64, [1] * 8, [3000] * 8, seed=3)
    y = Batch(F16, 64, 2, 4, 32, [100, 7], [4000, 6000], seed=4)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    kx, ky = x.kv(), y.kv()
    torch.cuda.synchronize()
    res = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            a = kx.attention(x.q, x.cu, x.len, max_q=1, with_lse=True)
        with torch.cuda.stream(s2):
            c = ky.attention(y.q, y.cu, y.len, with_lse=True)
        res.append((a, c))
    torch.cuda.synchronize()
    for a, c in res:
        x.check(*a)
        y.check(*c)


# ---- append ------------------------------------------------------------------------------------

def turned(x, alpha, pos, rot, halves, eps=1e-5, base=10000.0):
    x = x.double()
    if alpha is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * alpha.double()
    i = torch.arange(rot // 2, device="cuda").double()
    z = torch.polar(torch.ones((), device="cuda").double(),
                    pos.double()[:, None] * base ** (-2 * i / max(rot, 1)))[:, None]
    a, b = ((x[..., :rot // 2], x[..., rot // 2:rot]) if halves else
            (x[..., 0:rot:2], x[..., 1:rot:2]))
    y = torch.complex(a, b) * z
    out = x.clone()
    if halves:
        out[..., :rot // 2], out[..., rot // 2:rot] = y.real, y.imag
    else:
        out[..., 0:rot:2], out[..., 1:rot:2] = y.real, y.imag
    # fp32: the norm's scale is off by a few 2^-24 (D + 8 for the sum), the cosine and sine by
    # 2^-22 (their angle is below pi and off by pi 2^-24 2)
    size = x.abs()
    pair = size.clone()
    if halves:
        pair[..., :rot // 2] += size[..., rot // 2:rot]
        pair[..., rot // 2:rot] += size[..., :rot // 2]
    else:
        pair[..., 0:rot:2] += size[..., 1:rot:2]
        pair[..., 1:rot:2] += size[..., 0:rot:2]
    return out, (x.shape[-1] + 32) * 2.0 ** -24 * pair


@pytest.mark.parametrize("D,rot,halves", [(128, 128, False), (128, 128, True), (128, 64, True),
                                          (128, 2, False), (128, 94, True), (128, 0, False),
                                          (64, 64, False), (64, 64, True), (64, 50, True),
                                          (64, 30, False)])
@pytest.mark.parametrize("type,src", [(BF16, F32), (BF16, BF16), (F16, F16), (F16, F32)])
def test_append(D, rot, halves, type, src):
    chunks, lens = [3, 0, 1, 40, 5], [3, 100, 1, 700, 2]
    b = Batch(type, D, 3, 5, 16, chunks, lens, pad=4, lead=2)
    g = b.g
    x = (torch.randn((b.T, (b.H + 2 * b.Hk) * D), generator=g, device="cuda") * 3).to(src)
    q, k, v = (t.unflatten(1, (-1, D)) for t in x.split([b.H * D, b.Hk * D, b.Hk * D], 1))
    qa = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")
    ka = 1 + 0.3 * torch.randn(D, generator=g, device="cuda")
    half = torch.finfo(type).eps / 2
    tiny = torch.finfo(type).smallest_normal * half
    for alphas in ((qa, ka), (None, None), (None, ka)):
        for far in (0, 1000003, 2 ** 31 - 1000, -70000):
            own = far == 0
            pos = torch.zeros(b.T, dtype=torch.int32, device="cuda")
            for s in range(len(lens)):
                a = b.at[s]
                pos[a:a + chunks[s]] = torch.arange(lens[s] - chunks[s], lens[s],
                                                    device="cuda") + far
            K, V, M = b.k.clone(), b.v.clone(), b.mass.clone()
            kv = pp_().PagedKV(K, V, b.table, mass=M)
            out = torch.full((b.T, b.H, D), 3.0, dtype=type, device="cuda")
            got = kv.append(q, k, v, b.cu, b.len, positions=None if own else pos,
                            q_alpha=alphas[0], k_alpha=alphas[1], rot_dim=rot, halves=halves,
                            out=out)
            assert got is out and kv.read_status() == 0
            rows = slice(2, b.T - 4)
            want, tol = turned(q, alphas[0], pos, rot, halves)
            err = (got.double() - want).abs() - tol - half * want.abs() - tiny
            assert (err[rows] <= 0).all(), (far, float(err[rows].max()))
            assert (out[:2] == 3).all() and (out[-4:] == 3).all()
            kw, ktol = turned(k, alphas[1], pos, rot, halves)
            touched = torch.zeros(b.n_pages, b.page, dtype=torch.bool, device="cuda")
            for s in range(len(lens)):
                n = min(chunks[s], lens[s])          # the others have no entry
                if n == 0:
                    continue
                a = b.at[s] + chunks[s]
                p, r = (t[-n:] for t in b.where(s))
                touched[p, r] = True
                w = kw[a - n:a]
                assert ((K[p, :, r].double() - w).abs() <= ktol[a - n:a] + half * w.abs() + tiny).all()
                assert torch.equal(V[p, :, r], v[a - n:a].to(type))
                assert (M[p, :, r] == 0).all()
            for new, old in ((K, b.k), (V, b.v), (M, b.mass)):
                assert torch.equal(new.transpose(1, 2)[~touched], old.transpose(1, 2)[~touched])


def test_append_in_place_and_without_mass():
    b = Batch(BF16, 128, 2, 2, 64, [5, 1], [90, 64])
    x = torch.randn((6, 4, 128), device="cuda").bfloat16()
    k = torch.randn((6, 2, 128), device="cuda").bfloat16()
    kv = pp_().PagedKV(b.k, b.v, b.table)
    want = kv.append(x, k, k, b.cu, b.len)
    assert torch.equal(kv.append(x, k, k, b.cu, b.len, out=x), want) and want is not x


def test_append_skips_pages_outside_the_pool():
    b = Batch(BF16, 64, 1, 1, 16, [4, 4], [20, 10])
    b.table[0, 1] = b.n_pages + 5
    K, V = b.k.clone(), b.v.clone()
    kv = pp_().PagedKV(K, V, b.table)
    x = torch.ones((8, 1, 64), device="cuda", dtype=BF16)
    kv.append(x, x, x, b.cu, b.len, rot_dim=0)
    assert kv.read_status() == pp_().PP_S_INDEX
    p, r = b.where(1)
    assert (V[p[-4:], 0, r[-4:]] == 1).all()
    V[p[-4:], 0, r[-4:]] = b.v[p[-4:], 0, r[-4:]]
    assert torch.equal(V, b.v)


# ---- mass -----------------------------------------------------------------------------------------

def check_mass(b, s, before, after, lse, decay):
    sc, size = b.scores(s)
    a, n = b.at[s], b.chunks[s]
    l = lse[a:a + n].double().transpose(0, 1).unflatten(0, (b.Hk, b.G))[..., None]
    w = torch.exp(sc - l).masked_fill(l == -math.inf, 0)
    got = b.entries(after, s)
    old = b.entries(before, s) * decay if decay else torch.zeros_like(got)
    want = old + w.sum((1, 2))
    # each weight: the score's rounding, the row sum's and the exponential's (2^-21 and the
    # exponent's own 2^-23 |s - lse|); the additions of n rows and the last one
    rel = b.D * 2.0 ** -23 * size + 2.0 ** -20 + 2.0 ** -22 * (sc - l).abs().masked_fill(w == 0, 0) \
        + 2.0 ** -22 * l.abs().masked_fill(l == -math.inf, 0)
    tol = (w * rel).sum((1, 2)) + (n * b.G + 8) * 2.0 ** -23 * (want + old)
    err = (got - want).abs()
    assert (err <= tol + 1e-30).all(), (s, float((err / (tol + 1e-30)).max()))


@pytest.mark.parametrize("decay", [0.0, 0.7, 1.0])
@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "-".join(str(x) for x in c[1:]))
def test_mass(case, decay):
    type, D, Hk, G, page, chunks, lens, window = case
    b = Batch(type, D, Hk, G, page, chunks, lens, window=window)
    kv = b.kv()
    _, lse = kv.attention(b.q, b.cu, b.len, window=window, with_lse=True)
    if decay == 0:
        b.mass.fill_(float("nan"))
    for max_q in (max(chunks), 1):
        before = b.mass.clone()
        kv.attention_mass(b.q, lse, b.cu, b.len, max_q=max_q, window=window, decay=decay)
        touched = torch.zeros(b.n_pages, page, dtype=torch.bool, device="cuda")
        for s in range(len(lens)):
            check_mass(b, s, before, b.mass, lse, decay)
            touched[b.where(s)] = True
        assert torch.equal(b.mass.transpose(1, 2)[~touched].isnan(),
                           before.transpose(1, 2)[~touched].isnan())
        if decay:
            assert torch.equal(b.mass.transpose(1, 2)[~touched], before.transpose(1, 2)[~touched])
        else:
            again = torch.full_like(b.mass, 5.0)
            kv.attention_mass(b.q, lse, b.cu, b.len, max_q=max_q, window=window, decay=0.0,
                              mass=again)
            assert torch.equal(again.transpose(1, 2)[touched], b.mass.transpose(1, 2)[touched])
    assert kv.read_status() == 0


def test_mass_of_the_last_rows_only_and_of_none():
    b = Batch(BF16, 128, 2, 4, 64, [300, 200], [1000, 200])
    kv = b.kv()
    _, lse = kv.attention(b.q, b.cu, b.len, with_lse=True)
    last = 32
    pick = torch.cat([torch.arange(e - last, e) for e in (300, 500)]).cuda()
    b.q, lse, b.chunks, b.at = b.q[pick], lse[pick], [last, last], [0, last, 2 * last]
    cu = torch.tensor(b.at, dtype=torch.int32, device="cuda")
    before = b.mass.clone()
    kv.attention_mass(b.q, lse, cu, b.len, max_q=last)
    for s in range(2):
        check_mass(b, s, before, b.mass, lse, 1.0)
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    before = b.mass.clone()
    kv.attention_mass(b.q[:0], lse[:0], none, b.len, decay=0.5)
    for s in range(2):
        p, r = b.where(s)
        assert torch.equal(b.mass[p, :, r], before[p, :, r] * 0.5)


def test_mass_does_not_see_what_rows_do_not_see():
    b = Batch(BF16, 64, 1, 2, 32, [150, 3], [400, 300])
    kv = b.kv()
    _, lse = kv.attention(b.q, b.cu, b.len, with_lse=True)
    kv.attention_mass(b.q, lse, b.cu, b.len, decay=0.0)
    live = torch.zeros(b.n_pages, b.page, dtype=torch.bool, device="cuda")
    for s in range(2):
        live[b.where(s)] = True
    k = b.k.clone()
    k.transpose(1, 2)[~live] = float("nan")
    got = torch.zeros_like(b.mass)
    pp_().PagedKV(k, b.v, b.table, mass=got).attention_mass(b.q, lse, b.cu, b.len, decay=0.0)
    assert torch.equal(got.transpose(1, 2)[live], b.mass.transpose(1, 2)[live])


# ---- evict ---------------------------------------------------------------------------------------

def run_evict(b, budget, recent, page, mass=None):
    n = [min(x, budget) for x in b.lens]
    need = [-(-x // page) for x in n]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=b.g, device="cuda").int()
    width = -(-min(budget, b.table.shape[1] * b.page) // page)
    table = torch.full((len(n), width), -3, dtype=torch.int32, device="cuda")
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m]
        at += m
    K = torch.full((pages, b.Hk, page, b.D), 9.0, dtype=b.type, device="cuda")
    V, M = K.clone(), torch.full((pages, b.Hk, page), 9.0, device="cuda")
    to = pp_().PagedKV(K, V, table, mass=M)
    kv = b.kv()
    to_len, kept = kv.evict(b.len, budget, recent, to)
    assert kv.read_status() == 0
    assert to_len.tolist() == n
    touched = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    for s, m in enumerate(n):
        w = b.entries(b.mass, s).cpu()
        safe = min(recent, b.lens[s])
        for h in range(b.Hk):
            key = [(x != x, -x if x == x else 0.0, j) for j, x in enumerate(w[h].tolist())]
            old = sorted(range(b.lens[s] - safe), key=lambda j: key[j])
            want = sorted(old[:m - safe] + list(range(b.lens[s] - safe, b.lens[s])))[:m]
            assert kept[s, h].tolist() == want + [-1] * (budget - m), (s, h)
        p, r = b.where(s, table, m, page)
        touched[p, r] = True
        idx = kept[s, :, :m].long()
        for new, old in ((K, b.k), (V, b.v), (M, b.mass)):
            src = old[b.where(s)[0], :, b.where(s)[1]].transpose(0, 1)
            head = torch.arange(b.Hk, device="cuda")[:, None]
            x, y = new[p, :, r].transpose(0, 1), src[head, idx]
            assert torch.equal(x.view(torch.int16 if x.dtype != F32 else torch.int32),
                               y.contiguous().view(torch.int16 if x.dtype != F32 else torch.int32))
    for new in (K, V, M):
        assert (new.transpose(1, 2)[~touched] == 9).all()


@pytest.mark.parametrize("type,D,Hk,page,lens,budget,recent,to_page", [
    (BF16, 128, 2, 64, [300, 64, 0, 1], 100, 10, 16),
    (F16, 64, 3, 16, [1025, 1024, 1023], 512, 0, 256),
    (BF16, 64, 1, 256, [5000, 4999], 4999, 4999, 64),
    (BF16, 128, 1, 32, [5000, 2], 1, 0, 32),
    (BF16, 128, 1, 32, [5000, 2], 1, 1, 32),
    (F16, 128, 1, 128, [60000, 50001], 20000, 777, 128),
    (BF16, 64, 1, 16, [100, 200], 1000, 100, 16),
])
def test_evict(type, D, Hk, page, lens, budget, recent, to_page):
    b = Batch(type, D, Hk, 1, page, [0] * len(lens), lens)
    run_evict(b, budget, recent, to_page)


def test_evict_breaks_ties_by_index_and_takes_any_weight():
    b = Batch(BF16, 64, 2, 1, 16, [0, 0, 0], [2500, 300, 40])
    b.mass.mul_(4).round_()                      # few distinct values
    run_evict(b, 700, 30, 32)
    b.mass.zero_()
    run_evict(b, 129, 0, 32)
    r = torch.rand(b.mass.shape, generator=b.g, device="cuda")
    b.mass = torch.randn(b.mass.shape, generator=b.g, device="cuda")
    b.mass[r < 0.1] = float("nan")
    b.mass[(r > 0.1) & (r < 0.2)] = float("inf")
    b.mass[(r > 0.2) & (r < 0.3)] = -float("inf")
    b.mass[(r > 0.3) & (r < 0.4)] = -0.0
    b.mass[(r > 0.4) & (r < 0.5)] = 0.0
    b.mass[(r > 0.5) & (r < 0.6)] = 1e-42
    run_evict(b, 1000, 5, 16)
    run_evict(b, 290, 5, 16)


def test_evict_reports_pages_outside_the_pool():
    b = Batch(BF16, 64, 1, 1, 16, [0], [100])
    b.table[0, 2] = -1
    K = torch.zeros((8, 1, 16, 64), dtype=BF16, device="cuda")
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None].contiguous()
    table[0, 1] = 8
    kv = b.kv()
    kv.evict(b.len, 100, 0, pp_().PagedKV(K, K.clone(), table))
    assert kv.read_status() == pp_().PP_S_INDEX


# ---- the calls together ---------------------------------------------------------------------------

@pytest.mark.parametrize("type", [BF16, F16])
def test_a_session_of_chunks_ticks_and_evictions(type):
    """A prompt in two chunks, single tokens, an eviction, more tokens: every attention against
    64-bit arithmetic on the cache as it stands, every weight against the sums so far."""
    pp = pp_()
    D, Hk, G, page, n_seqs = 64, 2, 3, 16, 3
    H, cap = Hk * G, 40
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    pages = n_seqs * cap
    pools = [(torch.zeros((pages, Hk, page, D), dtype=type, device="cuda"),
              torch.zeros((pages, Hk, page, D), dtype=type, device="cuda"),
              torch.full((pages, Hk, page), float("nan"), device="cuda")) for _ in range(2)]
    table = torch.randperm(pages, generator=g, device="cuda").int().view(n_seqs, cap)
    caches = [pp.PagedKV(k, v, table, mass=m) for k, v, m in pools]
    side, lens, pos = 0, [0] * n_seqs, [0] * n_seqs
    total = [torch.zeros((Hk, 0), device="cuda").double() for _ in range(n_seqs)]
    alpha = [1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    steps = [[100, 7, 0], [63, 200, 1], [1, 1, 1], [1, 1, 1], "evict", [1, 1, 1], [5, 0, 90],
             "evict", [1, 1, 1]]
    for step in steps:
        kv = caches[side]
        length = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if step == "evict":
            to_len, kept = kv.evict(length, 120, 16, caches[1 - side])
            side = 1 - side
            lens = to_len.tolist()
            total = [t.gather(1, kept[s, :, :lens[s]].long()) for s, t in enumerate(total)]
            continue
        b = Batch(type, D, Hk, G, page, step, [x + c for x, c in zip(lens, step)], seed=1)
        b.k, b.v, b.mass = pools[side]
        b.table, b.lens = table, [x + c for x, c in zip(lens, step)]
        lens = b.lens
        T = sum(step)
        x = torch.randn((T, H + 2 * Hk, D), generator=g, device="cuda")
        p = torch.cat([torch.arange(q, q + c) for q, c in zip(pos, step)]).int().cuda()
        pos = [q + c for q, c in zip(pos, step)]
        b.q = kv.append(x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], b.cu, b.len, positions=p,
                        q_alpha=alpha[0], k_alpha=alpha[1])
        want, tol = turned(x[:, :H], alpha[0], p, D, False)
        assert ((b.q.double() - want).abs() <= tol + torch.finfo(type).eps / 2 * want.abs()
                + 1e-7).all()
        out, lse = kv.attention(b.q, b.cu, b.len, max_q=max(step), with_lse=True)
        b.check(out, lse)
        before = b.mass.clone()
        kv.attention_mass(b.q, lse, b.cu, b.len, max_q=max(step))
        for s in range(n_seqs):
            check_mass(b, s, before, b.mass, lse, 1.0)
            total[s] = torch.nn.functional.pad(total[s], (0, step[s]))
            if step[s]:
                sc, _ = b.scores(s)
                a = b.at[s]
                l = lse[a:a + step[s]].double().transpose(0, 1).unflatten(0, (Hk, G))[..., None]
                total[s] = total[s] + torch.exp(sc - l).sum((1, 2))
            assert torch.allclose(b.entries(b.mass, s), total[s], rtol=1e-4, atol=1e-5)
        assert kv.read_status() == 0


def test_the_wrapper_refuses_what_does_not_fit():
    pp = pp_()
    b = Batch(BF16, 64, 2, 2, 16, [1, 1], [20, 30])
    kv = b.kv()
    with pytest.raises(ValueError):
        kv.attention(b.q.float(), b.cu, b.len)
    with pytest.raises(ValueError):
        kv.attention(b.q, b.cu.long(), b.len)
    with pytest.raises(ValueError):
        kv.attention(b.q, b.cu[:-1], b.len)
    with pytest.raises(ValueError):
        kv.attention(b.q[..., :32], b.cu, b.len)
    with pytest.raises(ValueError):
        kv.attention(b.q, b.cu.cpu(), b.len)
    with pytest.raises(pp.PPError):
        kv.attention(b.q[:, :3], b.cu, b.len)
    with pytest.raises(pp.PPError):
        kv.attention(b.q, b.cu, b.len, scale=-1.0)
    with pytest.raises(pp.PPError):
        kv.attention(b.q, b.cu, b.len, window=-1)
    with pytest.raises(ValueError):
        pp.PagedKV(b.k, b.v, b.table).attention_mass(b.q, torch.zeros(2, 4, device="cuda"), b.cu,
                                                     b.len)
    with pytest.raises(ValueError):
        pp.PagedKV(b.k.transpose(1, 2), b.v.transpose(1, 2), b.table)
    with pytest.raises(ValueError):
        pp.PagedKV(b.k, b.v.half(), b.table)
    with pytest.raises(pp.PPError):
        kv.evict(b.len, 10, 11, kv)
    with pytest.raises(pp.PPError):
        kv.evict(b.len, 0, 0, kv)
