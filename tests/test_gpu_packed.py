"""The 8-bit paged cache (pp_packed_append, pp_packed_attention, pp_packed_read) against plain 64-bit
arithmetic on the same inputs (GPU).

Tolerances count roundings, as in test_gpu_paged.py, of what the codes stand for.  Beyond those, of the
kernel for short chunks: queries enter the first product as sums of e4m3 numbers of 4 bits each, two for
bf16 (which has 8 bits) and three for fp16 (11), down to a floor of 2^-14 (2^-18) where the row's largest
value is 224 or more: 2^-21 of it.  Softmax weights enter the second product rounded to fp16 (2^-11 of
themselves: eps_t / 2 or less), as three such numbers: below their floor of 2^-18, where a tile's largest
is 256, off by 2^-26 of the row's largest weight.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_paged import BF16, F16, F32, SHAPES, Batch, pp_  # noqa: E402

E4M3 = torch.float8_e4m3fn


def quantise(y):
    """Codes and scale bytes of rows of 64-bit values (finite), as 64-bit codes and integers."""
    a = y.abs().amax(-1)
    e = torch.full(a.shape, -127, dtype=torch.int64, device=y.device)
    for i in range(-126, 130):
        e[a > 448 * 2.0 ** (i - 1)] = i
    x = y * torch.exp2(-e.double())[..., None]
    step = torch.full_like(x, 2.0 ** -9)
    for i in range(-5, 9):
        step[x.abs() >= 2.0 ** i] = 2.0 ** (i - 3)
    return torch.round(x / step) * step, e + 127


def value(codes, byte):
    """What entries read as, in 64 bits."""
    f = torch.exp2(byte.double() - 127)
    f[byte == 255] = math.nan
    return codes.double() * f[..., None]


class Packed(Batch):
    """A Batch whose pages hold 8-bit entries; k and v are what they read as, in 64 bits."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        # entries of very different size
        spread = torch.exp2(torch.randint(-6, 4, self.mass.shape, generator=self.g, device="cuda"))
        for name in "kv":
            c, b = quantise(getattr(self, name).double() * spread[..., None])
            setattr(self, name + "8", self._pool(c.to(E4M3), getattr(self, name)))
            setattr(self, name + "s", b.to(torch.uint8))
            setattr(self, name, value(c, b))

    @staticmethod
    def _pool(codes, like):
        """The codes with pages as far apart as those of `like`."""
        far = like.stride(0) // codes[0].numel()
        pool = torch.zeros((codes.shape[0], far) + tuple(codes.shape[1:]), dtype=E4M3, device="cuda")
        pool.view(torch.uint8)[:, 0] = codes.view(torch.uint8)
        return pool[:, 0]

    def kv(self, **kw):
        return pp_().PagedKV8(self.k8, self.v8, self.ks, self.vs, self.table, dtype=self.type, **kw)

    def attention(self, b):
        out, lse, tol, ltol = super().attention(b)
        a, n = self.at[b], self.chunks[b]
        if self.lens[b]:
            q = self.q[a:a + n].double().abs().amax(-1)                       # [n, H]
            k = self.entries(self.k, b).abs().sum(-1).amax(-1).repeat_interleave(self.G)
            ds = 2.0 ** -21 * self.scale * q * k
            v = self.entries(self.v, b).abs().amax((1, 2)).repeat_interleave(self.G)[None, :, None]
            # a weight is at most 1, and a shift of the scores by ds changes it by 2 ds of itself at most
            tol = tol + (2 * ds[..., None] + self.lens[b] * 2.0 ** -26) * v
            ltol = ltol + ds
        return out, lse, tol, ltol


EDGES = [0.0, -0.0, 1e-45, -3e-39, 2.0 ** -130, 1.75, 1.7500001, 448.0, 449.0, 3.0e38, -3.4e38, 1e-30]


@pytest.mark.parametrize("type,in_type", [(BF16, F32), (BF16, BF16), (F16, F16), (F16, F32)])
@pytest.mark.parametrize("D", [64, 128])
def test_codes_of_plain_rows_are_exact(type, in_type, D):
    """Without norm and rotation: codes and scales by the definition, whatever the rows hold."""
    b = Packed(type, D, 2, 3, 16, [70, 0, 33], [100, 5, 33], lead=2, pad=3, stride_pages=2)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn((b.T, 10, D), generator=g, device="cuda") * torch.exp2(
        torch.randint(-30, 15, (b.T, 10, 1), generator=g, device="cuda"))
    x[5, 6:] = 0
    for i, edge in enumerate(EDGES):        # a row's largest value, all of it, and among others
        x[10 + i, 6] = torch.rand(D, generator=g, device="cuda") * edge
        x[10 + i, 6, i] = edge
        x[10 + i, 7] = edge
        x[10 + i, 8, 3] = edge
    bad = {30: math.nan, 31: math.inf, 32: -math.inf}
    for i, edge in bad.items():
        x[i, 7, D - 1] = edge
    x = x.to(in_type)
    if in_type == F16:
        x[10 + 9:10 + 11] = 1               # (beyond fp16)
    old = [t.clone() for t in (b.k8.view(torch.uint8), b.ks, b.v8.view(torch.uint8), b.vs)]
    kv = b.kv()
    q = kv.append(x[:, :6], x[:, 6:8], x[:, 8:], b.cu, b.len, rot_dim=0)
    assert kv.read_status() == 0
    rows = slice(2, b.T - 3)
    assert torch.equal(q[rows][torch.isfinite(q[rows])], x[rows, :6].to(type)[torch.isfinite(q[rows])])
    for s in (0, 2):
        p, r = (t[b.lens[s] - b.chunks[s]:] for t in b.where(s))
        for name, pool, first in (("k8", old[0], 6), ("v8", old[2], 8)):
            y = x[b.at[s]:b.at[s] + b.chunks[s], first:first + 2].double()
            wild = ~torch.isfinite(y).all(-1)
            codes, byte = quantise(y.masked_fill(wild[..., None], 0))
            byte[wild] = 255
            got = getattr(b, name)[p, :, r]
            assert torch.equal(got.double(), codes)
            assert torch.equal(getattr(b, name[0] + "s")[p, :, r].long(), byte)
            # nothing else changed
            pool[p, :, r] = got.view(torch.uint8)
            (old[1] if name == "k8" else old[3])[p, :, r] = getattr(b, name[0] + "s")[p, :, r]
    for t, o in zip((b.k8.view(torch.uint8), b.ks, b.v8.view(torch.uint8), b.vs), old):
        assert torch.equal(t, o)


@pytest.mark.parametrize("type,in_type,D,rot,halves,norm", [
    (BF16, F32, 128, 128, False, True), (BF16, BF16, 128, 64, True, True),
    (F16, F16, 64, 64, True, False), (F16, F32, 64, 22, True, True), (BF16, BF16, 64, 32, False, False)])
def test_append_with_norm_and_rotation(type, in_type, D, rot, halves, norm):
    b = Packed(type, D, 2, 2, 32, [40, 1, 7], [300, 1, 64])
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    x = (torch.randn((b.T, 8, D), generator=g, device="cuda") * 3).to(in_type)
    alpha = [1 + torch.randn(D, generator=g, device="cuda") / 4 if norm else None for _ in range(2)]
    pos = torch.randint(0, 2 ** 31 - 1, (b.T,), generator=g, device="cuda").int()
    q = b.kv().append(x[:, :4], x[:, 4:6], x[:, 6:], b.cu, b.len, positions=pos, q_alpha=alpha[0],
                      k_alpha=alpha[1], rot_dim=rot, halves=halves)

    def turned(y, alpha):
        y = y.double()
        if alpha is not None:
            y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-5) * alpha.double()
        half = rot // 2
        i = torch.arange(half, device="cuda")
        t = pos.double()[:, None] * 10000.0 ** (-2.0 * i.double() / rot)
        c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
        lo, hi = (i, i + half) if halves else (2 * i, 2 * i + 1)
        z = y.clone()
        z[..., lo] = y[..., lo] * c - y[..., hi] * s
        z[..., hi] = y[..., lo] * s + y[..., hi] * c
        # fp32: the norm to 2^-20, each turn to 2^-21 of its pair (the angle to 2^-20 at 2^31)
        err = 2.0 ** -19 * y.abs()
        for u, w in ((lo, hi), (hi, lo)):
            err[..., u] = 2.0 ** -18 * (y[..., u].abs() + y[..., w].abs())
        return z, err
    want, err = turned(x[:, :4], alpha[0])
    assert ((q.double() - want).abs() <= torch.finfo(type).eps / 2 * want.abs() + err + 1e-7).all()
    for name, y, err in (("k", *turned(x[:, 4:6], alpha[1])),
                         ("v", x[:, 6:].double(), torch.zeros_like(x[:, 6:]).double())):
        for s in range(3):
            p, r = (t[b.lens[s] - b.chunks[s]:] for t in b.where(s))
            codes, byte = getattr(b, name + "8")[p, :, r], getattr(b, name + "s")[p, :, r].long()
            z, d = (t[b.at[s]:b.at[s] + b.chunks[s]] for t in (y, err))
            got = value(codes, byte)
            # half a step of e4m3: 2^-4 of the value, or 2^-10 scales
            half = torch.maximum(2.0 ** -4 * z.abs(), 2.0 ** -10 * torch.exp2(byte.double() - 127)[..., None])
            assert ((got - z).abs() <= half * (1 + 2.0 ** -18) + d).all()
            # the scale is the least that holds the largest value
            a = z.abs().amax(-1)
            da = d.amax(-1)
            f = torch.exp2(byte.double() - 127)
            assert (a - da <= 448 * f).all() and (a + da > 224 * f).all()


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: "-".join(str(x) for x in c[1:]))
def test_attention(case):
    type, D, Hk, G, page, chunks, lens, window = case
    b = Packed(type, D, Hk, G, page, chunks, lens, window=window)
    kv = b.kv()
    for max_q in (max(chunks), None, 1):
        out, lse = kv.attention(b.q, b.cu, b.len, max_q=max_q, window=window, with_lse=True)
        b.check(out, lse)
    assert kv.read_status() == 0


def test_attention_of_large_scores_and_scales():
    b = Packed(BF16, 128, 2, 2, 64, [7, 1], [500, 3000], seed=5)
    b.q.mul_(12)
    b.scale = 0.3
    for max_q in (7, 200):
        out, lse = b.kv().attention(b.q, b.cu, b.len, scale=0.3, with_lse=True, max_q=max_q)
        b.check(out, lse)


@pytest.mark.parametrize("type", [BF16, F16])
def test_a_heavy_entry_with_small_values(type):
    """One entry takes nearly all the weight and has next to no value: the others' sum still counts."""
    b = Packed(type, 128, 1, 1, 64, [1], [2000], seed=8)
    p, r = b.where(0)
    k = b.k[p, 0, r].clone()
    k[0] = b.q[0, 0].double() * 9 / (b.q[0, 0].double().square().sum() * b.scale)
    c, byte = quantise(k[:1])
    b.k8[p[0], 0, r[0]], b.ks[p[0], 0, r[0]] = c[0].to(E4M3), byte[0].to(torch.uint8)
    b.k[p[0], 0, r[0]] = value(c, byte)[0]
    b.v8[p[0], 0, r[0]] = torch.zeros(128, device="cuda").to(E4M3)
    b.vs[p[0], 0, r[0]] = 0
    b.v[p[0], 0, r[0]] = 0
    out, lse = b.kv().attention(b.q, b.cu, b.len, max_q=1, with_lse=True)
    b.check(out, lse)
    want = Batch.attention(b, 0)[0]
    assert float((out.double() - want).norm() / want.norm()) < 4 * torch.finfo(type).eps


@pytest.mark.parametrize("chunks,lens", [([1, 1], [130, 3000]), ([9, 300], [200, 1000]),
                                         ([3, 20], [20, 500])])
def test_padding_rows_are_left_alone(chunks, lens):
    b = Packed(BF16, 128, 2, 4, 64, chunks, lens, pad=7, lead=3)
    out = torch.full((b.T, b.H, b.D), 7.0, dtype=b.type, device="cuda")
    _, lse = b.kv().attention(b.q, b.cu, b.len, with_lse=True, out=out, max_q=max(chunks))
    b.check(out, lse)
    assert (out[:3] == 7).all() and (out[-7:] == 7).all()


@pytest.mark.parametrize("D,type", [(128, BF16), (64, F16), (64, BF16), (128, F16)])
@pytest.mark.parametrize("chunks,lens,window", [([1, 1], [130, 3000], 0), ([1, 4], [260, 700], 100),
                                                ([9, 5], [9, 300], 3), ([200, 3], [600, 300], 0),
                                                ([150, 300], [150, 900], 60)])
def test_what_a_row_does_not_see_never_reaches_it(D, type, chunks, lens, window):
    """Stale rows, unused pages and later or older entries may hold any codes and scales."""
    b = Packed(type, D, 2, 2, 32, chunks, lens, window=window)
    kw = dict(window=window, with_lse=True, max_q=max(chunks))
    want, wl = b.kv().attention(b.q, b.cu, b.len, **kw)
    b.check(want, wl)
    live = torch.zeros(b.k.shape[0], b.page, dtype=torch.bool, device="cuda")
    for s in range(len(lens)):
        p, r = b.where(s)
        live[p, r] = True
        if window:
            old = max(0, lens[s] - chunks[s] - window + 1)
            live[p[:old], r[:old]] = False
    stale = ~live
    for code, scale in ((0x7f, 127), (0xff, 255), (0, 255), (0x7e, 254), (0xfe, 0)):
        for t, x in ((b.k8, code), (b.v8, code), (b.ks, scale), (b.vs, scale)):
            t.view(torch.uint8).transpose(1, 2)[stale] = x
        got, gl = b.kv().attention(b.q, b.cu, b.len, **kw)
        assert torch.equal(got, want) and torch.equal(gl, wl), (code, scale)
    # one entry inside a chunk: only the rows that see it change
    for s in range(len(lens)):
        if chunks[s] < 3:
            continue
        i = chunks[s] // 2
        p, r = (int(t[lens[s] - chunks[s] + i]) for t in b.where(s))
        see = torch.zeros(b.T, dtype=torch.bool, device="cuda")
        see[b.at[s] + i:b.at[s] + (min(chunks[s], i + window) if window else chunks[s])] = True
        for t, x, dims in ((b.vs, 255, slice(None)), (b.ks, 255, slice(None)), (b.v8, 0x7f, 3),
                           (b.v8, 0xff, 3), (b.k8, 0x7f, slice(None))):
            bits = t.view(torch.uint8)
            keep = bits[p, :, r].clone()
            if t.dim() == 4:
                bits[p, :, r, 3] = x
            else:
                bits[p, :, r] = x
            got, gl = b.kv().attention(b.q, b.cu, b.len, **kw)
            bits[p, :, r] = keep
            assert torch.equal(got[~see], want[~see]) and torch.equal(gl[~see], wl[~see])
            assert torch.isnan(got[see][..., dims]).all()
            is_key = t is b.ks or t is b.k8
            assert torch.isnan(gl[see]).all() if is_key else torch.equal(gl, wl)


@pytest.mark.parametrize("chunk", [1, 9, 200])
def test_pages_outside_the_pool_take_no_part(chunk):
    b = Packed(BF16, 128, 1, 2, 32, [chunk, chunk], [700, 300])
    b.table[0, 3] = b.n_pages
    b.table[1, 0] = -1
    kv = b.kv()
    out, lse = kv.attention(b.q, b.cu, b.len, with_lse=True, max_q=chunk)
    assert kv.read_status() == pp_().PP_S_INDEX and kv.read_status() == 0
    whole, hide = b.sees, {0: slice(96, 128), 1: slice(0, 32)}

    def sees(s):
        m = whole(s)
        m[:, hide[s]] = False
        return m
    b.sees = sees
    b.table[0, 3] = b.table[1, 0] = 0
    b.check(out, lse)


@pytest.mark.parametrize("chunk", [1, 5, 100])
def test_lengths_past_the_table_keep_live_entries(chunk):
    """Entries that kv_len counts past the table's row take no part; the rest is attended to."""
    b = Packed(BF16, 128, 2, 2, 16, [chunk, chunk], [320, 200])
    width = 12                                           # 192 entries have a place
    table = b.table[:, :width].contiguous()
    kv = pp_().PagedKV8(b.k8, b.v8, b.ks, b.vs, table, dtype=b.type)
    out, lse = kv.attention(b.q, b.cu, b.len, with_lse=True, max_q=chunk)
    assert kv.read_status() == pp_().PP_S_INDEX
    whole = b.sees

    def sees(s):
        m = whole(s)
        m[:, width * 16:] = False
        return m
    b.sees = sees
    b.check(out, lse)


def test_attention_reads_strided_rows_and_pages():
    b = Packed(BF16, 128, 2, 3, 64, [1, 4], [500, 300], joint=True, stride_pages=2)
    assert b.q.stride(0) > b.H * b.D and b.k8.stride(0) > b.Hk * b.page * b.D
    out, lse = b.kv().attention(b.q, b.cu, b.len, with_lse=True, max_q=4)
    b.check(out, lse)


@pytest.mark.parametrize("max_q", [3, 150])
def test_offsets_past_32_bits(max_q):
    """A pool of more than 2^32 codes, its last pages in use."""
    n, page, D = 40, 256, 128
    stride = ((1 << 32) // (n - 8) + 4096) // 16 * 16
    b = Packed(BF16, D, 1, 2, page, [3, max_q], [600, 800], spare=0)
    big = torch.zeros((n - 1) * stride + page * D, dtype=torch.uint8, device="cuda").view(E4M3)
    k = big.as_strided((n, 1, page, D), (stride, page * D, D, 1))
    v = torch.zeros_like(big).as_strided(k.size(), k.stride())
    ks, vs = (torch.zeros((n, 1, page), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = torch.where(b.table >= 0, n - 1 - b.table, b.table)
    for s in range(2):
        old, new = b.table[s][b.table[s] >= 0].long(), table[s][table[s] >= 0].long()
        for i, j in zip(old.tolist(), new.tolist()):
            k[j], v[j], ks[j], vs[j] = b.k8[i], b.v8[i], b.ks[i], b.vs[i]
    kv = pp_().PagedKV8(k, v, ks, vs, table)
    out, lse = kv.attention(b.q, b.cu, b.len, with_lse=True, max_q=max_q)
    b.check(out, lse)
    x = torch.randn((3 + max_q, 4, D), device="cuda", dtype=BF16)
    kv.append(x[:, :2], x[:, 2:3], x[:, 3:], b.cu, b.len, rot_dim=0)
    p, r = b.where(1, table)
    codes, byte = quantise(x[3:, 3].double())
    assert torch.equal(torch.stack([v[i, 0, j].double() for i, j in zip(
        p[-max_q:].tolist(), r[-max_q:].tolist())]), codes)
    assert torch.equal(vs[p[-max_q:], 0, r[-max_q:]].long(), byte)


@pytest.mark.parametrize("type", [BF16, F16])
@pytest.mark.parametrize("G", [1, 4, 16])
def test_a_sequence_does_not_depend_on_its_neighbours(type, G):
    chunks, lens = [1, 1, 4, 2], [3000, 77, 20000, 300]
    b = Packed(type, 128, 2, G, 64, chunks, lens)
    if G > 8:
        chunks = None
    out, lse = b.kv().attention(b.q, b.cu, b.len, max_q=4, with_lse=True)
    b.check(out, lse)
    for s in range(4 if chunks else 0):
        a, e = b.at[s], b.at[s + 1]
        kv = pp_().PagedKV8(b.k8, b.v8, b.ks, b.vs, b.table[s:s + 1].contiguous(), dtype=type)
        one, l = kv.attention(b.q[a:e], b.cu[s:s + 2] - a, b.len[s:s + 1], max_q=4, with_lse=True)
        assert torch.equal(one, out[a:e]) and torch.equal(l, lse[a:e])


def test_many_sequences():
    n = 2048
    chunks = [i % 3 for i in range(n)]
    lens = [(i * 7) % 41 + chunks[i] for i in range(n)]
    b = Packed(BF16, 64, 1, 2, 16, chunks, lens)
    out, lse = b.kv().attention(b.q, b.cu, b.len, max_q=2, with_lse=True)
    for s in list(range(0, n, 97)) + [n - 1]:
        if chunks[s]:
            o, l, tol, ltol = b.attention(s)
            a = b.at[s]
            assert ((out[a:a + chunks[s]].double() - o).abs() <= tol).all()


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 128, 129])
@pytest.mark.parametrize("type,D", [(BF16, 128), (F16, 64), (F16, 128)])
def test_every_count_of_rows(rows, type, D):
    """Next to the sizes at which tiles and kernels change, one head and three."""
    for G in (1, 3):
        n = -(-rows // G)
        b = Packed(type, D, 2, G, 16, [n, 1], [max(n, 333), 40], seed=rows)
        out, lse = b.kv().attention(b.q, b.cu, b.len, max_q=n, with_lse=True)
        b.check(out, lse)


@pytest.mark.parametrize("type,D,page,to_page", [(BF16, 128, 64, 16), (F16, 64, 16, 256),
                                                 (F16, 128, 256, 64), (BF16, 64, 32, 32)])
def test_read(type, D, page, to_page):
    lens = [1000, 0, 1, 65, 64]
    b = Packed(type, D, 3, 2, page, [1, 0, 1, 1, 1], lens, spare=3)
    b.ks[:, 1, 5], b.vs[:, 2, 7] = 255, 255
    b.k8.view(torch.uint8)[:, 0, 3, 1] = 0x7f
    b.vs[:, 0, 9] = 127 + 12                             # beyond fp16 in part
    need = [-(-n // to_page) for n in lens]
    table = torch.full((5, max(need)), -1, dtype=torch.int32, device="cuda")
    order = torch.randperm(sum(need) + 2, generator=b.g, device="cuda").int()
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m]
        at += m
    k = torch.full((sum(need) + 2, 3, to_page, D), 7.0, dtype=type, device="cuda")
    v, mass = k.clone(), torch.ones(k.shape[:3], device="cuda")
    kv = b.kv()
    kv.read(b.len, pp_().PagedKV(k, v, table, mass=mass))
    assert kv.read_status() == 0
    live = torch.zeros(k.shape[0], to_page, dtype=torch.bool, device="cuda")
    for s, n in enumerate(lens):
        p, r = b.where(s)
        tp, tr = b.where(s, table, n, to_page)
        live[tp, tr] = True
        for got, codes, byte in ((k, b.k8, b.ks), (v, b.v8, b.vs)):
            want = value(codes[p, :, r], byte[p, :, r].long()).to(type)
            assert torch.equal(got[tp, :, tr].nan_to_num(7e4, 6e4, 5e4),
                               want.nan_to_num(7e4, 6e4, 5e4))
        assert (mass[tp, :, tr] == 0).all()
    for t, x in ((k, 7), (v, 7), (mass, 1)):
        assert (t.transpose(1, 2)[~live] == x).all()


def test_read_leaves_what_has_no_place():
    b = Packed(BF16, 128, 2, 1, 64, [1, 1], [300, 200])
    k = torch.full((12, 2, 32, 128), 7.0, dtype=BF16, device="cuda")
    v = k.clone()
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6)   # 192 entries each
    table[1, 2] = 12
    b.table[0, 1] = -1
    kv = b.kv()
    kv.read(b.len, pp_().PagedKV(k, v, table))
    assert kv.read_status() == pp_().PP_S_INDEX
    p, r = b.where(0, n=192)
    got = torch.stack([k[j // 32, :, j % 32] for j in range(192)]).double()
    hole = torch.arange(192, device="cuda") // 64 == 1
    assert (got[hole] == 7).all() and torch.equal(got[~hole], b.k[p, :, r][~hole])
    p, r = b.where(1, n=192)
    got = torch.stack([v[6 + j // 32, :, j % 32] for j in range(192)]).double()
    hole = torch.arange(192, device="cuda") // 32 == 2
    assert (got[hole] == 7).all() and torch.equal(got[~hole], b.v[p, :, r][~hole])


@pytest.mark.parametrize("chunk", [1, 4, 200])
def test_graphs_replay_with_new_lengths_and_share_nothing(chunk):
    b = Packed(BF16, 128, 2, 2, 64, [chunk, chunk], [2000, 900])
    kv = b.kv()
    kv.attention(b.q, b.cu, b.len, max_q=chunk)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kv.attention(b.q, b.cu, b.len, max_q=chunk, with_lse=True))
        graphs.append(g)
    for lens in ([2000, 900], [chunk, 900], [1500, chunk]):
        b.lens = lens
        b.len.copy_(torch.tensor(lens, dtype=torch.int32))
        streams = [torch.cuda.Stream() for _ in graphs]
        for o, l in outs:
            o.fill_(9)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):          # side by side: each has its own scratch
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, l in outs:
            b.check(o, l)


@pytest.mark.parametrize("chunk", [1, 5])
def test_two_calls_at_once(chunk):
    b = Packed(F16, 128, 4, 2, 16, [chunk] * 3, [5000, 700, 90])
    want = b.kv().attention(b.q, b.cu, b.len, max_q=chunk, with_lse=True)
    b.check(*want)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(4)], []
    kv = b.kv()
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(kv.attention(b.q, b.cu, b.len, max_q=chunk, with_lse=True))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


@pytest.mark.parametrize("type,D,G,chunks", [(BF16, 128, 1, [1, 1]), (F16, 64, 4, [4, 2]),
                                             (BF16, 128, 8, [4, 1]), (F16, 128, 16, [4, 2]),
                                             (BF16, 128, 2, [200, 3])])
def test_a_wait_runs_out_and_the_next_call_is_whole(type, D, G, chunks):
    pp = pp_()
    b = Packed(type, D, 2, G, 64, chunks, [900, 500])
    kv = b.kv()
    run = lambda: kv.attention(b.q, b.cu, b.len, max_q=max(chunks), with_lse=True)
    want = run()
    assert kv.read_status() == 0
    pp.pp_test_paged_faults(4096, 1)
    try:
        run()
        torch.cuda.synchronize()
    finally:
        pp.pp_test_paged_faults(0, 0)
    assert kv.read_status() == pp.PP_S_TIMEOUT
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(run(), want))
    assert kv.read_status() == 0


def test_wrapper_refuses():
    b = Packed(BF16, 128, 2, 2, 64, [1], [100])
    make = pp_().PagedKV8
    for bad in ([b.k8.view(torch.uint8), b.v8, b.ks, b.vs], [b.k8, b.v8[:1], b.ks, b.vs],
                [b.k8, b.v8, b.ks[:, :1], b.vs], [b.k8, b.v8, b.ks.float(), b.vs],
                [b.k8, b.v8, b.ks, b.vs.cpu()], [b.k8, b.v8, b.ks.int(), b.vs]):
        with pytest.raises(ValueError):
            make(*bad, b.table)
    with pytest.raises(ValueError):
        make(b.k8, b.v8, b.ks, b.vs, b.table, dtype=F32)
    with pytest.raises(ValueError):
        make(b.k8, b.v8, b.ks, b.vs, b.table.long())
    with pytest.raises(ValueError):
        b.kv().attention(b.q.half(), b.cu, b.len)
    other = pp_().PagedKV(torch.zeros_like(b.k8, dtype=F16), torch.zeros_like(b.k8, dtype=F16), b.table)
    with pytest.raises(pp_().PPError):
        b.kv().read(b.len, other)
    # the same bytes as e8m0 scales
    kv = make(b.k8, b.v8, b.ks.view(torch.float8_e8m0fnu), b.vs.view(torch.float8_e8m0fnu), b.table)
    b.check(*kv.attention(b.q, b.cu, b.len, with_lse=True))


def test_a_session_of_prompt_ticks_and_scores():
    """The operators as they are used: a prompt in one call, ticks beside it, each followed by the
    attention, a projection to logits and the log probabilities of the forced tokens; then back to 16
    bits, where an eviction and the 16-bit attention go on."""
    pp = pp_()
    type, Hk, G, D, page, vocab = BF16, 2, 3, 64, 16, 301
    H = Hk * G
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    n = lambda *s: torch.randn(s, generator=g, device="cuda")
    head = n(H * D, vocab) / 8
    table = torch.randperm(24, generator=g, device="cuda").int().view(2, 12)
    k8 = torch.zeros((24, Hk, page, D), dtype=E4M3, device="cuda")
    v8 = torch.zeros_like(k8)
    ks, vs = (torch.zeros((24, Hk, page), dtype=torch.uint8, device="cuda") for _ in range(2))
    kv = pp.PagedKV8(k8, v8, ks, vs, table, dtype=type)
    lens, keys, values = [0, 0], [[], []], [[], []]
    for chunks in ([70, 33], [1, 1], [1, 0], [5, 1]):
        T = sum(chunks)
        lens = [a + c for a, c in zip(lens, chunks)]
        cu = torch.tensor([0, chunks[0], T], dtype=torch.int32, device="cuda")
        ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
        x = n(T, H + 2 * Hk, D)
        q = kv.append(x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], cu, ln, rot_dim=0)
        out, lse = kv.attention(q, cu, ln, max_q=max(chunks), with_lse=True)
        logits = out.flatten(1).float() @ head
        tokens = torch.randint(0, vocab, (T,), generator=g, device="cuda").int()
        got = pp.token_logprobs(logits, tokens, top=3, with_entropy=True, status=kv.status)
        # plainly
        ck, bk = quantise(x[:, H:H + Hk].double())
        cv, bv = quantise(x[:, H + Hk:].double())
        for s in range(2):
            a, e = cu[s], cu[s + 1]
            keys[s].append(value(ck[a:e], bk[a:e]))
            values[s].append(value(cv[a:e], bv[a:e]))
            k, v = torch.cat(keys[s]), torch.cat(values[s])
            y = q[a:e].double().unflatten(1, (Hk, G))
            z = torch.einsum("ihgd,jhd->hgij", y, k) * D ** -0.5
            see = torch.arange(len(k), device="cuda") <= torch.arange(
                len(k) - chunks[s], len(k), device="cuda")[:, None]
            w = torch.softmax(z.masked_fill(~see, -math.inf), -1)
            o = torch.einsum("hgij,jhd->ihgd", w, v).flatten(1, 2)
            m = torch.einsum("hgij,jhd->ihgd", w, v.abs()).flatten(1, 2)
            # the output's rounding, the weights', and scores of 2^-12 at most off
            assert ((out[a:e].double() - o).abs() <= 2.0 ** -8 * o.abs() + 2.0 ** -7 * m).all()
        lp = torch.log_softmax(logits.double(), -1)
        want = lp.gather(1, tokens.long()[:, None])[:, 0]
        assert ((got["logprob"].double() - want).abs() <= 2.0 ** -18 * (1 + want.abs())).all()
        assert torch.equal(got["top_tokens"][:, 0].long(), lp.argmax(-1))
    assert kv.read_status() == 0
    # back to 16 bits, and on
    k, v = (torch.zeros((24, Hk, page, D), dtype=type, device="cuda") for _ in range(2))
    wide = pp.PagedKV(k, v, table, mass=torch.rand((24, Hk, page), generator=g, device="cuda"))
    kv.read(ln, wide)
    again, lse16 = wide.attention(q, cu, ln, max_q=max(chunks), with_lse=True)
    m = torch.stack([x.abs().amax() for x in (torch.cat(values[0]), torch.cat(values[1]))]).amax()
    assert ((again.double() - out.double()).abs() <= 2.0 ** -5 * m).all()
    assert ((lse16 - lse).abs() <= 2.0 ** -12).all()
    wide.attention_mass(q, lse16, cu, ln, max_q=max(chunks))
    to = pp.PagedKV(torch.zeros_like(k), torch.zeros_like(v), table, mass=torch.zeros_like(wide.mass))
    to_len, kept = wide.evict(ln, 40, 4, to)
    assert to_len.tolist() == [min(n, 40) for n in lens]
    assert wide.read_status() == 0


def test_a_captured_tick_is_the_eager_one():
    """append, attention and the log probabilities of one token per session, replayed over growing
    lengths: bit for bit what the calls give one by one."""
    pp = pp_()
    Hk, G, D, page, n, cap = 2, 2, 128, 16, 5, 20
    H = Hk * G
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    table = torch.randperm(n * cap, generator=g, device="cuda").int().view(n, cap)
    start = torch.tensor([1, 300, 17, 128, 255], dtype=torch.int32, device="cuda")
    pools = [torch.randint(0, 0x78, (n * cap, Hk, page, D), generator=g, device="cuda").byte()
             for _ in range(2)]
    scales = [torch.randint(118, 122, (n * cap, Hk, page), generator=g, device="cuda").byte()
              for _ in range(2)]
    ticks = [torch.randn((n, H + 2 * Hk, D), generator=g, device="cuda") for _ in range(6)]
    head = torch.randn((H * D, 1000), generator=g, device="cuda").to(BF16)
    tokens = torch.randint(0, 1000, (n,), generator=g, device="cuda").int()
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")

    def session():
        k, v, ks, vs = (t.clone() for t in pools + scales)
        kv = pp.PagedKV8(k.view(E4M3), v.view(E4M3), ks, vs, table)
        x, length = torch.empty_like(ticks[0]), start.clone()

        def tick():
            length.add_(1)
            q = kv.append(x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], cu, length)
            out, lse = kv.attention(q, cu, length, max_q=1, with_lse=True)
            s = pp.token_logprobs(out.flatten(1) @ head, tokens, top=5, with_entropy=True)
            return (q, out, lse) + tuple(s.values())
        return tick, x, (k, v, ks, vs, length), kv

    tick, x, state, kv = session()
    want = []
    for t in ticks:
        x.copy_(t)
        want.append([y.clone() for y in tick() + state])
    assert kv.read_status() == 0
    tick, x, state, kv = session()
    begin = [y.clone() for y in state]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x.copy_(ticks[0])
        tick()
    torch.cuda.synchronize()
    for y, z in zip(state, begin):
        y.copy_(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = tick()
    for t, w in zip(ticks, want):
        x.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for y, z in zip(out + state, w):
            assert torch.equal(y, z)


@pytest.mark.parametrize("type", [BF16, F16])
def test_a_value_that_some_rows_do_not_see_costs_them_no_precision(type):
    """Later entries of a chunk with values 2^60 (2^12) larger: the rows before them keep their bits."""
    b = Packed(type, 128, 1, 2, 16, [6], [90], seed=4)
    want, wl = b.kv().attention(b.q, b.cu, b.len, max_q=6, with_lse=True)
    b.check(want, wl)
    p, r = (t[87:] for t in b.where(0))
    b.vs[p, :, r] += 60 if type == BF16 else 12
    got, gl = b.kv().attention(b.q, b.cu, b.len, max_q=6, with_lse=True)
    assert torch.equal(got[:3], want[:3]) and torch.equal(gl, wl)
    b.v[p, :, r] *= 2.0 ** (60 if type == BF16 else 12)
    b.check(got[:, :], gl) if type == BF16 else None


@pytest.mark.parametrize("type", [BF16, F16])
@pytest.mark.parametrize("G", [1, 4, 20])
def test_values_at_the_end_of_the_range(type, G):
    """Powers of two of V reach the output as they are, up to where bf16 ends (fp16: infinity), the
    sums over the entries on their way to it included."""
    b = Packed(type, 128, 2, G, 64, [1, 1], [300, 3000], seed=31)
    low = b.vs.clone()
    for up in (0, int(245 - int(low.max()))):
        b.vs = low + up
        out = b.kv().attention(b.q, b.cu, b.len, max_q=1)
        if up == 0:
            # (weights of 1 in all at most: a value of the output is the largest of V at most)
            want = out.double()
            tiny = want.abs() < 2.0 ** -100 if type == BF16 else want.abs() < 2.0 ** -14
        else:
            got, scaled = out.double(), want * 2.0 ** up
            if type == F16:
                scaled = torch.where(scaled.abs() >= 65520, scaled.sign() * math.inf, scaled)
            assert (tiny | (got == scaled)).all()


@pytest.mark.parametrize("type", [BF16, F16])
def test_the_largest_power_of_two(type):
    b = Packed(type, 128, 2, 2, 64, [1], [1], seed=32)
    b.v8.view(torch.uint8).bitwise_and_(0x87)            # codes below 2^-6: 2^121 with the largest scale
    b.vs.fill_(254)
    out = b.kv().attention(b.q, b.cu, b.len, max_q=1)
    p, r = b.where(0)
    want = value(b.v8[p[0], :, r[0]].double(), b.vs[p[0], :, r[0]]).repeat_interleave(2, 0)[None]
    if type == F16:
        want = torch.where(want == 0, want, want.sign() * math.inf)
    assert want.abs().max() > 2.0 ** 118 and (out.double() == want).all()
