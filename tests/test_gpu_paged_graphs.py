"""The paged-cache calls of a tick, captured once and replayed, and sizes at the limits (GPU)."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_paged import BF16, F16, Batch, check_mass, pp_  # noqa: E402


@pytest.mark.parametrize("type,D", [(BF16, 128), (F16, 64)])
def test_a_captured_tick_is_the_eager_one(type, D):
    """append, attention and mass of one token per session, then an eviction, replayed over growing
    lengths: bit for bit what the calls give one by one."""
    Hk, G, page, n, cap = 4, 2, 16, 5, 20
    H = Hk * G
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    table = torch.randperm(n * cap, generator=g, device="cuda").int().view(n, cap)
    start = torch.tensor([1, 300, 17, 128, 255], dtype=torch.int32, device="cuda")
    pools = [torch.randn((n * cap, Hk, page, D), generator=g, device="cuda").to(type)
             for _ in range(2)]
    weights = torch.rand((n * cap, Hk, page), generator=g, device="cuda")
    ticks = [torch.randn((n, H + 2 * Hk, D), generator=g, device="cuda") for _ in range(6)]
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")

    def session():
        k, v, m = pools[0].clone(), pools[1].clone(), weights.clone()
        other = [torch.zeros_like(t) for t in (k, v, m)]
        kv = pp_().PagedKV(k, v, table, mass=m)
        to = pp_().PagedKV(other[0], other[1], table, mass=other[2])
        x, length = torch.empty_like(ticks[0]), start.clone()

        def tick():
            length.add_(1)
            q = kv.append(x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], cu, length)
            out, lse = kv.attention(q, cu, length, max_q=1, with_lse=True)
            kv.attention_mass(q, lse, cu, length, max_q=1, decay=0.9)
            return (q, out, lse) + tuple(kv.evict(length, 200, 7, to))
        return tick, x, (k, v, m, length) + tuple(other), kv

    tick, x, state, kv = session()
    want = []
    for t in ticks:
        x.copy_(t)
        want.append([y.clone() for y in tick() + state])
    assert kv.read_status() == 0
    tick, x, state, kv = session()
    begin = [y.clone() for y in state]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        x.copy_(ticks[0])
        tick()
    torch.cuda.synchronize()
    for y, z in zip(state, begin):
        y.copy_(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res = tick()
    for y, z in zip(state, begin):
        y.copy_(z)
    for t, w in zip(ticks, want):
        x.copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for got, exp in zip(tuple(res) + state, w):
            assert torch.equal(got, exp)
    assert kv.read_status() == 0


@pytest.mark.parametrize("Hk,G,chunks,lens", [
    (1024, 1, [1, 1], [40, 300]), (160, 1, [1, 3], [700, 1500]), (1024, 2, [20, 1], [20, 130]),
    (3, 64, [1, 1], [600, 20])])
def test_many_heads(Hk, G, chunks, lens):
    b = Batch(BF16, 64, Hk, G, 16, chunks, lens)
    kv = b.kv()
    out, lse = kv.attention(b.q, b.cu, b.len, max_q=max(chunks), with_lse=True)
    b.check(out, lse)
    before = b.mass.clone()
    kv.attention_mass(b.q, lse, b.cu, b.len, max_q=max(chunks))
    for s in range(2):
        check_mass(b, s, before, b.mass, lse, 1.0)
    x = torch.randn((b.T, Hk * (G + 2), 64), generator=b.g, device="cuda").to(BF16)
    kv.append(x[:, :Hk * G], x[:, Hk * G:Hk * (G + 1)], x[:, Hk * (G + 1):], b.cu, b.len)
    for s in range(2):
        p, r = (t[-chunks[s]:] for t in b.where(s))
        assert torch.equal(b.v[p, :, r], x[b.at[s]:b.at[s + 1], Hk * (G + 1):])
    assert kv.read_status() == 0


def test_two_calls_at_once_on_one_cache():
    """Attention of two batches over one cache on two streams, as a draft and a check might run."""
    b = Batch(BF16, 128, 4, 2, 64, [1, 1, 1], [3000, 900, 1500])
    c = Batch(BF16, 128, 4, 2, 64, [40, 2, 9], [3000, 900, 1500])
    c.k, c.v, c.mass, c.table = b.k, b.v, b.mass, b.table
    kv = b.kv()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    res = []
    for _ in range(8):
        with torch.cuda.stream(s1):
            x = kv.attention(b.q, b.cu, b.len, max_q=1, with_lse=True)
        with torch.cuda.stream(s2):
            y = kv.attention(c.q, c.cu, c.len, max_q=40, with_lse=True)
        res.append((x, y))
    torch.cuda.synchronize()
    for x, y in res:
        b.check(*x)
        c.check(*y)
    assert kv.read_status() == 0 and not math.isnan(float(res[0][1][1].sum()))
