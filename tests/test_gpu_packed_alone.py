"""A sequence of an 8-bit cache gives the same bits alone and in any batch, in every form of short chunks,
those of several row tiles among them, and beside sequences whose pages are missing (GPU)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_packed import Packed, pp_  # noqa: E402
from test_gpu_paged import BF16, F16  # noqa: E402

FORMS = [(BF16, 128, 1), (F16, 128, 2), (BF16, 64, 3), (F16, 64, 8), (BF16, 128, 16), (F16, 128, 16),
         (BF16, 64, 13), (F16, 64, 16)]


def alone(b, s, **kw):
    a, e = b.at[s], b.at[s + 1]
    kv = pp_().PagedKV8(b.k8, b.v8, b.ks, b.vs, b.table[s:s + 1].contiguous(), dtype=b.type)
    return kv.attention(b.q[a:e], b.cu[s:s + 2] - a, b.len[s:s + 1], with_lse=True, **kw)


@pytest.mark.parametrize("type,D,G", FORMS)
@pytest.mark.parametrize("window", [0, 700])
def test_alone_and_among_others(type, D, G, window):
    b = Packed(type, D, 2, G, 64, [1, 1, 4, 2, 3], [3000, 77, 20000, 300, 1537], window=window)
    kw = dict(max_q=4, window=window)
    out, lse = b.kv().attention(b.q, b.cu, b.len, with_lse=True, **kw)
    b.check(out, lse)
    for s in range(5):
        one, l = alone(b, s, **kw)
        a, e = b.at[s], b.at[s + 1]
        assert torch.equal(one, out[a:e]) and torch.equal(l, lse[a:e])


@pytest.mark.parametrize("type,D,G", FORMS)
def test_beside_sequences_without_some_pages(type, D, G):
    chunks, lens = [4, 1, 3, 4] * 4, [1500, 200, 900, 333] * 4
    b = Packed(type, D, 2, G, 64, chunks, lens)
    kv = b.kv()
    want = kv.attention(b.q, b.cu, b.len, max_q=4, with_lse=True)
    b.check(*want)
    assert kv.read_status() == 0
    b.table[::4, 1] = -1
    got = kv.attention(b.q, b.cu, b.len, max_q=4, with_lse=True)
    assert kv.read_status() == pp_().PP_S_INDEX
    for s in range(16):
        a, e = b.at[s], b.at[s + 1]
        same = torch.equal(got[0][a:e], want[0][a:e]) and torch.equal(got[1][a:e], want[1][a:e])
        assert same == (s % 4 != 0), s
