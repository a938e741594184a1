"""Long chunks over an 8-bit cache whose copy does not fit at once: sequences are taken in turns (GPU)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_packed import Packed, pp_  # noqa: E402
from test_gpu_paged import BF16, F16  # noqa: E402

# 262144 entries of 2 x 128 dims: 268 MB of copy a sequence, 8 at a time at most
WIDE = 262144


def batch(type, chunks, lens, G=2, page=64, **kw):
    b = Packed(type, 128, 2, G, page, chunks, lens, width=WIDE // page, **kw)
    taken = pp_().pp_packed_attention_scratch_bytes(b.kv().c, b.H, b.T, max(chunks), 0)
    assert taken < len(lens) * WIDE * 2 * 128 * 4      # (not all at once)
    return b


CHUNKS = [1, 0, 100, 3, 0, 0, 1, 200, 0, 5, 64, 1, 0, 0, 9, 0, 40]
LENS = [3000, 500, 100, 0, 7, 0, 1, 1300, 20000, 2, 300, 129, 0, 1, 9, 40, 4000]


@pytest.mark.parametrize("type,window", [(BF16, 0), (F16, 0), (BF16, 150)])
def test_every_sequence_has_its_turn(type, window):
    b = batch(type, CHUNKS, LENS, lead=3, pad=5, window=window)
    out = torch.full((b.T, b.H, b.D), 7.0, dtype=type, device="cuda")
    kv = b.kv()
    for _ in range(2):
        _, lse = kv.attention(b.q, b.cu, b.len, max_q=200, window=window, with_lse=True, out=out)
        b.check(out, lse)
        assert (out[:3] == 7).all() and (out[-5:] == 7).all()
    assert kv.read_status() == 0


def test_pages_that_are_missing_are_told_of_in_every_turn():
    chunks, lens = [70] * 16, [300] * 16
    b = batch(BF16, chunks, lens)
    kv = b.kv()
    for s in (0, 15):
        keep = int(b.table[s, 1])
        b.table[s, 1] = -1
        kv.attention(b.q, b.cu, b.len, max_q=70)
        assert kv.read_status() == pp_().PP_S_INDEX
        b.table[s, 1] = keep
    out, lse = kv.attention(b.q, b.cu, b.len, max_q=70, with_lse=True)
    b.check(out, lse)
    assert kv.read_status() == 0


def test_turns_in_a_graph():
    b = batch(F16, CHUNKS, LENS)
    kv = b.kv()
    want = kv.attention(b.q, b.cu, b.len, max_q=200, with_lse=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kv.attention(b.q, b.cu, b.len, max_q=200, with_lse=True)
    rows = slice(0, b.T)
    for _ in range(3):
        for x in got:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x[rows], y[rows]) for x, y in zip(got, want))
    b.check(*got)
