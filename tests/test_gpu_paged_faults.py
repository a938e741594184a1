"""A bounded wait of the paged-cache kernels runs out (GPU).  A tile never counts as loaded
under a short poll limit (pp_test_paged_faults): the call returns, PP_S_TIMEOUT is reported, and the
next call gives what it gave before."""
import time

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_paged import BF16, F16, Batch, pp_  # noqa: E402

# (the first three in k_paged_attn's tiles of 16 and 32 rows, the others in k_paged_attn_tc's units of
# one row tile and of two)
CASES = [(BF16, 128, 1, [1, 1]), (F16, 64, 4, [4, 2]), (BF16, 128, 8, [4, 1]), (BF16, 128, 2, [40, 3]),
         (F16, 64, 2, [200, 1])]


@pytest.mark.parametrize("call", ["attention", "mass"])
@pytest.mark.parametrize("type,D,G,chunks", CASES)
def test_a_wait_runs_out_and_the_next_call_is_whole(type, D, G, chunks, call):
    pp = pp_()
    b = Batch(type, D, 2, G, 64, chunks, [900, 500])
    kv = b.kv()
    lse = kv.attention(b.q, b.cu, b.len, max_q=max(chunks), with_lse=True)[1]

    def run():
        if call == "attention":
            return kv.attention(b.q, b.cu, b.len, max_q=max(chunks), with_lse=True)
        mass = torch.zeros_like(b.mass)
        kv.attention_mass(b.q, lse, b.cu, b.len, max_q=max(chunks), mass=mass)
        return (mass,)
    want = run()
    assert kv.read_status() == 0
    start = time.time()
    pp.pp_test_paged_faults(4096, 1)
    try:
        run()
        torch.cuda.synchronize()
    finally:
        pp.pp_test_paged_faults(0, 0)
    assert kv.read_status() == pp.PP_S_TIMEOUT
    assert time.time() - start < 30
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(run(), want))
    assert kv.read_status() == 0
