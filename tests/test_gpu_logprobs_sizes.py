"""token_logprobs refuses sizes that the library's 32-bit counts do not hold (GPU)."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("shape", [(2 ** 32 + 5, 1), (2 ** 28, 1), (2 ** 31, 3), (2 ** 16, 2 ** 16 + 1, 1),
                                   (1, 2 ** 32 + 3, 1)])
def test_more_rows_than_can_be_counted(shape):
    import full_duplex_speech_lockstep_gb300 as pp
    x = torch.zeros((1,) * (len(shape) - 1) + (shape[-1],), device="cuda").expand(shape)
    with pytest.raises(pp.PPError):
        pp.token_logprobs(x, with_entropy=True)


@pytest.mark.parametrize("n", [2 ** 24 + 1, 2 ** 32 + 7])
def test_longer_rows_than_can_be_counted(n):
    import full_duplex_speech_lockstep_gb300 as pp
    x = torch.empty((1, n), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pp.PPError):
        pp.token_logprobs(x, with_entropy=True)
