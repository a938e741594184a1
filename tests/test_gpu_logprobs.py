"""pp_token_logprobs and Engine.score against plain 64-bit arithmetic on the same logits (GPU).

Tolerances: exponentials are off by 2^-22 of themselves, plus that of their argument d log2(e), rounded
to 2^-24 of its size (at most 2^-24 |d| log2(e), weighed by exp(d): below 2^-24).  A row's sum of n terms
is off by at most (n / 256 + 64) 2^-24 of itself: a thread's own terms one after the other (a thread has
n / 256 or, of a longer row, n / 2048), then trees and joins, each with two more roundings and an
exponential.  The logarithm turns that into an absolute error; differences of logits are off by 2^-24 of
their size.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def pp_():
    import full_duplex_speech_lockstep_gb300 as pp
    return pp


def check(x, tokens, got, top):
    n, x = x.shape[-1], x.double()
    live = torch.isfinite(x)
    y = x.masked_fill(~live, -math.inf)
    some = live.any(-1)
    # distances below the maximum, and sums of their exponentials: beside a maximum of -3e38, 64 bits
    # would lose the logarithm of the sum
    m = y.amax(-1, keepdim=True).masked_fill(~some[..., None], 0)
    d = y - m
    p = torch.exp(d)
    l = p.sum(-1, keepdim=True)
    p, lse = (p / l).masked_fill(~live, 0), l.log()
    rel = (n / 256 + 64) * 2.0 ** -24 + 2.0 ** -21
    if tokens is not None:
        t = tokens.long()
        v = d.gather(-1, t.clamp(0, n - 1)[..., None])
        want = (v - lse)[..., 0].masked_fill(~some | (v[..., 0] == -math.inf), -math.inf)
        want = want.masked_fill((t < 0) | (t >= n), 0)
        out = got["logprob"].double()
        dead = want == -math.inf
        assert torch.equal(out == -math.inf, dead)
        off = (out - want).abs()[~dead]
        tol = (rel + 2.0 ** -22 * (1 + want.abs()))[~dead]
        assert (off <= tol).all(), float((off / tol).max())
    if "entropy" in got:
        want = -(p * (d - lse).masked_fill(~live, 0)).sum(-1)
        # log l - t / l: both sums off by rel, t / l being the mean distance below the maximum
        far = (p * d.masked_fill(~live, 0).abs()).sum(-1)
        tol = rel * (1 + 2 * far) + 2.0 ** -22 * (far + lse[..., 0].abs().masked_fill(~some, 0)) + 1e-30
        assert ((got["entropy"].double() - want.masked_fill(~some, 0)).abs() <= tol).all()
        assert (got["entropy"] >= 0).all()
    if top:
        k = min(top, n)
        i = torch.argsort(-y, dim=-1, stable=True)[..., :k]
        v = d.gather(-1, i).masked_fill(~some[..., None], -math.inf)
        ids = torch.where(v > -math.inf, i, -1)
        assert torch.equal(got["top_tokens"][..., :k].long(), ids)
        lp = got["top_logprobs"][..., :k].double()
        dead = v == -math.inf
        assert torch.equal(lp == -math.inf, dead)
        want = v - lse
        assert ((lp - want).abs() <= rel + 2.0 ** -22 * (1 + want.abs()))[~dead].all()
        assert (got["top_tokens"][..., k:] == -1).all()
        assert (got["top_logprobs"][..., k:] == -math.inf).all()


def make(type, shape, seed=1, spread=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randn(shape, generator=g, device="cuda") * spread).to(type)
    return x, torch.randint(-1, shape[-1], shape[:-1], generator=g, device="cuda").int()


@pytest.mark.parametrize("type", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 2), (2, 7), (5, 255), (4, 2048), (3, 8192), (3, 8193),
                                    (2, 16390), (4, 32000), (3, 32769), (2, 50257), (2, 65537),
                                    (1, 200003), (700, 100)])
def test_rows_of_every_length(type, rows, n):
    for top in (0, 1, 5, 64):
        x, t = make(type, (rows, n), seed=top + 1)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        check(x, t, pp_().token_logprobs(x, t, top=top, with_entropy=True, status=status), top)
        assert status.item() == 0
    got = pp_().token_logprobs(x, None, top=3)
    assert sorted(got) == ["top_logprobs", "top_tokens"]
    check(x, None, got, 3)


@pytest.mark.parametrize("type", [F32, BF16])
@pytest.mark.parametrize("lead,gap", [(1, 0), (3, 5), (7, 1), (13, 8)])
def test_any_alignment_and_stride(type, lead, gap):
    """Rows in groups with other values between them, at every place within 16 bytes."""
    for n in (1, 9, 2048, 9001):
        x, _ = make(type, (4, lead + 3 * n + gap), seed=n)
        view = x[:, lead:lead + 3 * n].unflatten(1, (3, n))
        column = torch.randint(0, n, (4, 9), device="cuda").int()
        t = column[:, 2:5]
        before = x.clone()
        check(view, t, pp_().token_logprobs(view, t, top=4, with_entropy=True), 4)
        assert torch.equal(x, before)


def test_rows_that_are_given_more_than_once():
    x, t = make(F32, (1, 5000))
    many = x.expand(9, 5000)
    t = torch.arange(9, device="cuda").int()
    check(many, t, pp_().token_logprobs(many, t, top=2), 2)


@pytest.mark.parametrize("type", [F32, BF16, F16])
@pytest.mark.parametrize("n", [5, 300, 8192, 9000, 70000, 140000])
def test_ties_go_to_the_lowest_index(type, n):
    """Flat rows, rows of few values, the type's lowest value as a mask, rising and falling rows, and
    zeros of both signs."""
    flat = torch.zeros((7, n), dtype=type, device="cuda")
    flat[1] = torch.finfo(type).min
    flat[2] = (torch.arange(n, device="cuda") % 3).to(type)
    flat[3] = torch.finfo(type).min
    flat[3, n // 2] = 1
    flat[4] = (torch.arange(n, device="cuda") / n * 20).to(type)
    flat[5] = flat[4].flip(0)
    flat[6, 1::2] = -0.0
    t = torch.full((7,), n - 1, dtype=torch.int32, device="cuda")
    for top in (1, 20, 64):
        check(flat, t, pp_().token_logprobs(flat, t, top=top, with_entropy=True), top)


@pytest.mark.parametrize("type", [F32, BF16, F16])
@pytest.mark.parametrize("n", [40, 9000, 66000])
def test_values_that_are_not_finite_take_no_part(type, n):
    pp = pp_()
    x, _ = make(type, (8, n))
    t = torch.full((8,), 3, dtype=torch.int32, device="cuda")
    x[0, 5:30] = -math.inf
    x[1] = -math.inf
    x[2] = -math.inf
    x[2, n - 1] = 2
    x[3, 3] = -math.inf
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = pp.token_logprobs(x[:4], t[:4], top=9, with_entropy=True, status=status)
    check(x[:4], t[:4], got, 9)
    assert status.item() == 0                   # masked by -infinity: ordinary
    x[4, 3] = math.nan
    x[5, n - 1] = math.inf
    x[6] = math.nan
    x[7, ::2] = math.inf
    got = pp.token_logprobs(x, t, top=9, with_entropy=True, status=status)
    check(x, t, got, 9)
    assert status.item() == pp.PP_S_NAN


def test_tokens_without_a_logit():
    pp = pp_()
    x, _ = make(F32, (5, 100))
    t = torch.tensor([-1, -2 ** 31, 99, 100, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = pp.token_logprobs(x[:3], t[:3], status=status)
    assert status.item() == 0
    check(x[:3], t[:3], got, 0)
    got = pp.token_logprobs(x, t, status=status)
    assert status.item() == pp.PP_S_INDEX
    check(x, t, got, 0)


def test_large_and_far_apart_logits():
    x, t = make(F32, (4, 33000))
    x[0] *= 1e30
    x[1] += 1e4
    x[2] = x[2] * 1e-30
    x[3, ::2] = -3e38
    check(x, t, pp_().token_logprobs(x, t, top=6, with_entropy=True), 6)


def test_a_row_does_not_depend_on_its_neighbours():
    x, t = make(BF16, (300, 32000))
    all_ = pp_().token_logprobs(x, t, top=8, with_entropy=True)
    for i in (0, 7, 299):
        one = pp_().token_logprobs(x[i:i + 1], t[i:i + 1], top=8, with_entropy=True)
        assert all(torch.equal(one[k], all_[k][i:i + 1]) for k in one)


def test_rows_past_32_bits():
    ld = (1 << 30) + 24
    big = torch.empty(3 * ld + 1000, dtype=F32, device="cuda")
    x = big.as_strided((4, 1000), (ld, 1))
    x.normal_()
    t = torch.zeros(4, dtype=torch.int32, device="cuda")
    check(x, t, pp_().token_logprobs(x, t, top=2), 2)


def test_streams_and_graphs():
    x, t = make(F32, (64, 32000))
    want = pp_().token_logprobs(x, t, top=4, with_entropy=True)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(3)], []
    for s in streams:
        with torch.cuda.stream(s):
            got.append(pp_().token_logprobs(x, t, top=4, with_entropy=True))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got.append(pp_().token_logprobs(x, t, top=4, with_entropy=True))
    g.replay()
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(o[k], want[k]) for k in want)
    x2, t2 = make(F32, (64, 32000), seed=9)
    x.copy_(x2)
    t.copy_(t2)
    g.replay()
    torch.cuda.synchronize()
    check(x, t, got[-1], 4)


def test_wrapper_refuses():
    f, pp = pp_().token_logprobs, pp_()
    x, t = make(F32, (4, 6, 50))
    for bad in (lambda: f(x.double()), lambda: f(x.transpose(1, 2)), lambda: f(x[0, 0]),
                lambda: f(x, t.long()), lambda: f(x, t[:3]), lambda: f(x, t.t().contiguous().t()),
                lambda: f(x, t.cpu()), lambda: f(x, t, status=t)):
        with pytest.raises(ValueError):
            bad()
    for top in (-1, 65):
        with pytest.raises(pp.PPError):
            f(x, t, top=top)
    none = f(x[:0], t[:0], top=2)
    assert none["logprob"].shape == (0, 6) and none["top_tokens"].shape == (0, 6, 2)
    assert f(x[:, :0], t[:, :0])["logprob"].shape == (4, 0)


def test_the_columns_of_a_tick():
    """Engine.score on a tick's own logits: text row and codebook rows, closed slots, initial tokens."""
    import synth
    from harness import device_weights
    pp = pp_()
    s = synth.TINY
    eng = pp.Engine(s, 3, device_weights(synth.make_weights_host(s, 0)))
    eng.open(0)
    eng.open(2)
    prev = torch.full((3, 17), s.audio_card, dtype=torch.int32, device="cuda")
    prev[:, 0] = s.text_vocab
    user = torch.randint(0, s.audio_card, (3, 8), device="cuda").int()
    logits = torch.zeros((3, eng.logits_ld), device="cuda")
    column = eng.step(prev, user, logits=logits).clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    text, audio = eng.score(logits, column, top=2, with_entropy=True, status=status)
    assert eng.status() == 0 and status.item() == 0
    check(logits[:, :s.text_vocab], column[:, 0], text, 2)
    rows = logits[:, s.text_vocab:].unflatten(1, (s.n_q, s.audio_card))
    check(rows, column[:, 1:], audio, 2)
    live = [0, 2]
    assert torch.equal(text["top_tokens"][live, 0], column[live, 0])        # greedy: the likeliest
    assert torch.equal(audio["top_tokens"][live, :8, 0], column[live, 1:9])
    assert (column[1] == -1).all() and (audio["logprob"][1] == 0).all()
    text, audio = eng.score(logits, prev, status=status)
    assert (text["logprob"] == 0).all() and (audio["logprob"] == 0).all()
    assert status.item() == pp.PP_S_INDEX
    eng.close_engine()


@pytest.mark.parametrize("type", [F32, BF16, F16])
@pytest.mark.parametrize("n", [31, 33, 64, 65, 256, 257, 512, 513, 1024, 1025, 2049, 4096, 4097, 8200, 16385])
def test_where_one_form_ends(type, n):
    """Lengths on both sides of a change of kernels, with equal values and some that are not finite."""
    x, t = make(type, (9, n), seed=n)
    x[1] = x[1].round()
    x[2] = 2.5
    x[3] = -math.inf
    x[4, ::3] = math.nan
    x[5, n // 2:] = -math.inf
    x[6, -1] = torch.finfo(type).max
    x[7, 0] = torch.finfo(type).min
    t[8] = n - 1
    for top in (0, 3, 64):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = pp_().token_logprobs(x, t, top=top, with_entropy=True, status=status)
        check(x, t, got, top)
        alone = pp_().token_logprobs(x[5:6], t[5:6], top=top, with_entropy=True)
        assert all(torch.equal(alone[k][0], got[k][5]) for k in alone)
        assert status.item() == pp_().PP_S_NAN
