"""8-bit attention where powers of two of V differ widely from key to key (GPU): an output is as exact as
what weighs in it, weight times value, not as the largest value that a row sees.

Tolerances, relative to the terms w_j |v_j| of a row's sum in 64 bits over the same codes: each weight is
rounded to fp16 (2^-11) and to the output's type at the end (eps_t / 2); a score off by ds_j changes its own
term by ds_j and all of them by the weighted mean of ds, where ds_j has the fp32 sum of D products and the
exponential's argument (D 2^-23 of the products' absolute sum, n 2^-23, 2^-21: test_gpu_paged.py) and
the queries' parts (2^-21 of the row's largest: test_gpu_packed.py).  A step of up to 512 keys
holds weights to 2^-18 where its largest is between 2^2 and 2^8: a term of it is off by 2^-20 of the
step's largest w_i 2^ev_i, times a code of 448 at most."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from test_gpu_packed import E4M3, Packed, quantise, value  # noqa: E402
from test_gpu_paged import BF16, F16  # noqa: E402


def terms(b, s):
    """out and its error bound for sequence s: [n, H, D] each."""
    x, size = b.scores(s)                                  # [Hk, G, n, len]
    see = b.sees(s)
    w = torch.softmax(x, -1).masked_fill(~see, 0)
    v = b.entries(b.v, s)[:, None]
    ev = torch.exp2(b.entries(b.vs, s) - 127)[:, None, None]           # [Hk, 1, 1, len]
    a, n = b.at[s], b.chunks[s]
    q = b.q[a:a + n].double().abs().amax(-1).transpose(0, 1).unflatten(0, (b.Hk, b.G))
    k = b.entries(b.k, s).abs().sum(-1)[:, None, None]
    length = x.shape[-1]
    ds = (b.D * 2.0 ** -23 * size + length * 2.0 ** -23 + 2.0 ** -21
          + 2.0 ** -21 * b.scale * q[..., None] * k)
    out, mass = w @ v, w @ v.abs()
    tol = torch.finfo(b.type).eps / 2 * out.abs() + 2.0 ** -11 * mass
    tol += (w * ds) @ v.abs() + (w * ds).sum(-1, keepdim=True) * mass
    tol *= 1 + 2.0 ** -6                                   # (products of two errors)
    tol += min(length, 512) * 448 * 2.0 ** -20 * (w * ev).amax(-1, keepdim=True)
    if b.type == F16:
        tol += 2.0 ** -25                                  # the output below fp16's normal numbers
    back = lambda t: t.flatten(0, 1).transpose(0, 1)
    return back(out), back(tol)


def check(b, out):
    for s in range(len(b.lens)):
        a, n = b.at[s], b.chunks[s]
        want, tol = terms(b, s)
        got = out[a:a + n].double()
        fits = want.abs() < (6e4 if b.type == F16 else 1e38)
        assert fits.any()
        off = ((got - want).abs() / tol)[fits]
        assert (off <= 1).all(), (s, float(off.max()))


def plant(b, s, j, up, drop):
    """Entry j of sequence s: values 2^up larger, a score `drop` below what the rest of its key gives."""
    p, r = (int(t[j]) for t in b.where(s))
    b.vs[p, :, r] += up
    b.v[p, :, r] *= 2.0 ** up
    y = torch.zeros((b.Hk, b.D), dtype=torch.float64, device="cuda")
    y[:, 0] = -drop / (4 * b.scale)
    c, byte = quantise(y)
    b.k8[p, :, r], b.ks[p, :, r] = c.to(E4M3), byte.to(torch.uint8)
    b.k[p, :, r] = value(c, byte)


def batch(type, D, G, chunks, lens, **kw):
    b = Packed(type, D, 2, G, 64, chunks, lens, **kw)
    b.q[..., 0] = 4                                        # one dim that only planted keys use
    b.k8.view(torch.uint8)[..., 0] = 0
    b.k[..., 0] = 0
    return b


@pytest.mark.parametrize("type", [BF16, F16])
@pytest.mark.parametrize("D,G,chunk", [(128, 1, 1), (64, 4, 1), (128, 8, 1), (64, 16, 1), (128, 20, 1),
                                       (128, 1, 3), (64, 5, 3), (128, 16, 4)])
@pytest.mark.parametrize("up,drop", [(10, 2), (20, 10), (30, 15), (30, 21), (30, 200), (60, 30), (60, 200),
                                     (100, 60)])
def test_a_large_value_that_hardly_weighs(type, D, G, chunk, up, drop):
    b = batch(type, D, G, [chunk, chunk], [3000, 700], seed=up + drop)
    plant(b, 0, 1311, up, drop)
    plant(b, 1, 2, up, drop)
    check(b, b.kv().attention(b.q, b.cu, b.len, max_q=chunk))


@pytest.mark.parametrize("type", [BF16, F16])
@pytest.mark.parametrize("G", [1, 4, 10])
def test_a_large_value_that_only_later_rows_see(type, G):
    b = batch(type, 128, G, [5], [1111])
    plant(b, 0, 1108, 40, 60)
    out = b.kv().attention(b.q, b.cu, b.len, max_q=5)
    check(b, out)
    # the rows before it: the same bits whatever it holds
    p, r = (int(t[1108]) for t in b.where(0))
    for scale in (0, 127, 254, 255):
        b.vs[p, :, r] = scale
        again = b.kv().attention(b.q, b.cu, b.len, max_q=5)
        assert torch.equal(again[:2], out[:2])


@pytest.mark.parametrize("type,most", [(BF16, 40), (BF16, 3), (F16, 6)])
@pytest.mark.parametrize("D,G,chunk,window", [(128, 1, 1, 0), (64, 2, 2, 300), (128, 8, 1, 0), (128, 6, 4, 77),
                                              (64, 32, 2, 0)])
def test_powers_of_two_all_over_the_range(type, most, D, G, chunk, window):
    b = Packed(type, D, 2, G, 16, [chunk, chunk], [2222, 300], window=window)
    up = torch.randint(-most, most + 1, b.vs.shape, generator=b.g, device="cuda")
    b.vs = (b.vs.int() + up).to(torch.uint8)
    b.v *= torch.exp2(up.double())[..., None]
    check(b, b.kv().attention(b.q, b.cu, b.len, max_q=chunk, window=window))


@pytest.mark.parametrize("type", [BF16, F16])
def test_later_large_values_are_right_for_the_rows_that_see_them(type):
    """In fp16 as well, where the sum fits it."""
    b = Packed(type, 128, 1, 2, 16, [6], [90], seed=4)
    p, r = (t[87:] for t in b.where(0))
    b.vs[p, :, r] += 9
    b.v[p, :, r] *= 2.0 ** 9
    out, lse = b.kv().attention(b.q, b.cu, b.len, max_q=6, with_lse=True)
    b.check(out, lse)
    check(b, out)


def test_a_value_whose_weight_underflows_takes_nothing_from_the_rest():
    b = batch(BF16, 128, 1, [1], [400])
    plant(b, 0, 7, 90, 2000)
    out = b.kv().attention(b.q, b.cu, b.len, max_q=1)
    assert math.isfinite(float(out.float().norm()))
    check(b, out)
