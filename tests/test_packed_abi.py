"""The calls of the 8-bit paged cache and of token log probabilities refuse malformed arguments on
the host, before any CUDA call (no GPU needed); the binding's structure mirrors the header's."""
import ctypes
import os
import shutil
import subprocess
import sys

import pytest

import full_duplex_speech_lockstep_gb300 as pp
from test_paged_abi import A
from test_paged_abi import cache as wide

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def cache(**kw):
    f = dict(k=A, v=A, k_scale=A, v_scale=A, table=A, page_stride=2 * 64 * 128, scale_stride=2 * 64,
             n_pages=10, page_size=64, n_kv_heads=2, head_dim=128, type=pp.PP_BF16, n_seqs=3,
             table_ld=4)
    f.update(kw)
    return pp.pp_packed_kv(**f)


BAD_CACHES = [dict(k=0), dict(v=0), dict(k_scale=0), dict(v_scale=0), dict(table=0), dict(k=A + 8),
              dict(v=A + 2), dict(k_scale=A + 8), dict(v_scale=A + 1), dict(table=A + 1),
              dict(type=pp.PP_F32), dict(type=7), dict(head_dim=32), dict(head_dim=96),
              dict(head_dim=256), dict(page_size=8), dict(page_size=48), dict(page_size=512),
              dict(page_size=0), dict(n_kv_heads=0), dict(n_kv_heads=1025), dict(n_pages=0),
              dict(n_seqs=0), dict(n_seqs=2049), dict(table_ld=0), dict(table_ld=1 << 30),
              dict(page_stride=2 * 64 * 128 - 16), dict(page_stride=2 * 64 * 128 + 8),
              dict(page_stride=1 << 40), dict(scale_stride=2 * 64 - 16),
              dict(scale_stride=2 * 64 + 8), dict(scale_stride=1 << 40)]


def append(kv, q=A, qs=4 * 128, k=A, ks=2 * 128, v=A, vs=2 * 128, in_type=pp.PP_BF16, qa=None,
           ka=None, eps=1e-5, base=1e4, rot=128, halves=0, pos=None, cu=A, ln=A, T=5, H=4, out=A):
    return pp.lib().pp_packed_append(ctypes.byref(kv) if kv else None, q, qs, k, ks, v, vs, in_type,
                                     qa, ka, eps, base, rot, halves, pos, cu, ln, T, H, out, None,
                                     None)


def attention(kv, q=A, qs=4 * 128, cu=A, ln=A, T=5, max_q=5, H=4, scale=0.1, window=0, out=2 * A,
              lse=None, scratch=A, nbytes=1 << 40):
    return pp.lib().pp_packed_attention(ctypes.byref(kv) if kv else None, q, qs, cu, ln, T, max_q, H,
                                        scale, window, out, lse, None, scratch, nbytes, None)


def read(kv, to, ln=A):
    return pp.lib().pp_packed_read(ctypes.byref(kv) if kv else None, ln,
                                   ctypes.byref(to) if to else None, None, None)


def other(**kw):
    return wide(k=1 << 30, v=1 << 31, **kw)


def score(x=A, type=pp.PP_F32, ld=100, rows=3, inner=1, inner_ld=0, n=100, tokens=A, token_ld=1,
          top=0, lp=A, ent=None, ti=None, tl=None):
    return pp.lib().pp_token_logprobs(x, type, ld, rows, inner, inner_ld, n, tokens, token_ld, top,
                                      lp, ent, ti, tl, None, None)


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_every_call_refuses_a_bad_cache(bad):
    kv = cache(**bad)
    assert append(kv) == attention(kv) == read(kv, other()) == pp.PP_EINVAL
    with pytest.raises(pp.PPError):
        pp.pp_packed_attention_scratch_bytes(kv, 4, 3, 1, 0)


def test_null_cache():
    assert append(None) == attention(None) == read(None, other()) == pp.PP_EINVAL
    assert read(cache(), None) == pp.PP_EINVAL


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(k=0), dict(v=0), dict(out=0), dict(cu=0), dict(ln=0), dict(q=A + 8),
    dict(k=A + 2), dict(v=A + 4), dict(out=A + 8), dict(qa=A + 4), dict(ka=A + 8), dict(pos=A + 2),
    dict(cu=A + 2), dict(ln=A + 1), dict(qs=4 * 128 - 8), dict(ks=128), dict(vs=128),
    dict(qs=4 * 128 + 4), dict(in_type=pp.PP_F16), dict(in_type=5), dict(eps=-1.0),
    dict(eps=float("nan")), dict(base=0.5), dict(base=float("inf")), dict(rot=127), dict(rot=130),
    dict(rot=-2), dict(T=-1), dict(H=3), dict(H=0), dict(H=130), dict(T=1 << 29)], ids=str)
def test_append_refuses(bad):
    assert append(cache(), **bad) == pp.PP_EINVAL


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(out=0), dict(cu=0), dict(ln=0), dict(scratch=0), dict(q=A + 8),
    dict(out=A + 8), dict(lse=A + 2), dict(scratch=A + 128), dict(qs=4 * 128 - 8),
    dict(qs=4 * 128 + 4), dict(qs=1 << 40), dict(T=-1), dict(max_q=0), dict(H=5), dict(H=130),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(window=-1), dict(out=A), dict(out=A + 4 * 4 * 128 * 2)], ids=str)
def test_attention_refuses(bad):
    assert attention(cache(), **bad) == pp.PP_EINVAL
    assert attention(cache(), **{"max_q": 300, **bad}) == pp.PP_EINVAL


@pytest.mark.parametrize("max_q", [1, 5, 300])
def test_attention_refuses_small_scratch(max_q):
    n = pp.pp_packed_attention_scratch_bytes(cache(), 4, 5, max_q, 0)
    assert attention(cache(), max_q=max_q, nbytes=n - 1) == pp.PP_E_NOSPACE


def test_scratch_refuses():
    for bad in [dict(n_heads=5), dict(n_heads=0), dict(max_q=0), dict(window=-1), dict(T=-1)]:
        a = dict(n_heads=4, T=9, max_q=1, window=0)
        a.update(bad)
        with pytest.raises(pp.PPError):
            pp.pp_packed_attention_scratch_bytes(cache(), *a.values())


@pytest.mark.parametrize("to", [dict(type=pp.PP_F16), dict(head_dim=64), dict(n_kv_heads=1),
                                dict(n_seqs=2), dict(table=0), dict(page_size=20)], ids=str)
def test_read_refuses_another_kind_of_destination(to):
    assert read(cache(), other(**to)) == pp.PP_EINVAL


@pytest.mark.parametrize("bad", [dict(ln=0), dict(ln=A + 2)], ids=str)
def test_read_refuses_its_lengths(bad):
    assert read(cache(), other(), **bad) == pp.PP_EINVAL


@pytest.mark.parametrize("name", ["k", "v"])
@pytest.mark.parametrize("source", ["k", "v", "k_scale", "v_scale"])
def test_read_refuses_memory_that_both_caches_hold(name, source):
    base = {"k": 1 << 32, "v": 1 << 33, "k_scale": 1 << 34, "v_scale": 1 << 35}
    kv = cache(**base)
    last = 9 * (kv.page_stride if source in "kv" else kv.scale_stride)
    to = {"k": 1 << 36, "v": 1 << 37}
    to[name] = base[source] + last
    assert read(kv, wide(**to)) == pp.PP_EINVAL
    to[name] = base[source] - 16
    assert read(kv, wide(**to)) == pp.PP_EINVAL


@pytest.mark.parametrize("bad", [
    dict(x=0), dict(x=A + 2), dict(type=3), dict(type=-1), dict(ld=-1), dict(inner_ld=-1),
    dict(token_ld=-1), dict(ld=1 << 40), dict(rows=-1), dict(inner=0), dict(n=0),
    dict(n=(1 << 24) + 1), dict(top=-1), dict(top=65), dict(tokens=0), dict(tokens=A + 2),
    dict(lp=A + 1), dict(ent=A + 2), dict(ti=A + 2), dict(tl=A + 3), dict(rows=1 << 28),
    dict(rows=1 << 20, inner=1 << 8), dict(type=pp.PP_BF16, x=A + 1)], ids=str)
def test_logprobs_refuses(bad):
    assert score(**bad) == pp.PP_EINVAL


def test_no_rows_is_no_work():
    assert append(cache(), T=0, q=0, k=0, v=0, out=0) == pp.PP_OK
    assert attention(cache(), T=0, q=0, out=0, scratch=0) == pp.PP_OK
    assert score(rows=0, x=0) == pp.PP_OK


def test_structure_matches_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "pp.h"', 'int main(void) {',
             '  printf("%zu\\n", sizeof(pp_packed_kv));']
    lines += ['  printf("%%zu\\n", offsetof(pp_packed_kv, %s));' % f[0]
              for f in pp.pp_packed_kv._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                           str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    assert got == [ctypes.sizeof(pp.pp_packed_kv)] + [getattr(pp.pp_packed_kv, f[0]).offset
                                                      for f in pp.pp_packed_kv._fields_]


# (its own process, from which every device is hidden: nothing can be launched with these addresses)
CHILD = """
import test_packed_abi as t
for f in (t.append, t.attention, lambda kv: t.attention(kv, max_q=300),
          lambda kv: t.read(kv, t.other()), lambda kv: t.score()):
    print(f(t.cache()))
"""


def test_calls_without_a_device_fail_as_cuda_calls():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="-1",
               PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    got = subprocess.check_output([sys.executable, "-c", CHILD], env=env, text=True, cwd=ROOT)
    assert got.split() == ["-5"] * 5


def test_logprobs_of_host_tensors_is_refused():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        pp.token_logprobs(torch.zeros(3, 5))


def test_caches_of_one_kind_do_not_pass_for_the_other():
    wide_kv, packed = (c.__new__(c) for c in (pp.PagedKV, pp.PagedKV8))
    wide_kv.index = packed.index = 0
    wide_kv.mass, wide_kv.torch = object(), None
    for call in (lambda: wide_kv.evict(None, 4, 2, packed), lambda: packed.read(None, packed),
                 lambda: packed.read(None, None)):
        with pytest.raises(ValueError, match="expected a PagedKV"):
            call()
