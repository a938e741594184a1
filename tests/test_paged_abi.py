"""The paged-cache calls refuse malformed arguments on the host, before any CUDA call (no GPU
needed); the binding's structure mirrors the header's."""
import ctypes
import os
import shutil
import subprocess

import pytest

import full_duplex_speech_lockstep_gb300 as pp

A = 1 << 20          # a well-aligned address that is never followed


def cache(**kw):
    f = dict(k=A, v=A, mass=A, table=A, page_stride=2 * 64 * 128, n_pages=10, page_size=64,
             n_kv_heads=2, head_dim=128, type=pp.PP_BF16, n_seqs=3, table_ld=4)
    f.update(kw)
    return pp.pp_paged_kv(**f)


BAD_CACHES = [dict(k=0), dict(v=0), dict(table=0), dict(k=A + 8), dict(v=A + 2), dict(table=A + 1),
              dict(mass=A + 2), dict(type=pp.PP_F32), dict(type=7), dict(head_dim=32),
              dict(head_dim=96), dict(head_dim=256), dict(page_size=8), dict(page_size=48),
              dict(page_size=512), dict(page_size=0), dict(n_kv_heads=0), dict(n_pages=0),
              dict(n_seqs=0), dict(n_seqs=2049), dict(table_ld=0), dict(table_ld=1 << 30),
              dict(page_stride=2 * 64 * 128 - 8), dict(page_stride=2 * 64 * 128 + 4),
              dict(page_stride=1 << 40)]


def append(kv, q=A, qs=4 * 128, k=A, ks=2 * 128, v=A, vs=2 * 128, in_type=pp.PP_BF16, qa=None,
           ka=None, eps=1e-5, base=1e4, rot=128, halves=0, pos=None, cu=A, ln=A, T=5, H=4, out=A):
    return pp.lib().pp_paged_append(ctypes.byref(kv) if kv else None, q, qs, k, ks, v, vs, in_type,
                                    qa, ka, eps, base, rot, halves, pos, cu, ln, T, H, out, None,
                                    None)


def attention(kv, q=A, qs=4 * 128, cu=A, ln=A, T=5, max_q=5, H=4, scale=0.1, window=0, out=A,
              lse=None, scratch=A, nbytes=1 << 40):
    return pp.lib().pp_paged_attention(ctypes.byref(kv) if kv else None, q, qs, cu, ln, T, max_q, H,
                                       scale, window, out, lse, None, scratch, nbytes, None)


def mass(kv, q=A, qs=4 * 128, lse=A, cu=A, ln=A, T=5, max_q=5, H=4, scale=0.1, window=0, decay=1.0):
    return pp.lib().pp_paged_mass(ctypes.byref(kv) if kv else None, q, qs, lse, cu, ln, T, max_q, H,
                                  scale, window, decay, None, None)


def evict(kv, to, ln=A, budget=4, recent=2, to_len=A, kept=A):
    return pp.lib().pp_paged_evict(ctypes.byref(kv) if kv else None, ln, budget, recent,
                                   ctypes.byref(to) if to else None, to_len, kept, None, None)


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_every_call_refuses_a_bad_cache(bad):
    kv = cache(**bad)
    assert append(kv) == pp.PP_EINVAL
    assert attention(kv) == pp.PP_EINVAL
    assert mass(kv) == pp.PP_EINVAL
    assert evict(kv, cache()) == pp.PP_EINVAL
    assert evict(cache(), kv) == pp.PP_EINVAL
    with pytest.raises(pp.PPError):
        pp.pp_paged_attention_scratch_bytes(kv, 4, 3, 1, 0)


def test_null_cache():
    assert append(None) == attention(None) == mass(None) == pp.PP_EINVAL
    assert evict(None, cache()) == evict(cache(), None) == pp.PP_EINVAL


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(k=0), dict(v=0), dict(out=0), dict(cu=0), dict(ln=0), dict(q=A + 8),
    dict(k=A + 2), dict(v=A + 4), dict(out=A + 8), dict(qa=A + 4), dict(ka=A + 8), dict(pos=A + 2),
    dict(cu=A + 2), dict(ln=A + 1), dict(qs=4 * 128 - 8), dict(ks=128), dict(vs=128),
    dict(qs=4 * 128 + 4), dict(in_type=pp.PP_F16), dict(in_type=5), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(base=0.5), dict(base=float("nan")),
    dict(base=float("inf")), dict(rot=127), dict(rot=130), dict(rot=-2), dict(T=-1), dict(H=3),
    dict(H=0), dict(H=130), dict(T=1 << 29)], ids=str)
def test_append_refuses(bad):
    assert append(cache(), **bad) == pp.PP_EINVAL


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(out=0), dict(cu=0), dict(ln=0), dict(scratch=0), dict(q=A + 8),
    dict(out=A + 8), dict(lse=A + 2), dict(scratch=A + 128), dict(qs=4 * 128 - 8),
    dict(qs=4 * 128 + 4), dict(qs=1 << 40), dict(T=-1), dict(max_q=0), dict(H=5), dict(H=130),
    dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(window=-1)], ids=str)
def test_attention_refuses(bad):
    assert attention(cache(), **bad) == pp.PP_EINVAL


def test_attention_refuses_small_scratch():
    n = pp.pp_paged_attention_scratch_bytes(cache(), 4, 5, 5, 0)
    assert attention(cache(), nbytes=n - 1) == pp.PP_E_NOSPACE


def test_scratch_grows_with_the_table():
    one = pp.pp_paged_attention_scratch_bytes(cache(table_ld=400), 4, 9, 1, 0)
    assert pp.pp_paged_attention_scratch_bytes(cache(table_ld=4000), 4, 9, 1, 0) > one
    assert pp.pp_paged_attention_scratch_bytes(cache(table_ld=400), 4, 9, 1, 200) < one
    for bad in [dict(n_heads=5), dict(n_heads=0), dict(max_q=0), dict(window=-1)]:
        a = dict(n_heads=4, max_q=1, window=0)
        a.update(bad)
        with pytest.raises(pp.PPError):
            pp.pp_paged_attention_scratch_bytes(cache(), a["n_heads"], 9, a["max_q"],
                                                a["window"])


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(lse=0), dict(cu=0), dict(ln=0), dict(q=A + 8), dict(lse=A + 1),
    dict(qs=4 * 128 - 8), dict(T=-1), dict(max_q=0), dict(H=5), dict(scale=0.0),
    dict(scale=float("nan")), dict(window=-1), dict(decay=-0.1), dict(decay=1.5),
    dict(decay=float("nan"))], ids=str)
def test_mass_refuses(bad):
    assert mass(cache(), **bad) == pp.PP_EINVAL


def test_mass_and_evict_need_the_weights():
    assert mass(cache(mass=0)) == pp.PP_EINVAL
    assert evict(cache(mass=0), cache()) == pp.PP_EINVAL


@pytest.mark.parametrize("bad", [
    dict(ln=0), dict(to_len=0), dict(kept=0), dict(ln=A + 2), dict(to_len=A + 1), dict(kept=A + 2),
    dict(budget=0), dict(budget=-3), dict(recent=-1), dict(recent=5)], ids=str)
def test_evict_refuses(bad):
    assert evict(cache(), cache(), **bad) == pp.PP_EINVAL


@pytest.mark.parametrize("to", [dict(type=pp.PP_F16), dict(head_dim=64), dict(n_kv_heads=1),
                                dict(n_seqs=2)], ids=str)
def test_evict_refuses_another_kind_of_destination(to):
    assert evict(cache(), cache(**to)) == pp.PP_EINVAL


def test_evict_refuses_a_destination_that_is_too_narrow():
    assert evict(cache(), cache(table_ld=1), budget=65, recent=0) == pp.PP_E_RANGE
    # the source cannot hold more than 4 * 64 entries, whatever the budget
    assert evict(cache(), cache(table_ld=3), budget=10000, recent=0) == pp.PP_E_RANGE


@pytest.mark.parametrize("budget", [(1 << 28) + 1, 2**31 - 1])
def test_evict_refuses_a_budget_beyond_any_table(budget):
    assert evict(cache(), cache(), budget=budget, recent=0) == pp.PP_EINVAL


def test_no_rows_is_no_work():
    assert append(cache(), T=0, q=0, k=0, v=0, out=0) == pp.PP_OK
    assert attention(cache(), T=0, q=0, out=0, scratch=0) == pp.PP_OK


def test_structure_matches_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "pp.h"', 'int main(void) {',
             '  printf("%zu\\n", sizeof(pp_paged_kv));']
    lines += ['  printf("%%zu\\n", offsetof(pp_paged_kv, %s));' % f[0]
              for f in pp.pp_paged_kv._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", inc, str(src), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    assert got == [ctypes.sizeof(pp.pp_paged_kv)] + [getattr(pp.pp_paged_kv, f[0]).offset
                                                     for f in pp.pp_paged_kv._fields_]
