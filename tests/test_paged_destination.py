"""What a cache's evict and read take as their destination: a 16-bit cache, a PagedKV or an object of the
caller's with the same `ref` and `index`; no 8-bit cache (no GPU needed)."""
import ctypes
import types

import pytest

import full_duplex_speech_lockstep_gb300 as pp

torch = pytest.importorskip("torch")


class Recorder:
    """A cache whose calls are kept, not made."""

    def __new__(cls, kind):
        kv = kind.__new__(kind)
        kv.torch, kv.index, kv.device, kv.n, kv.heads = torch, -1, torch.device("cpu"), 3, 2
        kv.mass = kv.status = torch.zeros(1, dtype=torch.int32)
        kv.calls = []
        kv._call = lambda *args: kv.calls.append(args)
        kv._bind(pp.pp_packed_kv() if kind is pp.PagedKV8 else pp.pp_paged_kv())
        return kv


LENS = torch.zeros(3, dtype=torch.int32)


def calls_with(to):
    wide, packed = Recorder(pp.PagedKV), Recorder(pp.PagedKV8)
    wide.evict(LENS, 4, 2, to)
    packed.read(LENS, to)
    return wide.calls + packed.calls


def test_a_cache_of_16_bits_is_taken():
    to = Recorder(pp.PagedKV)
    evict, read = calls_with(to)
    assert evict[0] == "pp_paged_evict" and to.ref in evict
    assert read[0] == "pp_packed_read" and to.ref in read


def test_an_object_with_the_same_structure_is_taken():
    to = types.SimpleNamespace(ref=ctypes.byref(pp.pp_paged_kv()), index=-1)
    evict, read = calls_with(to)
    assert to.ref in evict and to.ref in read


@pytest.mark.parametrize("to", [None, types.SimpleNamespace(index=-1)], ids=str)
def test_what_is_no_cache_is_refused(to):
    for call in (lambda: Recorder(pp.PagedKV).evict(LENS, 4, 2, to),
                 lambda: Recorder(pp.PagedKV8).read(LENS, to)):
        with pytest.raises(ValueError, match="expected a PagedKV"):
            call()


def test_a_cache_of_8_bits_is_refused():
    to = Recorder(pp.PagedKV8)
    for call in (lambda: Recorder(pp.PagedKV).evict(LENS, 4, 2, to),
                 lambda: Recorder(pp.PagedKV8).read(LENS, to)):
        with pytest.raises(ValueError, match="expected a PagedKV"):
            call()


def test_a_cache_on_another_device_is_refused():
    to = Recorder(pp.PagedKV)
    to.index = 1
    with pytest.raises(ValueError, match="one device"):
        Recorder(pp.PagedKV).evict(LENS, 4, 2, to)
