"""Scratch of long chunks over an 8-bit cache: a 16-bit copy of some sequences at a time (no GPU needed)."""
import pytest

import full_duplex_speech_lockstep_gb300 as pp
from test_packed_abi import cache
from test_paged_abi import cache as wide

LIMIT = 2 << 30


def scratch(n_seqs, entries, heads=32, dim=128, page=64, max_q=100, T=100):
    size = dict(n_seqs=n_seqs, table_ld=entries // page, n_kv_heads=heads, head_dim=dim, page_size=page)
    kv = cache(page_stride=heads * page * dim, scale_stride=heads * page, **size)
    # what the 16-bit call takes for the same sequences: parts of outputs
    own = pp.pp_paged_attention_scratch_bytes(wide(page_stride=heads * page * dim, **size), heads, T, max_q, 0)
    return pp.pp_packed_attention_scratch_bytes(kv, heads, T, max_q, 0), own


@pytest.mark.parametrize("n_seqs,entries", [(64, 65536), (64, 3008), (2048, 3008), (3, 262144), (1, 65536),
                                            (300, 4096)])
def test_a_copy_is_bounded(n_seqs, entries):
    got, own = scratch(n_seqs, entries)
    one = entries * 32 * 128 * 4
    table = n_seqs * (entries // 64) * 4 + 256
    assert got <= max(LIMIT, one) + own + table


def test_few_sequences_are_copied_at_once():
    got, own = scratch(8, 3008)
    copy = 8 * 3008 * 32 * 128 * 4
    assert copy < got <= copy + own + 8 * 47 * 4 + 256


def test_sequences_are_shared_out_evenly():
    # 43 fit: 44 are taken as 22 and 22
    per = 3008 * 32 * 128 * 4
    for n_seqs, at_once in ((43, 43), (44, 22), (64, 32), (86, 43), (87, 29)):
        got, own = scratch(n_seqs, 3008)
        assert at_once * per < got <= at_once * per + own + at_once * 47 * 4 + 256


def test_short_chunks_take_no_copy():
    got, own = scratch(64, 65536, max_q=1, T=64)
    assert got < LIMIT // 2
