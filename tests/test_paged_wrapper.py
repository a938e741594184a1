"""What PagedKV hands to the library, as far as it shows without a GPU."""
import pytest

import full_duplex_speech_lockstep_gb300 as pp


@pytest.mark.parametrize("rows", [0, 1, 4, 1000])
@pytest.mark.parametrize("max_q", [1, 5, 8, 300])
def test_a_callers_max_q_is_handed_on(max_q, rows):
    assert pp.PagedKV._longest(max_q, rows) == max_q


def test_without_max_q_all_rows_are_one_chunk():
    assert [pp.PagedKV._longest(None, rows) for rows in (0, 1, 64)] == [1, 1, 64]


@pytest.mark.parametrize("max_q,handed", [(0, 1), (-3, 1), (2 ** 40, 2 ** 31 - 1)])
def test_max_q_stays_within_what_the_library_takes(max_q, handed):
    assert pp.PagedKV._longest(max_q, 7) == handed
