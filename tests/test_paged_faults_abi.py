"""The paged calls' failure-detection switch checks its arguments (no GPU needed)."""
import pytest

import full_duplex_speech_lockstep_gb300 as pp


@pytest.mark.parametrize("polls,withhold", [(-1, 0), (0, -1), (4096, 2)])
def test_other_numbers_are_refused(polls, withhold):
    assert pp.lib().pp_test_paged_faults(polls, withhold) == pp.PP_EINVAL


def test_the_reset_is_taken():
    assert pp.lib().pp_test_paged_faults(0, 0) == pp.PP_OK
