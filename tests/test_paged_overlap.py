"""Calls whose outputs lie over what they read are refused on the host (no GPU needed).  Every call
here is refused for another reason at the latest where there is no device: see the child."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# five rows of 4 x 128 values of two bytes, 1024 bytes each, at A; the call runs in a process from
# which every device is hidden, so nothing can be launched with these addresses
CHILD = """
import sys
import test_paged_abi as t
A = t.A
print(eval(sys.argv[1]))
"""


def call(what):
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="-1",
               PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    return int(subprocess.check_output([sys.executable, "-c", CHILD, what], env=env, text=True,
                                       cwd=ROOT))


@pytest.mark.parametrize("at,stride,meets", [
    ("A", 512, True), ("A + 4096", 512, True), ("A + 5104", 512, True), ("A + 5120", 512, False),
    ("A - 5120", 512, False), ("A - 5104", 512, True), ("A", 8192, True),
    ("A + 1024", 8192, False),      # between the first row and the second
    ("A + 11264", 8192, False), ("A + 11280", 8192, True), ("A + 4 * 16384 + 1024", 8192, False)])
def test_attention_refuses_an_output_over_its_queries(at, stride, meets):
    assert call("t.attention(t.cache(), qs=%d, out=%s)" % (stride, at)) == (-1 if meets else -5)


def test_evict_refuses_the_cache_itself():
    assert call("t.evict(t.cache(), t.cache())") == -1
    assert call("t.evict(t.cache(), t.cache(table=2 * A))") == -5
    assert call("t.evict(t.cache(), t.cache(k=2 * A, v=2 * A))") == -5
