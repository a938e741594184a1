"""pp_packed_read refuses a destination over what it reads, and no other one (no GPU needed): pools end
with their last page, not a stride after it.  -1: refused; -5: accepted, and no device to run on."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# ten pages of 2 x 64 x 128 codes (16 KB), of 2 x 64 scales, and of 32 KB of values, each apart by some
# strides; in a process from which every device is hidden, so nothing can be launched with these addresses
CHILD = """
import sys
import test_packed_abi as t
import test_paged_abi as w
B = 1 << 40
PAGE, ROWS = 2 * 64 * 128, 2 * 64
def read(kv, to, ln=B << 8):
    base = dict(k=B, v=2 * B, k_scale=3 * B, v_scale=4 * B, table=5 * B)
    base.update(kv)
    dest = dict(k=6 * B, v=7 * B, table=8 * B, mass=9 * B)
    dest.update(to)
    return t.read(t.cache(**base), w.cache(**dest), ln)
for line in sys.argv[1:]:
    print(eval(line))
"""

CASES = [
    # right behind the last page of a pool with gaps between its pages, and 16 bytes into it
    ("read(dict(page_stride=4 * PAGE), dict(k=B + 9 * 4 * PAGE + PAGE))", -5),
    ("read(dict(page_stride=4 * PAGE), dict(k=B + 9 * 4 * PAGE + PAGE - 16))", -1),
    ("read(dict(page_stride=4 * PAGE), dict(v=2 * B + 9 * 4 * PAGE + PAGE))", -5),
    ("read(dict(page_stride=4 * PAGE), dict(v=2 * B + 9 * 4 * PAGE + PAGE - 16))", -1),
    ("read(dict(scale_stride=48 * ROWS), dict(k=3 * B + 9 * 48 * ROWS + ROWS))", -5),
    ("read(dict(scale_stride=48 * ROWS), dict(k=3 * B + 9 * 48 * ROWS + ROWS - 16))", -1),
    ("read(dict(scale_stride=48 * ROWS), dict(v=4 * B + 9 * 48 * ROWS + ROWS))", -5),
    # the source right behind the destination's last page
    ("read(dict(k=6 * B + 9 * 2 * 8 * PAGE + 2 * PAGE), dict(page_stride=8 * PAGE))", -5),
    ("read(dict(k=6 * B + 9 * 2 * 8 * PAGE + 2 * PAGE - 16), dict(page_stride=8 * PAGE))", -1),
    # dense pools: next to each other, and by 16 bytes over each other
    ("read({}, dict(k=B + 10 * PAGE))", -5),
    ("read({}, dict(k=B + 10 * PAGE - 16))", -1),
    ("read({}, dict(v=B - 20 * PAGE))", -5),
    ("read({}, dict(v=B - 20 * PAGE + 16))", -1),
    # many pages far apart: a size that is past 64 bits still meets
    ("read(dict(n_pages=2 ** 31 - 1, page_stride=2 ** 38 - 16, k=16 * B), dict(k=17 * B))", -1),
    ("read(dict(n_pages=2 ** 27 + 1, page_stride=2 ** 37, k=16 * B), dict(k=17 * B))", -1),
    # the tables and lengths that a call reads while it writes
    ("read(dict(table=6 * B + 64), {})", -1),
    ("read({}, dict(table=7 * B + 4))", -1),
    ("read({}, {}, 6 * B + 128)", -1),
    ("read(dict(table=8 * B), {})", -5),          # one table for both caches
]


@pytest.fixture(scope="module")
def answers():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="-1",
               PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    out = subprocess.check_output([sys.executable, "-c", CHILD] + [c for c, _ in CASES], env=env, text=True,
                                  cwd=ROOT)
    return dict(zip((c for c, _ in CASES), map(int, out.split())))


@pytest.mark.parametrize("case,want", CASES)
def test_read_refuses_what_meets_and_nothing_else(answers, case, want):
    assert answers[case] == want
