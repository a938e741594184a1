"""Well-formed paged-cache calls where there is no GPU fail as CUDA calls, not as bad arguments."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# (its own process, from which every device is hidden: nothing can be launched with these addresses)
CHILD = """
import test_paged_abi as t
import full_duplex_speech_lockstep_gb300 as pp
for f in (t.append, lambda kv: t.attention(kv, out=2 * t.A), t.mass,
          lambda kv: t.evict(kv, t.cache(k=2 * t.A, v=2 * t.A)),
          lambda kv: t.attention(kv, out=2 * t.A, max_q=300)):
    print(f(t.cache()))
"""


def test_calls_without_a_device_fail_as_cuda_calls():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="-1",
               PYTHONPATH=os.pathsep.join([ROOT, os.path.join(ROOT, "tests")]))
    got = subprocess.check_output([sys.executable, "-c", CHILD], env=env, text=True, cwd=ROOT)
    assert got.split() == ["-5"] * 5
