"""A lookup that failed once is tried again (the driver's tensor-map encoder is found so)."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "full_duplex_speech_lockstep_gb300", "csrc")

MAIN = """
#include <stdio.h>
#include "pp_found.cuh"
typedef int (*Fn)();
static int one() { return 1; }
static int tries = 0;
static Fn lookup() { return ++tries < 3 ? nullptr : one; }
int main() {
  static pp::Found<Fn> fn;
  for (int i = 0; i < 5; ++i) printf("%d ", fn.get(lookup) == one);
  printf("%d\\n", tries);
  return 0;
}
"""


def test_a_failed_lookup_is_tried_again_and_a_found_one_is_kept(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "main.cpp", tmp_path / "main"
    src.write_text(MAIN)
    subprocess.check_call(["g++", "-std=c++17", "-Wall", "-I", CSRC, str(src), "-o", str(exe)])
    assert subprocess.check_output([str(exe)], text=True).split() == ["0", "0", "1", "1", "1", "3"]
