"""What workgroup 0 of a launch with adapters leaves behind (csrc/hand_off.h): a
late word marks its own memory, and no other. Compiled for the host."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
#include "hand_off.h"
using mxg::hand_off;
// (scratch late, workspace late)
static_assert(!hand_off(false, false).mark_scratch && !hand_off(false, false).mark_workspace &&
              hand_off(false, false).advance_workspace, "nothing late");
static_assert(hand_off(true, false).mark_scratch && !hand_off(true, false).mark_workspace &&
              hand_off(true, false).advance_workspace, "a helping workgroup late");
static_assert(!hand_off(false, true).mark_scratch && hand_off(false, true).mark_workspace &&
              !hand_off(false, true).advance_workspace, "a split-K workgroup late");
static_assert(hand_off(true, true).mark_scratch && hand_off(true, true).mark_workspace &&
              !hand_off(true, true).advance_workspace, "both late");
int main() { return 0; }
"""


def test_hand_off(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src = tmp_path / "hand_off.cc"
    src.write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-fsyntax-only",
                        "-I" + os.path.join(ROOT, "mxfp8_decode_gemm_amd", "csrc"), str(src)],
                       capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
