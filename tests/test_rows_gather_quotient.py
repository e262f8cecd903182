"""csrc/gather_quotient.h: an entry of an order over a router's top_k, by a product (mxmoe_grouped allows entries up to
2^24 rows times 32). Compiled for the host."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
#include "gather_quotient.h"
#include <cstdio>
using namespace mxg;
int main() {
  for (int g = 2; g <= 32; ++g) {
    const GatherQuotient q = gather_quotient(g);
    // A quotient that is too large shows first before a multiple, and the further up the sooner.
    const uint32_t top = 0x7FFFFFFFu / g;
    for (uint32_t k = 0; k <= top; k += k + 100000 < top && k > 100000 ? 997 : 1)
      for (int d = -1; d <= 1; ++d) {
        const int64_t o = (int64_t)k * g + d;
        if (o < 0 || o > 0x7FFFFFFF) continue;
        if (over_gather((uint32_t)o, q) != (uint32_t)(o / g)) {
          printf("%lld / %d is not %u\\n", (long long)o, g, over_gather((uint32_t)o, q));
          return 1;
        }
      }
  }
  return 0;
}
"""


def test_quotient(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "quotient.cc", tmp_path / "quotient"
    src.write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-O2", "-I" + os.path.join(ROOT, "mxfp8_decode_gemm_amd", "csrc"), str(src), "-o",
                        str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


def test_the_program_finds_a_quotient_by_32_bits(tmp_path):
    """The product with floor(2^32 / gather) + 1 alone is right for the pairs of a call (below 2^24), not for entries of a
    longer order: 134217759 / 32 came out as 4194305."""
    assert [(134217759 * ((1 << 32) // 32 + 1)) >> 32, 134217759 // 32] == [4194305, 4194304]
