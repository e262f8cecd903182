"""csrc/rows_choice.h: which kernel sizes run on. The shapes by which the GPU tests mean to reach each kernel reach it, and
a workspace has room for what its choice writes. Compiled for the host."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
#include "rows_choice.h"
#include <cstdio>
using namespace mxg;
int main() {
  // Grids: whole runs, at least the tiles, threads of a row in 32 bits.
  for (int64_t t : {1, 7, 8, 255, 256, 257, 4096, 1 << 20, (1 << 20) + 1, 8978432, 1082130432}) {
    const TileGrid g = tile_grid(t);
    if ((int64_t)g.x * g.y < t || (uint64_t)g.x * 512 > 0xFFFFFFFFu || g.y > 65535 || g.x % 8 ||
        (t >= 256 && g.x % 256) || (g.y > 1 && (int64_t)g.x * (g.y - 1) >= t))
      return 1;
  }
  int a[8];
  while (scanf("%d %d %d %d %d %d %d %d", a, a + 1, a + 2, a + 3, a + 4, a + 5, a + 6, a + 7) == 8) {
    const RowsChoice c = rows_choice(rows_problem(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7]));
    printf("%d %lld %lld %d %zu\\n", c.side, (long long)c.row_tiles, (long long)c.col_tiles, c.split, choice_workspace(c));
  }
}
"""

FP4, FP8, FAST = 4, 8, 9
FORMS = [(FP4, FP4), (FP4, FP8), (FP8, FP8), (FP4, FAST), (FP8, FAST)]


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("choice")
    (d / "choice.cc").write_text(PROGRAM)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-I" + os.path.join(ROOT, "mxfp8_decode_gemm_amd", "csrc"),
                        str(d / "choice.cc"), "-o", str(d / "choice")], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr

    def ask(shapes):
        """(kernel, row tiles, column tiles, parts of K, workspace) of (form of W, of x, experts, n, k, gated, rows,
        grouped)."""
        text = "\n".join(" ".join(str(int(v)) for v in s) for s in shapes)
        r = subprocess.run([str(d / "choice")], input=text, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0
        found = []
        for s, line in zip(shapes, r.stdout.splitlines(), strict=True):
            side, rt, ct, split, nbytes = map(int, line.split())
            if side == 0:
                kernel = "stream"
            elif s[1] == FP8:
                kernel = "bf16"
            elif side == 256:
                kernel = "large"
            else:
                kernel = "alone" if rt * ct * split <= 256 else "by two"
            found.append((kernel, rt, ct, split, nbytes))
        return found

    return ask


def dense(form, rows, n, k, gated=False):
    return (*form, 1, n, k, gated, rows, False)


@pytest.mark.parametrize("form", FORMS)
def test_one_weight(choose, form):
    bf16 = form[1] == FP8
    small = choose([dense(form, 289, 1032, k) for k in (128, 256, 384, 512, 640, 768, 1024, 1152)])
    assert {c[0] for c in small} == {"bf16" if bf16 else "alone"} and {c[3] for c in small} == {1}
    assert {c[1] for c in small} == {5 if bf16 else 3}  # (64 rows each, or 128)
    two = choose([dense(form, 1100, 4104, k) for k in (128, 256, 384, 640, 896, 1280)])
    assert {c[0] for c in two} == {"bf16" if bf16 else "by two"} and {c[1] for c in two} == {9}
    large = choose([dense(form, 2060, 4104, k) for k in (128, 384, 512, 1152)] + [dense(form, 2060, 4160, 640, True)])
    assert {c[0] for c in large} == {"bf16" if bf16 else "large"}
    for gated in (False, True):
        divided = choose([dense(form, r, (n + 63) // 64 * 64 if gated else n, k, gated)
                          for r, n, k in ((130, 520, 8320), (40, 264, 16384), (200, 1088, 16512))])
        assert {c[0] for c in divided} == {"bf16" if bf16 else "alone"} and min(c[3] for c in divided) > 1
    few = choose([dense(form, r, n, k) for r, n, k in ((1, 40, 128), (7, 264, 2048), (24, 264, 640))])
    assert {c[0] for c in few} == {"stream"}


@pytest.mark.parametrize("form", FORMS)
def test_experts(choose, form):
    bf16 = form[1] == FP8
    one = lambda experts, n, k, gated, rows: choose([(*form, experts, n, k, gated, rows, True)])[0]  # noqa: E731
    rows = sum(256 + 32 * i + (5 if i % 2 else 32) for i in range(8))
    for gated in (False, True):
        assert one(8, 4416, 640, gated, rows + 3)[0] == ("bf16" if bf16 else "large")
        assert one(8, 192, 2304, gated, 454)[0] == ("bf16" if bf16 else "alone")
    assert one(5, 136, 2304, False, 16)[0] == "stream"
    assert one(4, 136, 640, False, 472)[0] == ("bf16" if bf16 else "alone")


@pytest.mark.parametrize("form", FORMS)
def test_workspaces(choose, form):
    """Sums of every part of every tile, at most 16 MiB: parts only of launches of at most 256 workgroups."""
    shapes = [dense(form, r, n, k, g) for r in (1, 8, 33, 64, 65, 128, 130, 257, 1000, 4096) for n in (64, 1088, 4096, 8192)
              for k in (128, 2048, 8320, 65536) for g in (False, True)]
    for s, (kernel, rt, ct, split, nbytes) in zip(shapes, choose(shapes)):
        rows, n, k = s[6], s[3], s[4]
        if kernel == "stream":
            assert (rt, ct, split, nbytes) == (0, 0, 0, 0)
            continue
        assert rt <= (rows + 31) // 32 and (kernel == "large" or (128 * rt >= rows and ct == (n + 127) // 128))
        assert split == 1 or (kernel in ("alone", "bf16") and rt * ct * split <= 256 and split <= (k + 255) // 256)
        assert nbytes == (rt * ct * split * 65536 if split > 1 else 0) <= 16 << 20
