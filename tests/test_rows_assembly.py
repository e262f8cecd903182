"""What the compiler makes of the kernels that copy to LDS by inline assembly, built for gfx950 here: nothing but those
copies uses m0, and the kernels that keep a CU's or half a CU's registers busy keep them out of memory."""

import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp8_decode_gemm_amd", "csrc")


@pytest.fixture(scope="module")
def assembly(tmp_path_factory):
    from mxfp8_decode_gemm_amd import build as b

    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("no hipcc")
    d = tmp_path_factory.mktemp("assembly")
    names = ("rows_tile", "rows_bf16", "rows_stream")
    jobs = [subprocess.Popen([hipcc, *b.HIPCC_FLAGS, "-S", "--cuda-device-only", os.path.join(CSRC, n + ".hip"), "-o",
                              str(d / (n + ".s"))], stdout=subprocess.DEVNULL, stderr=subprocess.DEVNULL) for n in names]
    assert [j.wait(timeout=600) for j in jobs] == [0] * len(names)
    return {n: (d / (n + ".s")).read_text() for n in names}


def _scratch(text):
    """Bytes of scratch of each kernel."""
    return {name: int(size) for name, size in
            re.findall(r"\.amdhsa_kernel (\S+)\n(?:.*\n)*?\s*\.amdhsa_private_segment_fixed_size (\d+)", text)}


def test_m0_belongs_to_the_copies(assembly):
    for name in ("rows_tile", "rows_bf16"):
        code = [ln.split(";")[0] for ln in assembly[name].splitlines()]
        at = [i for i, ln in enumerate(code) if re.search(r"\bm0\b", ln)]
        assert at and all(re.match(r"\s*s_mov_b32 m0, s\d+\s*$", code[i]) for i in at)
        assert all("s_nop" in code[i + 1] and "global_load_lds" in code[i + 2] for i in at)


def test_registers_stay_registers(assembly):
    found = {k: v for text in assembly.values() for k, v in _scratch(text).items()}
    assert len(found) == 3 * 3 + 2 + 2 + 10  # tiles of three forms, joins, BF16 tiles, streams
    # The tiles of 256 rows of x hold every register of a SIMD and reload four words of a lane's addresses.
    large = [k for k in found if "Li2ELi8ELi4ELi1E" in k]
    assert len(large) == 3 and max(found[k] for k in large) <= 20
    assert all(v == 0 for k, v in found.items() if k not in large)
