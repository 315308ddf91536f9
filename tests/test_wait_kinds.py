"""The two kinds of bounded waits cannot be taken for one another: a wait that must be waited
for in every build is told by the type of its limit, so no number makes it a pipeline wait,
and the two limits may be equal."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_fp8_gated_b200", "csrc")
NVCC = os.environ.get("NVCC", "nvcc")


def _compiles(tmp_path, call):
    src = tmp_path / "waits.cu"
    src.write_text('#include "gad_tc.cuh"\n'
                   "static_assert(gad::kGiveUpAtFirstMiss);\n"
                   "__global__ void waits(volatile int* flag, int* out) {\n"
                   f"    *out = gad::wait_bounded(0u, 0u, flag{call});\n}}\n")
    return subprocess.run([NVCC, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-I", CSRC,
                           "-DGAD_TEST_GIVE_UP_AT_FIRST_MISS=1", "-c", "-o", str(tmp_path / "waits.o"), str(src)],
                          capture_output=True, text=True).returncode == 0


@pytest.mark.skipif(shutil.which(NVCC) is None, reason="needs nvcc")
@pytest.mark.parametrize("call,ok", [
    ("", True), (", false, gad::TEARDOWN_LIMIT_NS", True), (", false, gad::LastWait{gad::WAIT_LIMIT_NS}", True),
    (", false, gad::WAIT_LIMIT_NS", False), (", false, 1ull", False), (", false", False),
])
def test_kind_of_a_wait_is_its_type(tmp_path, call, ok):
    assert _compiles(tmp_path, call) == ok
