"""Host rules of the tuning calls at the ends of their ranges, on the CPU."""
import os
import re
import shutil

import pytest

from tests.test_sanitizers import HIP_INCLUDE, ROOT, SAN, _env, _run

CSRC = os.path.join(ROOT, "dequant_matmul_int3_amd", "csrc")
needs_gxx = pytest.mark.skipif(
    shutil.which("g++") is None or not os.path.isdir(os.path.join(HIP_INCLUDE, "hip")),
    reason="g++ or the HIP headers not available")


def drive(tmp_path, *sources):
    exe = str(tmp_path / "driver")
    rc, out = _run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", *SAN, "-I", HIP_INCLUDE,
                    "-I", os.path.join(ROOT, "include"), "-I", CSRC, *sources, "-o", exe])
    assert rc == 0, out
    rc, out = _run([exe], env=_env())
    assert rc == 0 and re.search(r"\b0 failures", out) and "runtime error" not in out, out


@needs_gxx
def test_launches_of_documented_sizes(tmp_path):
    drive(tmp_path, os.path.join(ROOT, "tests", "sanitize", "launch_driver.cpp"))


@needs_gxx
def test_accepted_and_refused_arguments(tmp_path):
    drive(tmp_path, os.path.join(CSRC, "api_tune.cpp"),
          os.path.join(ROOT, "tests", "sanitize", "tune_stubs.cpp"),
          os.path.join(ROOT, "tests", "sanitize", "range_driver.cpp"))
