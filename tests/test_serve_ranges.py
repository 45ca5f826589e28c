"""Ends of the serving calls' ranges on the CPU (nothing may reach the GPU here)."""
import math
import os
import shutil

import pytest

import dequant_matmul_int3_amd as qt
from tests.test_sanitizers import HIP_INCLUDE, ROOT, SAN, _env, _run
from tests.test_serve_boundary import ALIGN, ARG, A, B, C_, D, E, F_, G_, H, I_


def test_scales_past_the_powers_of_two():
    """A scale that is a number, but not times log2 e, is refused; 2^127 is not (an
    address that no check takes stops that call behind this one)."""
    f = qt.lib().qt_attn_decode

    def call(scale, out=H):
        return f(A, 512, 1, 2, 8, D, E, 8, F_, G_, 4, 4, 16, 2, 64, B, 2, C_, 0, scale, out, I_,
                 None, 0, None)

    for s in (2.0 ** 127 * (1 + 2.0 ** -23), 3e38, -3e38, math.inf, math.nan):
        assert call(s) == ARG, s
    for s in (2.0 ** 127, -(2.0 ** 127), 0.0, 2.0 ** -149):
        assert call(s, out=H + 1) == ALIGN, s


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(os.path.join(HIP_INCLUDE, "hip")),
                    reason="g++ or the HIP headers not available")
def test_chunks_reach_every_position(tmp_path):
    """With windows too, whose spans start inside a tile."""
    exe = str(tmp_path / "plan_driver")
    rc, out = _run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", *SAN, "-I", HIP_INCLUDE,
                    "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "dequant_matmul_int3_amd", "csrc"),
                    os.path.join(ROOT, "tests", "sanitize", "plan_driver.cpp"), "-o", exe])
    assert rc == 0, out
    rc, out = _run([exe], env=_env())
    assert rc == 0 and " 0 failures" in out and "runtime error" not in out, out
