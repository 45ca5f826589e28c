"""Ends of the serving calls' ranges on the CPU (nothing may reach the GPU here)."""
import math

import dequant_matmul_int3_amd as qt
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
