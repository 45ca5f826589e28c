"""The C ABI of the tuning calls on the CPU: sizes, refusals through the built
library (nothing may reach the GPU here), and the validation layer under the
sanitizers with its launchers replaced by stubs."""
import os
import shutil

import pytest

import dequant_matmul_int3_amd as qt
from tests.test_sanitizers import HIP_INCLUDE, ROOT, SAN, _env, _run

A, B, C_, D = 0x7F0000000000, 0x7F1000000000, 0x7F2000000000, 0x7F3000000000
E, F_, G_, H = 0x7F4000000000, 0x7F5000000000, 0x7F6000000000, 0x7F7000000000
NULL, SHAPE, ALIGN, DTYPE, ARG, ALIAS, WORKSPACE = 1, 2, 3, 4, 5, 6, 8


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(os.path.join(HIP_INCLUDE, "hip")),
                    reason="g++ or the HIP headers not available")
def test_tuning_validation_under_sanitizers(tmp_path):
    exe = str(tmp_path / "tune_driver")
    csrc = os.path.join(ROOT, "dequant_matmul_int3_amd", "csrc")
    rc, out = _run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", *SAN, "-I", HIP_INCLUDE,
                    "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(csrc, "api_tune.cpp"),
                    os.path.join(ROOT, "tests", "sanitize", "tune_stubs.cpp"),
                    os.path.join(ROOT, "tests", "sanitize", "tune_driver.cpp"), "-o", exe])
    assert rc == 0, out
    rc, out = _run([exe], env=_env())
    assert rc == 0 and "0 failures" in out and "runtime error" not in out, out


def test_workspace_sizes():
    bf, f32 = qt.QT_BF16, qt.QT_F32
    # a few rows go through LDS, bf16 rows of whole groups are read in place;
    # other inputs are copied
    assert qt.qt_ffn_gated_workspace_bytes(1, 7200, 2048, bf) == 0
    assert qt.qt_ffn_gated_workspace_bytes(12, 7168, 2048, bf) == 0
    assert qt.qt_ffn_gated_workspace_bytes(12, 7200, 2048, bf) >= 12 * 7232 * 2
    assert qt.qt_ffn_gated_workspace_bytes(8, 64, 64, f32) >= 3 * 8 * 64 * 2
    assert qt.qt_ffn_gated_workspace_bytes(65, 64, 64, bf) >= 80 * 64 * 2
    both = qt.qt_ffn_gated_bwd_workspace_bytes(300, 200, 150, bf)
    dx = qt.qt_ffn_gated_bwd_workspace_bytes(300, 200, 150, bf, want_dscales=False)
    ds = qt.qt_ffn_gated_bwd_workspace_bytes(300, 200, 150, bf, want_dx=False)
    assert both == dx + ds and dx >= 300 * 2 * 192 * 2 and ds >= 300 * 256 * 2
    assert qt.qt_matmul_bwd_workspace_bytes(300, 200, 150, bf) > 0
    assert qt.qt_distill_topk_workspace_bytes(4096, 32000, bf) == 0
    assert qt.qt_distill_topk_workspace_bytes(4, 32000, bf) > 0
    assert qt.qt_ffn_gated_workspace_bytes(0, 64, 64, bf) == 0


def test_ffn_refusals():
    f = qt.lib().qt_ffn_gated

    def call(gp=A, gb=3, ub=4, F=64, D=64, act=0, X=E, xt=1, T=4, Hh=F_, pre=G_, ws=None, wsb=0):
        return f(gp, B, gb, C_, D_, ub, F, D, act, X, xt, T, Hh, pre, ws, wsb, None)

    D_ = D
    assert call(gp=None) == NULL and call(X=None) == NULL and call(Hh=None) == NULL
    assert call(xt=2) == DTYPE
    assert call(T=0) == SHAPE and call(F=0) == SHAPE and call(D=(1 << 20) + 1) == SHAPE
    assert call(gb=2) == ARG and call(ub=8) == ARG and call(act=2) == ARG
    assert call(T=20, D=65) == WORKSPACE and call(T=20, D=65, ws=H, wsb=16) == WORKSPACE
    assert call(gp=A + 4) == ALIGN and call(X=E + 2) == ALIGN and call(pre=G_ + 2) == ALIGN
    assert call(T=20, D=65, ws=H + 8, wsb=1 << 20) == ALIGN
    assert call(Hh=E) == ALIAS and call(pre=F_) == ALIAS and call(Hh=A + 64) == ALIAS


def test_backward_refusals():
    f, m = qt.lib().qt_ffn_gated_bwd, qt.lib().qt_matmul_bwd

    def ffn(pre=E, dH=F_, X=G_, dX=H, dg=None, du=None, acc=0, ws=None, wsb=0, T=4):
        return f(A, B, 3, C_, D, 4, 64, 64, 0, pre, dH, X, 1, T, dX, dg, du, acc, ws, wsb, None)

    ws, K = 0x7E0000000000, 1 << 20
    assert ffn(pre=None) == NULL and ffn(dX=None) == NULL
    assert ffn(dg=ws - K, ws=ws, wsb=K) == NULL                     # one of the two
    assert ffn(X=None, dg=ws - K, du=ws - 2 * K, ws=ws, wsb=K) == NULL
    assert ffn() == WORKSPACE and ffn(ws=ws, wsb=K, acc=2) == ARG
    assert ffn(ws=ws, wsb=K, T=(1 << 22) + 1) == SHAPE
    assert ffn(ws=ws + 4, wsb=K) == ALIGN and ffn(dX=H + 1, ws=ws, wsb=K) == ALIGN
    assert ffn(dX=F_, ws=ws, wsb=K) == ALIAS and ffn(ws=E, wsb=K) == ALIAS

    def lin(packed=A, bits=3, yt=0, xt=1, X=D, dX=E, ds=None, ws=ws, wsb=K):
        return m(packed, B, bits, 64, 64, C_, yt, X, xt, 4, dX, ds, 0, ws, wsb, None)

    assert lin(packed=None) == NULL and lin(dX=None) == NULL and lin(X=None, ds=F_) == NULL
    assert lin(yt=2) == DTYPE and lin(xt=-1) == DTYPE and lin(bits=5) == ARG
    assert lin(wsb=8) == WORKSPACE and lin(dX=C_) == ALIAS and lin(dX=E, ds=E) == ALIAS


def test_distill_refusals():
    f, b = qt.lib().qt_distill_topk, qt.lib().qt_distill_topk_bwd

    def fwd(z=A, lt=1, T=4, V=64, ldl=64, idx=B, k=4, tau=1.0, loss=D, lse=E, gl=None, dz=None,
            ldd=64, ws=None, wsb=0):
        return f(z, lt, T, V, ldl, idx, C_, k, tau, loss, lse, gl, dz, ldd, ws, wsb, None)

    assert fwd(z=None) == NULL and fwd(idx=None) == NULL and fwd(loss=None) == NULL
    assert fwd(lt=3) == DTYPE
    assert fwd(T=0) == SHAPE and fwd(V=0) == SHAPE and fwd(ldl=63) == SHAPE
    assert fwd(V=1 << 31, ldl=1 << 31) == SHAPE and fwd(dz=F_, ldd=3) == SHAPE
    assert fwd(k=0) == ARG and fwd(k=1025) == ARG and fwd(tau=-1.0) == ARG
    assert fwd(tau=float("nan")) == ARG
    assert fwd(V=32000, ldl=32000) == WORKSPACE
    assert fwd(z=A + 1) == ALIGN and fwd(gl=F_ + 1) == ALIGN and fwd(lse=E + 2) == ALIGN
    assert fwd(lse=D) == ALIAS and fwd(dz=A + 64) == ALIAS and fwd(dz=A, ldd=65) == ALIAS
    assert b(A, 1, 4, 64, 64, B, C_, 4, 1.0, None, None, D, 64, None) == NULL
    assert b(A, 1, 4, 64, 64, B, C_, 4, 1.0, E, None, E, 64, None) == ALIAS


def test_host_tensors_are_refused():
    import torch
    w = (torch.zeros(4 * 24, dtype=torch.uint8), torch.zeros(4, 1), 3)
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError, match="device tensors"):
        qt.qt_ffn_gated(w, w, x)
    with pytest.raises(ValueError, match="device tensors"):
        qt.qt_matmul_bwd(w, torch.zeros(2, 4), x)
    with pytest.raises(ValueError, match="device tensors"):
        qt.qt_distill_topk(x, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1))
