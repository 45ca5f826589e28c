"""The C ABI of the cache, attention and few-token expert calls on the CPU: sizes and refusals
through the built library (nothing may reach the GPU here), and the validation layer under the
sanitizers with its launchers replaced by stubs."""
import os
import shutil

import pytest
import torch

import dequant_matmul_int3_amd as qt
from tests.test_sanitizers import HIP_INCLUDE, ROOT, SAN, _env, _run

A, B, C_, D = 0x7F0000000000, 0x7F1000000000, 0x7F2000000000, 0x7F3000000000
E, F_, G_, H = 0x7F4000000000, 0x7F5000000000, 0x7F6000000000, 0x7F7000000000
I_, J = 0x7E0000000000, 0x7E1000000000
NULL, SHAPE, ALIGN, DTYPE, ARG, ALIAS, WORKSPACE = 1, 2, 3, 4, 5, 6, 8


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(os.path.join(HIP_INCLUDE, "hip")),
                    reason="g++ or the HIP headers not available")
def test_serving_validation_under_sanitizers(tmp_path):
    exe = str(tmp_path / "serve_driver")
    csrc = os.path.join(ROOT, "dequant_matmul_int3_amd", "csrc")
    rc, out = _run(["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", *SAN, "-I", HIP_INCLUDE,
                    "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(csrc, "api_serve.cpp"),
                    os.path.join(ROOT, "tests", "sanitize", "serve_stubs.cpp"),
                    os.path.join(ROOT, "tests", "sanitize", "serve_driver.cpp"), "-o", exe])
    assert rc == 0, out
    rc, out = _run([exe], env=_env())
    assert rc == 0 and "0 failures" in out and "runtime error" not in out, out


def test_cache_sizes():
    assert qt.qt_kv_bytes(3, 16, 2, 128, 8) == 3 * 16 * 2 * 128
    assert qt.qt_kv_bytes(3, 16, 2, 128, 4) == 3 * 16 * 2 * 64
    assert qt.qt_kv_bytes(1, 48, 1, 65, 4) == 48 * 64
    for bad in ((0, 16, 1, 64, 8), (1, 8, 1, 64, 8), (1, 24, 1, 64, 8), (1, 16, 0, 64, 8),
                (1, 16, 1, 0, 8), (1, 16, 1, 257, 8), (1, 16, 1, 64, 3), (1 << 27, 16, 1, 64, 8),
                (1, 65552, 1, 64, 8), (1, 16, 1025, 64, 8)):
        assert qt.qt_kv_bytes(*bad) == 0, bad


def test_workspace_sizes():
    w = qt.qt_attn_decode_workspace_bytes
    assert w(1, 32, 8, 128, 16, 16) == 0                    # one chunk
    assert w(1, 32, 8, 128, 64, 16) == 0                    # short: one block of eight waves
    assert w(1, 32, 8, 129, 64, 16) > 0                     # but for wide heads
    assert w(1, 32, 8, 128, 64, 64) > 0                     # a long context is cut
    assert w(256, 32, 8, 128, 32, 64) == 0                  # a batch fills the card uncut
    assert w(1, 32, 8, 128, 4096, 64, window=100) == 0      # a window bounds the span
    assert w(1, 8, 8, 64, 1 << 20, 16) == 8 * 8192 * 68 * 4  # chunks of 2048 at most
    for bad in ((0, 8, 8, 64, 1, 16), (1, 8, 3, 64, 1, 16), (1, 8, 8, 64, 0, 16),
                (1, 8, 8, 64, 1, 17), (65536, 8, 8, 64, 1, 16), (1, 257, 1, 64, 1, 16),
                (1, 8, 8, 64, 1 << 27, 16), (1, 8, 8, 64, 1, 16, -1)):
        assert w(*bad) == 0, bad


def test_write_refusals():
    f = qt.lib().qt_kv_write

    def call(K=A, ldk=128, V=B, ldv=128, xt=1, T=4, slots=C_, kc=D, ks=E, kb=8, vc=F_, vs=G_, vb=4,
             n=4, page=16, heads=2, dim=64):
        return f(K, ldk, V, ldv, xt, T, slots, kc, ks, kb, vc, vs, vb, n, page, heads, dim, None)

    for p in ("K", "V", "slots", "kc", "ks", "vc", "vs"):
        assert call(**{p: None}) == NULL
    assert call(xt=2) == DTYPE
    assert call(T=0) == SHAPE and call(T=(1 << 22) + 1) == SHAPE and call(ldk=127) == SHAPE
    assert call(ldv=1 << 40) == SHAPE and call(page=8) == SHAPE and call(page=20) == SHAPE
    assert call(heads=0) == SHAPE and call(dim=257, ldk=514, ldv=514) == SHAPE and call(n=0) == SHAPE
    assert call(n=1 << 27) == SHAPE and call(n=-3) == SHAPE and call(n=1 << 62) == SHAPE
    assert call(kb=3) == ARG and call(vb=16) == ARG
    assert call(K=A + 1) == ALIGN and call(kc=D + 8) == ALIGN and call(vs=G_ + 4) == ALIGN
    assert call(slots=C_ + 2) == ALIGN
    assert call(K=D + 64) == ALIAS and call(vc=D) == ALIAS and call(slots=E) == ALIAS


def test_read_refusals():
    f = qt.lib().qt_kv_read

    def call(slots=C_, R=4, kc=D, ks=E, kb=8, vc=F_, vs=G_, vb=4, n=4, page=16, heads=2, dim=64,
             K=A, V=B, xt=0):
        return f(slots, R, kc, ks, kb, vc, vs, vb, n, page, heads, dim, K, V, xt, None)

    assert call(slots=None) == NULL and call(K=None, V=None) == NULL and call(kc=None) == NULL
    assert call(xt=-1) == DTYPE and call(R=0) == SHAPE and call(dim=0) == SHAPE
    assert call(kb=5) == ARG and call(K=A + 2) == ALIGN and call(ks=E + 4) == ALIGN
    assert call(K=D) == ALIAS and call(V=A + 16) == ALIAS and call(V=C_) == ALIAS


def test_attention_refusals():
    f = qt.lib().qt_attn_decode

    def call(Q=A, ldq=512, xt=1, Bn=2, hq=8, kc=D, ks=E, kb=8, vc=F_, vs=G_, vb=4, n=4, page=16,
             heads=2, dim=64, table=B, pages=2, lens=C_, window=0, scale=0.125, out=H, lse=I_,
             ws=None, wsb=0):
        return f(Q, ldq, xt, Bn, hq, kc, ks, kb, vc, vs, vb, n, page, heads, dim, table, pages, lens,
                 window, scale, out, lse, ws, wsb, None)

    for p in ("Q", "kc", "ks", "vc", "vs", "table", "lens", "out"):
        assert call(**{p: None}) == NULL
    assert call(xt=7) == DTYPE
    assert call(Bn=0) == SHAPE and call(Bn=65536) == SHAPE and call(hq=7) == SHAPE
    assert call(hq=2 * 257, ldq=1 << 20) == SHAPE and call(ldq=511) == SHAPE
    assert call(pages=0) == SHAPE and call(pages=1 << 27) == SHAPE and call(window=-1) == SHAPE
    assert call(page=17) == SHAPE and call(dim=300) == SHAPE
    assert call(kb=2) == ARG and call(vb=0) == ARG
    assert call(scale=float("nan")) == ARG and call(scale=float("inf")) == ARG
    assert call(pages=128) == WORKSPACE and call(pages=128, ws=J, wsb=64) == WORKSPACE
    assert call(pages=128, ws=J + 4, wsb=1 << 24) == ALIGN
    assert call(out=H + 1) == ALIGN and call(lse=I_ + 2) == ALIGN and call(lens=C_ + 1) == ALIGN
    assert call(out=A) == ALIAS and call(lse=H) == ALIAS and call(out=D + 16) == ALIAS
    assert call(lse=B) == ALIAS and call(pages=128, ws=A, wsb=1 << 24) == ALIAS


def test_binding_refusals():
    """Refused before any device is touched."""
    k, v = qt.qt_kv_cache(2, 16, 2, 80, 4, 8, device="cpu")
    assert k[0].shape == (2, 2, 16, 64) and v[0].shape == (2, 2, 16, 128)
    assert k[1].shape == (2, 2, 16, 2) and k[2] == 4 and v[2] == 8
    with pytest.raises(ValueError, match="no such cache"):
        qt.qt_kv_cache(2, 10, 2, 80, device="cpu")
    x, slots = torch.zeros(3, 2, 80), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensors"):
        qt.qt_kv_write(x, x, slots, k, v)
    with pytest.raises(ValueError, match="device tensors"):
        qt.qt_kv_read(slots, k, v, 80)
    with pytest.raises(ValueError, match="contiguous tokens"):
        qt.qt_kv_write(torch.zeros(3, 2, 160)[..., ::2], x, slots, k, v)
    with pytest.raises(ValueError, match="contiguous tokens"):
        qt.qt_kv_write(torch.zeros(2, 3, 80).transpose(0, 1), x, slots, k, v)
    with pytest.raises(ValueError, match="same shape"):
        qt.qt_kv_write(x, x.bfloat16(), slots, k, v)
    with pytest.raises(ValueError, match="same heads"):
        qt.qt_kv_write(x[:, :1], x[:, :1], slots, k, v)
    with pytest.raises(ValueError, match="scales must be"):
        qt.qt_kv_write(torch.zeros(3, 2, 130), torch.zeros(3, 2, 130), slots, k, v)
    with pytest.raises(ValueError, match="slots must be"):
        qt.qt_kv_write(x, x, slots.long(), k, v)
    with pytest.raises(ValueError, match="codes do not match"):
        qt.qt_kv_read(slots, (k[0], k[1], 8), v, 80)
    q, table, lens = torch.zeros(3, 4, 80), torch.zeros(3, 2, dtype=torch.int32), slots
    with pytest.raises(ValueError, match="page_table must be"):
        qt.qt_attn_decode(q, k, v, table[:2], lens)
    with pytest.raises(ValueError, match="lens must be"):
        qt.qt_attn_decode(q, k, v, table, lens.long())
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        qt.qt_attn_decode(q.half(), k, v, table, lens)
    with pytest.raises(ValueError, match="device tensors"):
        qt.qt_attn_decode(q, k, v, table, lens)


def test_expert_layer_refusals():
    f, w = qt.lib().qt_moe_decode, qt.qt_moe_decode_workspace_bytes
    assert w(1, 8, 128, 7168, 2048, qt.QT_BF16) >= 2 * 8 * 2048 * 2
    assert w(16, 8, 128, 7168, 2049, qt.QT_F32) >= 3 * 128 * 2112 * 2
    for bad in ((0, 1, 1, 64, 64, 0), (17, 1, 1, 64, 64, 0), (1, 2, 1, 64, 64, 0),
                (1, 33, 64, 64, 64, 0), (1, 1, 513, 64, 64, 0), (1, 1, 1, 0, 64, 0),
                (1, 1, 1, 64, (1 << 20) + 1, 0), (1, 1, 1, 64, 64, 2)):
        assert w(*bad) == 0, bad
    K = 1 << 20

    def call(X=A, xt=1, T=2, Dm=128, F=64, lg=B, En=4, k=2, act=0, gp=C_, gs=D, gb=3, up=E, us=F_,
             ub=4, dp=G_, ds=H, db=3, out=I_, ws=J, wsb=K):
        return f(X, xt, T, Dm, F, lg, En, k, act, gp, gs, gb, up, us, ub, dp, ds, db, out, ws, wsb,
                 None)

    for p in ("X", "lg", "gp", "gs", "up", "us", "dp", "ds", "out"):
        assert call(**{p: None}) == NULL
    assert call(xt=3) == DTYPE
    assert call(T=17) == SHAPE and call(k=5) == SHAPE and call(k=0) == SHAPE
    assert call(En=513) == SHAPE and call(F=0) == SHAPE and call(Dm=-1) == SHAPE
    assert call(gb=5) == ARG and call(db=8) == ARG and call(act=2) == ARG
    assert call(ws=None) == WORKSPACE and call(wsb=64) == WORKSPACE
    assert call(gp=C_ + 8) == ALIGN and call(X=A + 1) == ALIGN and call(ws=J + 8) == ALIGN
    assert call(out=A) == ALIAS and call(out=C_ + 64) == ALIAS and call(ws=I_) == ALIAS


def test_expert_layer_binding_refusals():
    x, lg = torch.zeros(2, 100), torch.zeros(2, 4)
    w = (torch.zeros(4, 70 * 2 * 24, dtype=torch.uint8), torch.zeros(4, 70, 2), 3)
    dn = (torch.zeros(4, 100 * 2 * 32, dtype=torch.uint8), torch.zeros(4, 100, 2), 4)
    with pytest.raises(ValueError, match="device tensors"):
        qt.qt_moe_decode(x, lg, 2, w, w, dn)
    with pytest.raises(ValueError, match="act must be"):
        qt.qt_moe_decode(x, lg, 2, w, w, dn, act="relu")
    with pytest.raises(ValueError, match="down: scales"):
        qt.qt_moe_decode(x, lg, 2, w, w, w)
    with pytest.raises(ValueError, match="gate: packed"):
        qt.qt_moe_decode(x, lg, 2, (w[0], w[1], 4), w, dn)
    with pytest.raises(ValueError, match="logits"):
        qt.qt_moe_decode(x, lg.double(), 2, w, w, dn)
