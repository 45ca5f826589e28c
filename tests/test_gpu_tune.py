"""The gated feed-forward block, the backward passes through packed weights
and the distillation loss against plain 64-bit forms, at the sizes where each
kernel form begins and ends, ragged groups and rows, every pair of bits and
both types; refusals, graph replays, streams, and the operators as one chain."""
import math

import pytest
import torch

import dequant_matmul_int3_amd as qt
from tests.gpu_util import DEV, say
from tests.tune_util import (SUM, act64, dense, distill_ref, dx_bound, ffn_ref, grads_ref,
                             half_step, quantized, scale_grad, worst)

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def rnd(shape, seed, dtype=F32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def guarded(shape, dtype, pad=96):
    """A tensor of this shape inside a larger buffer, and a check that nothing
    outside of it was written."""
    n = math.prod(shape)
    buf = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device=DEV)
    view = buf[pad:pad + n].view(shape)
    return view, lambda: bool((buf[:pad] == 7.0).all()) and bool((buf[pad + n:] == 7.0).all())


# ------------------------------------------------------------------- forward
FFN = [
    # T, D, F, bits, act, dtype
    (1, 64, 16, (3, 3), "silu", F32),
    (1, 1, 1, (4, 3), "gelu", BF),
    (1, 7168, 96, (3, 3), "silu", BF),
    (1, 7200, 33, (3, 4), "silu", F32),
    (2, 65, 17, (4, 4), "gelu", F32),
    (5, 320, 47, (3, 4), "silu", BF),
    (16, 256, 64, (4, 3), "gelu", BF),
    (17, 192, 31, (3, 3), "silu", BF),
    (21, 448, 50, (4, 4), "silu", F32),    # 63 piece rows: the small form's last
    (22, 448, 50, (3, 4), "silu", F32),    # the tile
    (48, 640, 16, (3, 3), "silu", BF),
    (64, 100, 70, (4, 4), "silu", BF),
    (65, 100, 70, (3, 4), "gelu", BF),     # the tile
    (65, 2048, 64, (4, 3), "silu", BF),    # one block: the groups are split
    (128, 64, 65, (4, 4), "silu", BF),
    (129, 1088, 128, (3, 3), "silu", BF),
    (256, 192, 130, (4, 3), "gelu", F32),
    (257, 191, 200, (3, 3), "gelu", BF),
    (513, 577, 321, (3, 4), "silu", BF),
    (300, 2000, 67, (4, 4), "silu", F32),
    (1025, 256, 63, (4, 4), "silu", BF),
    (33, 2048, 40, (3, 3), "silu", BF),    # eight waves, 48 and 64 KB of sums
    (64, 2048, 40, (4, 3), "silu", BF),
    (21, 2048, 24, (3, 4), "gelu", F32),
    (4, 1536, 40, (3, 4), "silu", BF),     # 16 piece rows or less go through LDS
    (3, 1000, 40, (4, 3), "gelu", BF),
    (5, 1504, 24, (4, 4), "silu", F32),    # 15 of them
    (6, 1504, 24, (3, 3), "silu", F32),    # 18: planes
    (16, 1600, 24, (3, 4), "silu", BF),    # 16 rows, too long for LDS: in place
]


@pytest.mark.parametrize("T,D,F,bits,act,dtype", FFN)
def test_ffn_gated(T, D, F, bits, act, dtype):
    say(f"ffn T={T} D={D} F={F} bits={bits} {act} {dtype}")
    gate, vg = quantized(F, D, bits[0], 1)
    up, vu = quantized(F, D, bits[1], 2)
    x = rnd((T, D), T + D, dtype)
    H, fine_h = guarded((T, F), dtype)
    pre, fine_p = guarded((2, T, F), F32)
    qt.qt_ffn_gated(gate, up, x, act=act, H=H, pre=pre)
    h, g, u, bh, bg, bu = ffn_ref(x, dense(gate, vg, D), dense(up, vu, D), act, dtype)
    errs = worst(pre[0], g, bg), worst(pre[1], u, bu), worst(H, h, bh)
    say(f"  error / bound: g {errs[0]:.3f} u {errs[1]:.3f} h {errs[2]:.3f}")
    assert max(errs) <= 1.0
    assert fine_h() and fine_p(), "wrote outside its outputs"
    H2 = qt.qt_ffn_gated(gate, up, x, act=act)
    assert torch.equal(H, H2), "not deterministic, or differs without pre"


def test_ffn_gated_extreme_activations():
    # pre-activations of +-1e4: the sigmoid is exactly 0 or 1 there
    D, F, T = 64, 32, 3
    gate, vg = quantized(F, D, 3, 1)
    up, vu = quantized(F, D, 3, 2)
    for act in ("silu", "gelu"):
        x = rnd((T, D), 3) * 1e5
        H, pre = qt.qt_ffn_gated(gate, up, x, act=act, want_pre=True)
        h = ffn_ref(x, dense(gate, vg, D), dense(up, vu, D), act, F32)[0]
        assert pre.abs().max() > 1e4
        assert worst(H, h, 1e-4 * h.abs() + 1e-30 + 1e-5 * h.abs().max()) <= 1.0
        dX, dsg, dsu = qt.qt_ffn_gated_bwd(gate, up, pre, torch.ones_like(H), x, act=act)
        for t in (dX, dsg, dsu):
            assert torch.isfinite(t).all()


# ------------------------------------------------------------------ backward
BWD = [
    (1, 64, 16, (3, 3), "silu", F32),
    (1, 1, 1, (4, 3), "gelu", BF),
    (2, 65, 17, (4, 4), "gelu", F32),
    (16, 256, 64, (4, 3), "gelu", BF),
    (40, 100, 70, (3, 4), "silu", BF),
    (65, 2048, 65, (4, 3), "silu", BF),
    (128, 129, 127, (3, 3), "silu", F32),
    (129, 1088, 128, (3, 3), "silu", BF),
    (257, 191, 200, (3, 3), "gelu", F32),
    (300, 320, 2000, (3, 4), "silu", BF),
    (513, 577, 321, (4, 3), "gelu", BF),
    (1025, 256, 192, (4, 4), "silu", BF),
    (2050, 130, 90, (3, 4), "silu", BF),
    (1030, 64, 65, (4, 3), "gelu", F32),
]


@pytest.mark.parametrize("T,D,F,bits,act,dtype", BWD)
def test_ffn_gated_bwd(T, D, F, bits, act, dtype):
    say(f"ffn bwd T={T} D={D} F={F} bits={bits} {act} {dtype}")
    gate, vg = quantized(F, D, bits[0], 1)
    up, vu = quantized(F, D, bits[1], 2)
    x, dh = rnd((T, D), T + D, dtype), rnd((T, F), T + F, dtype, 0.1)
    _, pre = qt.qt_ffn_gated(gate, up, x, act=act, want_pre=True)
    dX, fine_x = guarded((T, D), dtype)
    dsg, fine_g = guarded(gate[1].shape, F32)
    dsu, fine_u = guarded(up[1].shape, F32)
    qt.qt_ffn_gated_bwd(gate, up, pre, dh, x, act=act, dX=dX, dgate_scales=dsg, dup_scales=dsu)
    dg, du, eg, eu = grads_ref(pre[0].double(), pre[1].double(), dh.double(), act)
    wg, wu = dense(gate, vg, D), dense(up, vu, D)
    ref = dg @ wg + du @ wu
    b = dx_bound([(dg, eg, wg), (du, eu, wu)], dtype, dtype)
    b = b + half_step(dtype) * (ref.abs() + b) + 1e-30
    X = x.double()
    errs = [worst(dX, ref, b)]
    for got, dy, e, v in ((dsg, dg, eg, vg), (dsu, du, eu, vu)):
        bound = scale_grad(SUM * dy.abs() + e, X.abs(), v.abs()) + 1e-30
        errs.append(worst(got, scale_grad(dy, X, v), bound))
    say("  error / bound: dX %.3f dsg %.3f dsu %.3f" % tuple(errs))
    assert max(errs) <= 1.0
    assert fine_x() and fine_g() and fine_u(), "wrote outside its outputs"
    # alone, again and added: the same bits
    a = qt.qt_ffn_gated_bwd(gate, up, pre, dh, x, act=act, want_dscales=False)
    assert torch.equal(a[0], dX) and a[1] is None and a[2] is None
    a = qt.qt_ffn_gated_bwd(gate, up, pre, dh, x, act=act, want_dx=False)
    assert a[0] is None and torch.equal(a[1], dsg) and torch.equal(a[2], dsu)
    one_g, one_u = rnd(dsg.shape, 5), rnd(dsu.shape, 6)
    acc_g, acc_u = one_g.clone(), one_u.clone()
    qt.qt_ffn_gated_bwd(gate, up, pre, dh, x, act=act, want_dx=False, dgate_scales=acc_g,
                        dup_scales=acc_u, accumulate=True)
    assert torch.equal(acc_g, one_g + dsg) and torch.equal(acc_u, one_u + dsu)


LIN = [
    (1, 64, 16, 3, F32, F32),
    (1, 130, 1, 4, BF, BF),
    (7, 63, 65, 4, F32, BF),
    (33, 256, 300, 3, BF, F32),
    (129, 640, 129, 4, BF, F32),
    (130, 128, 1000, 3, F32, F32),
    (513, 200, 257, 4, BF, BF),
    (600, 1024, 64, 3, BF, F32),
    (1024, 64, 20001, 4, BF, F32),   # 251 row blocks of 80 for 209 of 96 (a step is shorter)
    (1024, 70, 6000, 3, BF, BF),
]


@pytest.mark.parametrize("B,I,O,bits,dtype,ytype", LIN)
def test_matmul_bwd(B, I, O, bits, dtype, ytype):
    say(f"matmul bwd B={B} I={I} O={O} bits={bits} {dtype} dY {ytype}")
    w, v = quantized(O, I, bits, 3)
    x, dy = rnd((B, I), B + I, dtype), rnd((B, O), B + O, ytype, 0.1)
    dX, fine_x = guarded((B, I), dtype)
    ds, fine_s = guarded(w[1].shape, F32)
    qt.qt_matmul_bwd(w, dy, x, dX=dX, dscales=ds)
    W, X, Y = dense(w, v, I), x.double(), dy.double()
    ref = Y @ W
    # dY that is bf16 already is not rounded again; the bound covers both
    b = dx_bound([(Y, 0 * Y, W)], dtype, dtype)
    b = b + half_step(dtype) * (ref.abs() + b) + 1e-30
    errs = (worst(dX, ref, b),
            worst(ds, scale_grad(Y, X, v), SUM * scale_grad(Y.abs(), X.abs(), v.abs()) + 1e-30))
    say("  error / bound: dX %.3f ds %.3f" % errs)
    assert max(errs) <= 1.0
    assert fine_x() and fine_s(), "wrote outside its outputs"
    acc = torch.ones_like(ds)
    qt.qt_matmul_bwd(w, dy, x, want_dx=False, dscales=acc, accumulate=True)
    assert torch.equal(acc, 1 + ds)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_wide_ranges_of_gradients_and_scales(dtype):
    # tokens' gradients from 1e-30 to 1e20 and scales from 1e-6 to 1e4: the
    # powers of two that bring both into f16's range are exact; rows without
    # any gradient stay zero.  bf16: a term under 2^-26 of its token's largest
    # gradient or of the largest scale keeps an absolute error of 2^-39 of it
    # (2^-38 for the two together)
    B, I, O = 40, 200, 96
    w, v = quantized(O, I, 3, 3)
    w[1].mul_((10.0 ** torch.linspace(-4, 5, w[1].shape[1], device=DEV))[None, :])
    x = rnd((B, I), 1, dtype)
    dy = rnd((B, O), 2, F32) * (10.0 ** torch.linspace(-30, 20, B, device=DEV))[:, None]
    dy[7] = 0
    dX, ds = qt.qt_matmul_bwd(w, dy, x)
    W, Y = dense(w, v, I), dy.double()
    ref = Y @ W
    b = dx_bound([(Y, 0 * Y, W)], dtype, dtype)
    if dtype == BF:
        b = b + 2.0 ** -38 * O * 4 * Y.abs().amax(1, keepdim=True) * w[1].abs().max().double()
    b = b + half_step(dtype) * (ref.abs() + b) + 2.0 ** -126
    assert worst(dX, ref, b) <= 1.0 and (dX[7] == 0).all()
    bound = SUM * scale_grad(Y.abs(), x.double().abs(), v.abs()) + 1e-30
    assert worst(ds, scale_grad(Y, x.double(), v), bound) <= 1.0
    # no scale at all
    z = (w[0], torch.zeros_like(w[1]), 3)
    dX, _ = qt.qt_matmul_bwd(z, dy, x)
    assert (dX == 0).all()


def test_masked_tokens_leave_no_trace():
    # tokens whose gradient is zero (padding) add nothing, wherever they stand
    T, D, F = 150, 192, 96
    gate, _ = quantized(F, D, 3, 1)
    up, _ = quantized(F, D, 4, 2)
    x, dh = rnd((T, D), 1, BF), rnd((T, F), 2, BF)
    dh[50:120] = 0
    _, pre = qt.qt_ffn_gated(gate, up, x, want_pre=True)
    dX, dsg, _ = qt.qt_ffn_gated_bwd(gate, up, pre, dh, x)
    assert (dX[50:120] == 0).all()
    x2 = x.clone()
    x2[50:120] = 3.0
    _, dsg2, _ = qt.qt_ffn_gated_bwd(gate, up, pre, dh, x2)
    assert torch.equal(dsg, dsg2)


def test_gradients_against_differences():
    # f32: (L(s + e d) - L(s - e d)) / 2e for L = sum H R against the gradients;
    # the central difference is off by e^2 times the third derivative (relative
    # ~e^2) and by the f32 noise 1e-6 sqrt(n) / e of L; e = 2^-7 keeps both
    # under 1e-3 of the gradient's own magnitude
    T, D, F = 6, 128, 48
    gate, _ = quantized(F, D, 3, 1)
    up, _ = quantized(F, D, 4, 2)
    x, r = rnd((T, D), 1), rnd((T, F), 2)
    e = 2.0 ** -7

    def loss(gs, us, xx):
        h = qt.qt_ffn_gated((gate[0], gs, 3), (up[0], us, 4), xx)
        return float((h.double() * r.double()).sum())

    _, pre = qt.qt_ffn_gated(gate, up, x, want_pre=True)
    dX, dsg, dsu = qt.qt_ffn_gated_bwd(gate, up, pre, r, x)
    for n, (grad, base) in enumerate(((dsg, gate[1]), (dsu, up[1]), (dX, x))):
        # the direction of the gradient itself, at the base's magnitude
        d = grad / grad.norm() * base.norm()
        args = [[gate[1], up[1], x], [gate[1], up[1], x]]
        args[0][n], args[1][n] = base + e * d, base - e * d
        num = (loss(*args[0]) - loss(*args[1])) / (2 * e)
        want = float((grad.double() * d.double()).sum())
        say(f"differences {n}: {num:.6g} against {want:.6g}")
        assert abs(num - want) <= 1e-2 * abs(want)


# --------------------------------------------------------------- distillation
def teacher(T, V, k, seed, live=1.0):
    g = torch.Generator().manual_seed(seed)
    idx = torch.randint(0, V, (T, k), generator=g)
    idx[torch.rand((T, k), generator=g) > live] = -1
    return idx.to(torch.int32).to(DEV), (torch.randn((T, k), generator=g) * 3).to(DEV)


def check_distill(z, idx, tl, tau, gloss, loss, lse, dz):
    rl, rs, rz, q, P, g = distill_ref(z, idx, tl, tau, gloss)
    zt = z.double().masked_fill(torch.isinf(z), 0.0).abs().amax(1) / tau
    # exponents are off by 2^-22 of their magnitude (at most 2 max |z| / tau),
    # sums by a few 2^-22
    e = (2 * zt + 8) * 2.0 ** -22
    errs = [worst(lse, rs, e * 2 + rs.abs() * 2.0 ** -22)]
    tt = tl.double().masked_fill(torch.isinf(tl), 0.0).abs().amax(1) / tau
    el = tau * tau * (e + (2 * tt + rs.abs() + 8) * 2.0 ** -21) * 2
    fin = torch.isfinite(rl)
    assert torch.equal(fin, torch.isfinite(loss)) and torch.equal(loss[~fin].double(), rl[~fin])
    if fin.any():
        errs.append(worst(loss[fin], rl[fin], el[fin]))
    if dz is not None:
        b = g.abs() * (q * (e[:, None] * 2) + P * ((2 * tt + 8) * 2.0 ** -21)[:, None])
        b = b + half_step(dz.dtype) * (rz.abs() + b) + 1e-37
        errs.append(worst(dz, rz, b))
    say("  error / bound: " + " ".join("%.3f" % x for x in errs))
    assert max(errs) <= 1.0


DIST = [
    # T, V, k, tau, dtype, padding of the rows
    (1, 1, 1, 1.0, F32, 0),
    (3, 7, 3, 2.0, BF, 0),
    (5, 500, 16, 1.5, F32, 1),
    (2, 4095, 64, 1.0, BF, 2),
    (3, 4097, 65, 0.5, BF, 0),
    (4, 9001, 128, 1.0, F32, 3),
    (1, 131072, 1024, 2.0, BF, 0),
    (2, 70001, 300, 1.0, F32, 0),
    (130, 1023, 8, 1.0, BF, 0),
    (129, 5000, 33, 3.0, F32, 1),
    (128, 16001, 64, 1.0, BF, 7),
    (200, 40000, 64, 1.0, BF, 0),
    (128, 33001, 20, 1.0, F32, 0),
    (131, 65536, 64, 2.0, F32, 0),
    (128, 131072, 64, 2.0, BF, 0),
    (128, 131080, 64, 2.0, BF, 0),
    (140, 70000, 50, 1.0, F32, 0),
]


@pytest.mark.parametrize("T,V,k,tau,dtype,pad", DIST)
def test_distill_topk(T, V, k, tau, dtype, pad):
    say(f"distill T={T} V={V} k={k} tau={tau} {dtype} pad {pad}")
    buf = rnd((T, V + pad), V + k, dtype, 3.0)
    z = buf[:, :V]
    idx, tl = teacher(T, V, k, T + V, live=0.9)
    gl = torch.rand(T, device=DEV)
    out, fine = guarded((T, V + pad), dtype)
    out.fill_(7.0)
    dz = out[:, :V]
    loss, lse, _ = qt.qt_distill_topk(z, idx, tl, tau=tau, gloss=gl, dlogits=dz)
    check_distill(z, idx, tl, tau, gl, loss, lse, dz)
    assert fine() and (out[:, V:] == 7.0).all(), "wrote outside the rows"
    # without the gradient, and the gradient alone
    loss2, lse2, none = qt.qt_distill_topk(z, idx, tl, tau=tau)
    assert none is None and torch.equal(loss, loss2) and torch.equal(lse, lse2)
    dz2 = qt.qt_distill_topk_bwd(z, idx, tl, lse, gl, tau=tau)
    check_distill(z, idx, tl, tau, gl, loss, lse, dz2)
    # in place, both ways
    for bwd in (False, True):
        c = buf.clone()
        if bwd:
            qt.qt_distill_topk_bwd(c[:, :V], idx, tl, lse, gl, tau=tau, dlogits=c[:, :V])
            assert torch.equal(c[:, :V], dz2)
        else:
            l3, s3, _ = qt.qt_distill_topk(c[:, :V], idx, tl, tau=tau, gloss=gl, dlogits=c[:, :V])
            assert torch.equal(l3, loss) and torch.equal(s3, lse) and torch.equal(c[:, :V], dz)
        assert torch.equal(c[:, V:], buf[:, V:])


@pytest.mark.parametrize("T,V", [(6, 300), (6, 9000), (6, 140000), (140, 9000)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_distill_masks_and_repeats(T, V, dtype):
    # -inf and the type's lowest value among the logits, -inf teacher entries,
    # repeated and out-of-range indices, rows without entries holding garbage
    say(f"distill masks T={T} V={V} {dtype}")
    k = 24
    z = rnd((T, V), V, dtype, 2.0)
    idx, tl = teacher(T, V, k, 3)
    z[0, V // 2:] = -math.inf
    idx[0] = torch.arange(k, dtype=torch.int32) % (V // 4)
    z[1, ::2] = torch.finfo(dtype).min
    idx[1] = 2 * torch.arange(k, dtype=torch.int32) + 1
    tl[2, 3:] = -math.inf                      # three entries with mass
    idx[3] = 5                                 # one index k times
    idx[4, ::2] = -1
    idx[4, 1] = V
    idx[4, 3] = 2 ** 31 - 1
    idx[4, 5] = -2 ** 31
    idx[5] = -1                                # no entry
    loss, lse, dz = qt.qt_distill_topk(z, idx, tl, tau=2.0, want_dlogits=True)
    check_distill(z, idx, tl, 2.0, None, loss, lse, dz)
    assert loss[5] == 0 and (dz[5] == 0).all()
    dz2 = qt.qt_distill_topk_bwd(z, idx, tl, lse, tau=2.0)
    check_distill(z, idx, tl, 2.0, None, loss, lse, dz2)
    # mass on a masked logit: infinite loss, finite gradient
    z2 = z.clone()
    z2[2, idx[2, 0].long()] = -math.inf
    idx2 = idx.clone()
    l2, s2, d2 = qt.qt_distill_topk(z2, idx2, tl, tau=2.0, want_dlogits=True)
    assert math.isinf(float(l2[2])) and float(l2[2]) > 0 and torch.isfinite(d2[2]).all()
    # a row without entries (or with -inf ones only) is ignored whatever it holds
    z3 = z.clone()
    z3[5] = math.nan
    z3[4] = -math.inf
    tl3 = tl.clone()
    tl3[4] = -math.inf
    l3, _, d3 = qt.qt_distill_topk(z3, idx, tl3, tau=2.0, want_dlogits=True)
    assert (l3[4:6] == 0).all() and (d3[4:6] == 0).all()
    assert torch.equal(l3[:4], loss[:4]) and torch.equal(d3[:4], dz[:4])
    # a NaN, +inf, or nothing but -inf in a row that counts is seen
    for bad in (math.nan, math.inf):
        z4 = z.clone()
        z4[0, 1] = bad
        l4, s4, d4 = qt.qt_distill_topk(z4, idx, tl, tau=2.0, want_dlogits=True)
        assert math.isnan(float(l4[0])) and torch.isnan(d4[0]).any()
        assert torch.equal(l4[1:], loss[1:]) and torch.equal(d4[1:], dz[1:])
    z4 = z.clone()
    z4[0] = -math.inf
    l4, _, d4 = qt.qt_distill_topk(z4, idx, tl, tau=2.0, want_dlogits=True)
    assert math.isnan(float(l4[0])) and torch.isnan(d4[0]).all()
    # a NaN among the teacher's entries, too
    tl5 = tl.clone()
    tl5[0, 2] = math.nan
    l5, _, d5 = qt.qt_distill_topk(z, idx, tl5, tau=2.0, want_dlogits=True)
    assert math.isnan(float(l5[0])) and torch.equal(l5[1:], loss[1:])


def test_distill_against_differences():
    # d loss / dz along the gradient in f32; e^2 and the f32 noise stay under 1 %
    T, V, k = 3, 400, 12
    z = rnd((T, V), 1, F32, 2.0)
    idx, tl = teacher(T, V, k, 2)
    _, _, dz = qt.qt_distill_topk(z, idx, tl, tau=1.5, want_dlogits=True)
    e = 2.0 ** -6
    d = dz / dz.norm()
    up = qt.qt_distill_topk(z + e * d, idx, tl, tau=1.5)[0].double().sum()
    dn = qt.qt_distill_topk(z - e * d, idx, tl, tau=1.5)[0].double().sum()
    num, want = float((up - dn) / (2 * e)), float((dz.double() * d.double()).sum())
    say(f"distill differences {num:.6g} against {want:.6g}")
    assert abs(num - want) <= 1e-2 * abs(want)


# ----------------------------------------------------------------- the chain
@pytest.mark.parametrize("dtype,T", [(F32, 9), (F32, 70), (BF, 70), (BF, 300)])
def test_tuning_chain(dtype, T):
    """Block, down projection, head and loss forward, then every gradient
    backward through them, against autograd in f64 on the same weights."""
    D, F, V, k, tau = 128, 192, 500, 16, 2.0
    say(f"chain {dtype} T={T}")
    (gate, vg), (up, vu) = quantized(F, D, 3, 1), quantized(F, D, 4, 2)
    (down, vd), (head, vh) = quantized(D, F, 4, 3), quantized(V, D, 3, 4)
    # weights of useful size: outputs of order one
    for w in (gate, up, down, head):
        w[1].mul_(8.0)
    x = rnd((T, D), 1, dtype)
    idx, tl = teacher(T, V, k, 5, live=0.9)
    idx[3] = -1
    gl = torch.full((T,), 1.0 / T, device=DEV)

    h, pre = qt.qt_ffn_gated(gate, up, x, want_pre=True)
    y = qt.qt_matmul_i4(down[0], down[1], D, F, h).to(dtype)
    z = qt.qt_matmul_i3(head[0], head[1], V, D, y)
    loss, lse, dz = qt.qt_distill_topk(z, idx, tl, tau=tau, gloss=gl, want_dlogits=True)
    dy, dsh = qt.qt_matmul_bwd(head, dz, y)
    dhid, dsd = qt.qt_matmul_bwd(down, dy, h)
    dx, dsg, dsu = qt.qt_ffn_gated_bwd(gate, up, pre, dhid, x)

    S = [w[1].double().requires_grad_() for w in (gate, up, down, head)]
    xr = x.double().requires_grad_()

    def dns(v, s, I):
        return (v * s[..., None]).reshape(v.shape[0], -1)[:, :I]

    gr, ur = xr @ dns(vg, S[0], D).t(), xr @ dns(vu, S[1], D).t()
    hr = gr * torch.sigmoid(gr) * ur
    zr = hr @ dns(vd, S[2], F).t() @ dns(vh, S[3], D).t()
    live = idx >= 0
    p = torch.softmax((tl.double() / tau).masked_fill(~live, -math.inf), 1).nan_to_num(0.0)
    lq = torch.log_softmax(zr / tau, 1).gather(1, idx.clamp(min=0).long())
    lp = torch.where(p > 0, p, torch.ones_like(p)).log()
    lr = tau * tau * (p * (lp - lq)).sum(1)
    (lr * gl.double()).sum().backward()

    # errors in norm: f32 keeps about five digits through the four products;
    # bf16 rounds weights, activations and gradients at each of the seven
    # steps (2^-8 at most, about a third of it in the mean)
    tol = 2e-4 if dtype == F32 else 7 * half_step(BF)
    for name, a, b in (("loss", loss, lr.detach()), ("dX", dx, xr.grad), ("gate", dsg, S[0].grad),
                       ("up", dsu, S[1].grad), ("down", dsd, S[2].grad), ("head", dsh, S[3].grad)):
        err = float((a.double() - b).norm() / b.norm())
        say(f"  {name}: {err:.2e}")
        assert err <= tol, name


# ------------------------------------------------------------ streams, graphs
def cases():
    D, F, T = 200, 150, 70
    gate, up = quantized(F, D, 3, 1)[0], quantized(F, D, 4, 2)[0]
    out = []
    for dtype, T in ((BF, 1), (F32, 5), (BF, 70), (F32, 70), (BF, 300)):
        x, dh = rnd((T, D), T, dtype), rnd((T, F), T + 1, dtype)

        def ffn(x=x, dh=dh):
            h, pre = qt.qt_ffn_gated(gate, up, x, want_pre=True)
            return [h, pre, *qt.qt_ffn_gated_bwd(gate, up, pre, dh, x)]

        def lin(x=x, dh=dh):
            return list(qt.qt_matmul_bwd(gate, dh, x))

        out += [(f"ffn {dtype} T={T}", ffn, [x, dh]), (f"linear {dtype} T={T}", lin, [x, dh])]
    for dtype, T, V in ((F32, 4, 9000), (BF, 130, 9000), (BF, 3, 300)):
        z = rnd((T, V), V, dtype)
        idx, tl = teacher(T, V, 20, 1)

        def dist(z=z, idx=idx, tl=tl):
            loss, lse, dz = qt.qt_distill_topk(z, idx, tl, want_dlogits=True)
            return [loss, lse, dz, qt.qt_distill_topk_bwd(z, idx, tl, lse)]

        out.append((f"distill {dtype} T={T} V={V}", dist, [z, tl]))
    return out


def test_graph_replays_equal_eager():
    for tag, run, inputs in cases():
        say(f"graph {tag}")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            captured = run()
        for r in range(3):
            for n, t in enumerate(inputs):
                t.copy_(rnd(t.shape, 100 * r + n, t.dtype))
            torch.cuda.synchronize()
            g.replay()
            eager = run()
            torch.cuda.synchronize()
            for a, b in zip(captured, eager):
                assert torch.equal(a, b), f"{tag}: replay {r} differs"


def test_given_stream_and_workspace():
    D, F, T = 200, 150, 300
    gate, up = quantized(F, D, 3, 1)[0], quantized(F, D, 4, 2)[0]
    x, dh = rnd((T, D), 1, BF), rnd((T, F), 2, BF)
    h, pre = qt.qt_ffn_gated(gate, up, x, want_pre=True)
    want = qt.qt_ffn_gated_bwd(gate, up, pre, dh, x)
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        ws = torch.full((qt.qt_ffn_gated_bwd_workspace_bytes(T, D, F, qt.QT_BF16) + 64,), 0xA5,
                        dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        h2, pre2 = qt.qt_ffn_gated(gate, up, x, want_pre=True, stream=s)
        got = qt.qt_ffn_gated_bwd(gate, up, pre2, dh, x, workspace=ws, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(h, h2) and all(torch.equal(a, b) for a, b in zip(got, want))
        assert (ws[-64:] == 0xA5).all(), "wrote past the workspace"


def test_binding_refusals():
    D, F, T = 128, 64, 4
    gate, up = quantized(F, D, 3, 1)[0], quantized(F, D, 4, 2)[0]
    x = rnd((T, D), 1, BF)
    with pytest.raises(ValueError):
        qt.qt_ffn_gated(gate, up, x, act="relu")
    with pytest.raises(ValueError):
        qt.qt_ffn_gated(gate, (up[0], up[1], 3), x)          # bits do not fit the bytes
    with pytest.raises(ValueError):
        qt.qt_ffn_gated(gate, up, x.half())
    with pytest.raises(ValueError):
        qt.qt_ffn_gated(gate, up, rnd((D, T), 1, BF).t())     # not contiguous
    with pytest.raises(ValueError):
        qt.qt_ffn_gated(gate, up, rnd((T, D + 64), 1, BF))   # other inner size
    with pytest.raises(ValueError):
        qt.qt_ffn_gated(gate, up, x, H=torch.empty((T, F), device=DEV))
    with pytest.raises(qt.QtError):
        qt.qt_ffn_gated(gate, up, x[:0])
    h, pre = qt.qt_ffn_gated(gate, up, x, want_pre=True)
    with pytest.raises(ValueError):
        qt.qt_ffn_gated_bwd(gate, up, pre, h, x, accumulate=True)
    with pytest.raises(qt.QtError):
        qt.qt_ffn_gated_bwd(gate, up, pre, h, x, want_dx=False, want_dscales=False)
    with pytest.raises(qt.QtError):   # the gradient over an input
        qt.qt_ffn_gated_bwd(gate, up, pre, h, x, dX=x)
    z = rnd((T, 50), 1)
    idx, tl = teacher(T, 50, 4, 1)
    with pytest.raises(ValueError):
        qt.qt_distill_topk(z.t(), idx, tl)
    with pytest.raises(ValueError):
        qt.qt_distill_topk(z, idx.long(), tl)
    with pytest.raises(qt.QtError):
        qt.qt_distill_topk(z, idx, tl, tau=0.0)
    with pytest.raises(qt.QtError):   # overlaps the logits, but is not them
        qt.qt_distill_topk(z[:2], idx[:2], tl[:2], dlogits=z[1:3])
    with pytest.raises(qt.QtError):   # one row under all
        qt.qt_distill_topk(z, idx, tl, dlogits=torch.empty((1, 50), device=DEV).expand(T, 50))


def test_offsets_past_32_bits():
    # 70000 tokens x 40000 features (pre: 22 GB) and 20000 rows of 131072
    # logits: the last rows, tokens and sums against references of their own
    T, D, F = 70000, 64, 40000
    say(f"offsets: block {T} x {F}")
    (gate, vg), (up, vu) = quantized(F, D, 3, 1), quantized(F, D, 4, 2)
    x = rnd((T, D), 1, BF)
    H, pre = qt.qt_ffn_gated(gate, up, x, want_pre=True)
    g = torch.Generator(device=DEV).manual_seed(2)
    dh = torch.randn((T, F), generator=g, device=DEV, dtype=BF)
    dX, dsg, dsu = qt.qt_ffn_gated_bwd(gate, up, pre, dh, x)
    wg, wu = dense(gate, vg, D), dense(up, vu, D)
    n = 300
    h, gr, ur, bh, bg, bu = ffn_ref(x[-n:], wg, wu, "silu", BF)
    assert worst(H[-n:], h, bh) <= 1 and worst(pre[0, -n:], gr, bg) <= 1
    assert worst(pre[1, -n:], ur, bu) <= 1
    dg, du, eg, eu = grads_ref(pre[0, -n:].double(), pre[1, -n:].double(), dh[-n:].double(), "silu")
    ref = dg @ wg + du @ wu
    b = dx_bound([(dg, eg, wg), (du, eu, wu)], BF, BF)
    assert worst(dX[-n:], ref, b + half_step(BF) * (ref.abs() + b) + 1e-30) <= 1
    o, X = 40, x.double()
    dg, du, eg, eu = grads_ref(pre[0, :, -o:].double(), pre[1, :, -o:].double(),
                               dh[:, -o:].double(), "silu")
    for got, dy, e, v in ((dsg, dg, eg, vg[-o:]), (dsu, du, eu, vu[-o:])):
        bound = scale_grad(SUM * dy.abs() + e, X.abs(), v.abs()) + 1e-30
        assert worst(got[-o:], scale_grad(dy, X, v), bound) <= 1
    del H, pre, dh, dX, dg, du, eg, eu
    torch.cuda.empty_cache()
    T, V, k = 20000, 131072, 8
    say(f"offsets: loss {T} x {V}")
    z = torch.zeros((T, V), device=DEV, dtype=BF)
    z[-n:] = rnd((n, V), 3, BF)
    idx, tl = teacher(T, V, k, 4)
    loss, lse, dz = qt.qt_distill_topk(z, idx, tl, want_dlogits=True)
    check_distill(z[-n:], idx[-n:], tl[-n:], 1.0, None, loss[-n:], lse[-n:], dz[-n:])
    dz2 = qt.qt_distill_topk_bwd(z, idx, tl, lse)
    check_distill(z[-n:], idx[-n:], tl[-n:], 1.0, None, loss[-n:], lse[-n:], dz2[-n:])


def test_two_calls_at_once():
    # two streams, a workspace each (the binding's own), interleaved launches
    D, F, T = 640, 320, 400
    gate, up = quantized(F, D, 3, 1)[0], quantized(F, D, 4, 2)[0]
    xs = [rnd((T, D), s, BF) for s in (1, 2)]
    dh = rnd((T, F), 3, BF)
    z = [rnd((5, 40000), s, F32) for s in (4, 5)]
    idx, tl = teacher(5, 40000, 16, 6)

    def step(i, stream=None):
        h, pre = qt.qt_ffn_gated(gate, up, xs[i], want_pre=True, stream=stream)
        return [h, *qt.qt_ffn_gated_bwd(gate, up, pre, dh, xs[i], stream=stream),
                *qt.qt_distill_topk(z[i], idx, tl, want_dlogits=True, stream=stream)]

    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [step(i, streams[i]) for i in (0, 1)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
