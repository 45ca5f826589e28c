"""The tuning calls where their inputs' ranges and levels are extreme: closed
gates, tiny gradients, logits far from zero or at the type's lowest value,
rows at odd addresses, the largest sizes.  Bounds count the roundings that the
kernels make (U: half a step of f32) and know nothing of what a fault would do."""
import math

import pytest
import torch

import dequant_matmul_int3_amd as qt
from tests.gpu_util import DEV, say
from tests.tune_util import (SUM, act64, dense, distill_ref, dx_bound, ffn_ref, grads_ref,
                             half_step, quantized, scale_grad, worst)

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def rnd(shape, seed, dtype=F32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


# ------------------------------------------------------------ input gradient
@pytest.mark.parametrize("act,gates", [("silu", (-5.0, -12.0, -30.0, -60.0)),
                                       ("gelu", (-5.0, -6.0, -7.0, -9.0))])
@pytest.mark.parametrize("T", [4, 1028])
def test_gradients_behind_closed_gates(act, gates, T):
    # bf16 tokens whose gradient is not zero only where the gate is closed: the
    # largest gradients are 1e-3 down to 1e-26 there, and each token's own
    # power of two has to follow them.
    # The sigmoid's argument x has at most four roundings, so that the sigmoid
    # e^x is off by (4 |x| + 4) U relative, its products and sums by a few U; for
    # g <= -5 the two terms of act' are far from cancelling.
    D, F = 192, 160
    (gate, vg), (up, vu) = quantized(F, D, 3, 1), quantized(F, D, 4, 2)
    x, dh = rnd((T, D), 3, BF), rnd((T, F), 4, BF, 0.1)
    g = torch.tensor(gates, device=DEV).repeat(T // 4)[:, None]
    g = g * (1 + 0.02 * rnd((T, F), 5).clamp(-2, 2))
    g[:, F // 2:] = 3.0
    dh[:, F // 2:] = 0
    pre = torch.stack([g, rnd((T, F), 6)])
    dX = qt.qt_ffn_gated_bwd(gate, up, pre, dh, x, act=act, want_dscales=False)[0]
    G, u, H = pre[0].double(), pre[1].double(), dh.double()
    a, da = act64(G, act)
    dg, du = H * u * da, H * a
    arg = G if act == "silu" else 2 * math.sqrt(2 / math.pi) * (G + 0.044715 * G ** 3)
    e = (8 * arg.abs() + 32) * U
    wg, wu = dense(gate, vg, D), dense(up, vu, D)
    ref = dg @ wg + du @ wu
    b = dx_bound([(dg, e * dg.abs(), wg), (du, e * du.abs(), wu)], BF, BF)
    # f16's subnormals: 2^-39 of the token's largest gradient for each of 2 F terms
    top = torch.maximum(dg.abs().amax(1), du.abs().amax(1))[:, None]
    b = b + 2.0 ** -38 * 2 * F * 8 * top * max(float(gate[1].max()), float(up[1].max()))
    b = b + half_step(BF) * (ref.abs() + b) + 2.0 ** -133
    r = torch.nan_to_num((dX.double() - ref).abs() / b, nan=math.inf)
    say(f"{act} T={T}: error / bound " +
        " ".join(f"{v}: {float(r[n::4].max()):.3f}" for n, v in enumerate(gates)))
    assert float(r.max()) <= 1.0


def test_tiny_gradients_and_scales():
    # gradients of 2^-112 and scales of 2^-14: the powers of two that bring them
    # into f16's range multiply to 2^150, whose inverse is no f32 number, while dX
    # (2^-122) is a normal bf16 one
    B, I, O = 40, 200, 1024
    w, v = quantized(O, I, 3, 3)
    w[1].mul_(2.0 ** -14 / float(w[1].max()))
    x, dy = rnd((B, I), 1, BF), rnd((B, O), 2).clamp(-2, 2) * 2.0 ** -112
    dX = qt.qt_matmul_bwd(w, dy, x, want_dscales=False)[0]
    W, Y = dense(w, v, I), dy.double()
    ref = Y @ W
    b = dx_bound([(Y, 0 * Y, W)], BF, BF)
    b = b + half_step(BF) * (ref.abs() + b) + 2.0 ** -133  # bf16's smallest step
    assert float(ref.abs().mean()) > 2.0 ** -126
    err = worst(dX, ref, b)
    say(f"error / bound {err:.3f}")
    assert err <= 1.0


@pytest.mark.parametrize("ytype", [BF, F32, "block"])
def test_input_gradient_adds_little_to_its_rounding(ytype):
    # in norm: a rounding to f16 is off by at most 2^-11 / sqrt(3) in the mean
    # square, relative to the value; three of them per term (dY, the scale, its
    # product with the code), of terms of either sign, add (2^-11)^2 at most to
    # the square of what the one rounding of dX itself leaves.  (bf16 operands
    # would add eight times that, which bounds of single values do not see.)
    B, I, O = 256, 512, 1024
    w, v = quantized(O, I, 4, 3)
    x, dy = rnd((B, I), 1, BF), rnd((B, O), 2, BF if ytype == "block" else ytype, 0.1)
    if ytype == "block":
        up, vu = quantized(O, I, 3, 4)
        pre = rnd((2, B, O), 5)
        dX = qt.qt_ffn_gated_bwd(w, up, pre, dy, x, want_dscales=False)[0]
        a, da = act64(pre[0].double(), "silu")
        ref = (dy.double() * pre[1].double() * da) @ dense(w, v, I)
        ref = ref + (dy.double() * a) @ dense(up, vu, I)
    else:
        dX = qt.qt_matmul_bwd(w, dy, x, want_dscales=False)[0]
        ref = dy.double() @ dense(w, v, I)
    err = float((dX.double() - ref).norm() / ref.norm())
    own = float((ref.to(BF).double() - ref).norm() / ref.norm())
    say(f"dY {ytype}: {err:.4e} off in norm, its own rounding {own:.4e}")
    assert err ** 2 <= own ** 2 + half_step(torch.float16) ** 2


# --------------------------------------------------------------- distillation
def level_bounds(z, idx, tl, tau, gloss=None):
    """The 64-bit results and bounds that depend on differences of logits only.
    Relative to U: the row's sum is off by its longest chain of additions (160:
    16 vectors of 8, and the joins; + 40) and by eight roundings of the exponents, whose
    magnitude (m - z_v) / tau counts with its weight q_v; p_j by the same of the
    teacher's exponents and its k / 64 additions per lane.  An error of p_j
    counts with the terms that it multiplies in the loss."""
    T, V = z.shape
    loss, lse, dz, q, P, g = distill_ref(z, idx, tl, tau, gloss)
    z = z.double()
    m = z.amax(1, keepdim=True)
    live = (idx >= 0) & (idx < V)
    t = tl.double().masked_fill(~live, -math.inf)
    d = (t - t.amax(1, keepdim=True)) / tau
    p = torch.softmax(d, 1)
    on = p > 0

    def only(x):
        return torch.where(on, x, torch.zeros_like(p))

    zj = z.gather(1, torch.where(live, idx, torch.zeros_like(idx)).long())
    r = torch.where(on, zj, torch.full_like(zj, -math.inf)).amax(1, keepdim=True)
    span = torch.where(q > 0, (m - z) / tau, torch.zeros_like(q))
    es = U * (min(V, 160) + 40 + 8 * (q * span).sum(1))
    dj = only(d.abs())
    ep = only(U * (8 * dj + 8 * (p * dj).sum(1, keepdim=True) + 2 * (2 * -(-tl.shape[1] // 64) + 16)))
    term = only(p.clamp(min=1e-300).log().abs() + (r - zj) / tau)
    term = term + (m - r) / tau + (lse - m[:, 0] / tau).abs()[:, None] + 1
    el = tau * tau * ((p * only((ep + 8 * U) * term)).sum(1) + es)
    top = ep.amax(1, keepdim=True)
    ez = g.abs() * (q * (es[:, None] + 8 * U * (span + 1)) + P * (top + 4 * U))
    return loss, lse, dz, el, ez, g.abs() * q


def rounded(ref, b, dtype):
    return b + half_step(dtype) * (ref.abs() + b) + 1e-37


FORMS = [(6, 300), (6, 9000), (6, 140000), (140, 9000)]  # row, split, long split, wide row form


@pytest.mark.parametrize("T,V", FORMS)
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("level", [0.0, 300.0, -300.0, 3000.0])
def test_loss_does_not_know_the_logits_level(T, V, dtype, level):
    # softmax and loss do not change when all of a row's logits are shifted, and
    # neither may their error; the teacher's have another level
    k, tau = 32, 1.5
    z = (rnd((T, V), V, F32, 2.0) + level).to(dtype)
    idx = torch.randint(0, V, (T, k), generator=torch.Generator().manual_seed(1))
    idx = idx.to(torch.int32).to(DEV)
    tl = z.gather(1, idx.long()).float() + 0.05 * rnd((T, k), 9) - 2 * level
    gl = torch.rand(T, device=DEV)
    loss, lse, dz = qt.qt_distill_topk(z, idx, tl, tau=tau, gloss=gl, want_dlogits=True)
    rl, rs, rz, el, ez, gq = level_bounds(z, idx, tl, tau, gl)
    # the gradient alone knows lse only, with its rounding
    dz2 = qt.qt_distill_topk_bwd(z, idx, tl, lse, gl, tau=tau)
    ez2 = ez + gq * (4 * U * (1 + rs.abs()))[:, None]
    errs = (worst(loss, rl, el), worst(dz, rz, rounded(rz, ez, dtype)),
            worst(dz2, rz, rounded(rz, ez2, dtype)))
    say(f"T={T} V={V} {dtype} level {level}: error / bound " + " ".join("%.3f" % e for e in errs) +
        f"; loss off by {float((loss.double() - rl).abs().max()):.1e}")
    assert max(errs) <= 1.0


@pytest.mark.parametrize("T,V", FORMS)
@pytest.mark.parametrize("tau", [0.25, 0.5])
def test_loss_of_a_lowest_logit_at_low_temperature(T, V, tau):
    # z / tau passes the largest f32 number there, the loss does not
    z = rnd((T, V), V, F32, 2.0)
    z[:, 5] = torch.finfo(F32).min
    idx = torch.arange(5, 13, dtype=torch.int32).repeat(T, 1).to(DEV)
    tl = rnd((T, 8), 9)
    loss = qt.qt_distill_topk(z, idx, tl, tau=tau)[0]
    rl, _, _, el, _, _ = level_bounds(z, idx, tl, tau)
    assert torch.isfinite(loss).all() and worst(loss, rl, el) <= 1.0


@pytest.mark.parametrize("T,V", FORMS)
@pytest.mark.parametrize("dtype", [F32, BF])
def test_logits_masked_with_the_lowest_value(T, V, dtype):
    # half of every row masked with the type's lowest value; bounds of what is
    # left alone, and proof that they would see a wrong loss or gradient
    k, tau = 24, 2.0
    z = rnd((T, V), V, dtype, 2.0)
    z[:, ::2] = torch.finfo(dtype).min
    idx = (2 * torch.arange(k, dtype=torch.int32) + 1).repeat(T, 1).to(DEV)
    tl = rnd((T, k), 4, F32, 3.0)
    loss, lse, dz = qt.qt_distill_topk(z, idx, tl, tau=tau, want_dlogits=True)
    dz2 = qt.qt_distill_topk_bwd(z, idx, tl, lse, tau=tau)
    rl, rs, rz, el, ez, gq = level_bounds(z, idx, tl, tau)
    ez2 = ez + gq * (4 * U * (1 + rs.abs()))[:, None]
    errs = (worst(loss, rl, el), worst(lse, rs, el / tau ** 2 + 4 * U * (1 + rs.abs())),
            worst(dz, rz, rounded(rz, ez, dtype)), worst(dz2, rz, rounded(rz, ez2, dtype)))
    say(f"T={T} V={V} {dtype}: error / bound " + " ".join("%.3f" % e for e in errs))
    assert max(errs) <= 1.0
    assert (dz[:, ::2] == 0).all() and (dz2[:, ::2] == 0).all()
    assert worst(loss * 1.01, rl, el) > 1 and worst(dz * 1.02, rz, rounded(rz, ez, dtype)) > 1


@pytest.mark.parametrize("T,V", FORMS)
@pytest.mark.parametrize("tau", [2.0 ** -100, 1e-4, 100.0, 2.0 ** 60, 2.0 ** 100])
def test_temperatures(T, V, tau):
    z = rnd((T, V), V, F32, 2.0)
    idx = torch.randint(0, V, (T, 9), generator=torch.Generator().manual_seed(2))
    idx = idx.to(torch.int32).to(DEV)
    tl = rnd((T, 9), 9)
    loss, lse, dz = qt.qt_distill_topk(z, idx, tl, tau=tau, want_dlogits=True)
    rl, rs, rz, el, ez, _ = level_bounds(z, idx, tl, tau)
    if tau == 2.0 ** 100:  # tau^2 times any loss here passes the largest f32
        assert torch.isinf(loss).all() and (loss > 0).all()
    else:
        assert worst(loss, rl, el + 1e-37) <= 1.0
    assert worst(dz, rz, rounded(rz, ez, F32)) <= 1.0
    assert worst(lse, rs, 8 * U * (1 + rs.abs()) + 200 * U) <= 1.0
    say(f"tau {tau} V={V}: loss {float(loss[0]):.4g}")


# ------------------------------------------------------------------ alignment
@pytest.mark.parametrize("T", [4, 64, 65, 300])
def test_rows_at_an_odd_element(T):
    # bf16 inputs, gradients and outputs one element off: only the small forward
    # call, which may read rows of whole groups in place, wants 16 bytes
    D, F = 128, 64
    gate, up = quantized(F, D, 3, 1)[0], quantized(F, D, 4, 2)[0]

    def off(t):
        y = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:].view(t.shape)
        return y.copy_(t)

    x, dh = rnd((T, D), 1, BF), rnd((T, F), 2, BF)
    h, pre = qt.qt_ffn_gated(gate, up, x, want_pre=True)
    if T > 64:
        assert torch.equal(qt.qt_ffn_gated(gate, up, off(x), H=off(h)), h)
    else:
        with pytest.raises(qt.QtError):
            qt.qt_ffn_gated(gate, up, off(x))
    want = qt.qt_ffn_gated_bwd(gate, up, pre, dh, x)
    got = qt.qt_ffn_gated_bwd(gate, up, off(pre), off(dh), off(x), dX=off(x))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    want, got = qt.qt_matmul_bwd(gate, dh, x), qt.qt_matmul_bwd(gate, off(dh), off(x), dX=off(x))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------- ends of the documented sizes
def matrix(O, I, bits, seed):
    """A matrix of random codes and scales, drawn on the device, and its codes."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    half = 4 if bits == 3 else 8
    c = torch.randint(-half, half, (O, I), generator=g, device=DEV, dtype=torch.int8)
    s = torch.rand((O, -(-I // 64)), generator=g, device=DEV) * 0.02 + 0.001
    p = (qt.qt_pack_i3 if bits == 3 else qt.qt_pack_i4)(c)
    v = torch.nn.functional.pad(c.double(), (0, s.shape[1] * 64 - I)).view(O, -1, 64)
    return (p, s, bits), v


def drawn(shape, seed, dtype):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, device=DEV, generator=g).to(dtype)


@pytest.mark.parametrize("D", [7168, 8192, 1 << 17, 1 << 20])
@pytest.mark.parametrize("T,dtype", [(1, BF), (65, BF), (600, BF), (70, F32)])
def test_sums_of_equal_terms(T, dtype, D):
    # equal terms make every addition of a long sum round the same way: 2^-24 of
    # the sum for each of its groups at most, which is 1e-5 for 8192 inputs
    F = 24
    c = torch.ones((F, D), dtype=torch.int8, device=DEV)
    s = torch.linspace(0.01, 0.02, F, device=DEV)[:, None].expand(F, D // 64).contiguous()
    w = (qt.qt_pack_i3(c), s, 3)
    x = torch.full((T, D), 1.171875, dtype=dtype, device=DEV)
    _, pre = qt.qt_ffn_gated(w, w, x, want_pre=True)
    ref = (s[:, 0].double() * D * 1.171875).expand(T, F)
    err = float(((pre.double() - ref) / ref).abs().max())
    say(f"T={T} D={D} {dtype}: {err:.1e}")
    assert err <= SUM * max(1.0, D / 8192)


# -------------------------------------------------------------- largest sizes
def room(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of free device memory")


def test_most_tokens_through_the_input_planes():
    # 2^22 tokens of 8256: the planes' launch has more than 2^32 threads (69 GB
    # of inputs and as much of planes)
    room(140)
    T, D, F, n = 1 << 22, 8256, 16, 300
    say(f"block {T} x {D}")
    (gate, vg), (up, vu) = quantized(F, D, 3, 1), quantized(F, D, 4, 2)
    x = torch.zeros((T, D), dtype=BF, device=DEV)
    at = [0, T // 2 - n // 2, T - n]
    for i, t in enumerate(at):
        x[t:t + n] = rnd((n, D), i, BF)
    h = qt.qt_ffn_gated(gate, up, x)
    for t in at:
        ref, _, _, b, _, _ = ffn_ref(x[t:t + n], dense(gate, vg, D), dense(up, vu, D), "silu", BF)
        assert worst(h[t:t + n], ref, b) <= 1.0
        h[t:t + n] = 0
    assert not h.any()
    del x, h
    torch.cuda.empty_cache()


def test_most_rows_of_logits():
    # 2^22 rows that take 1024 threads each: 2^32 threads (137 GB of logits, whose
    # gradient replaces them)
    room(140)
    T, V, n = 1 << 22, 16392, 300
    say(f"loss {T} x {V}")
    z = torch.zeros((T, V), dtype=BF, device=DEV)
    idx = torch.full((T, 2), -1, dtype=torch.int32, device=DEV)
    tl = torch.zeros((T, 2), device=DEV)
    at = [0, T // 2 - n // 2, T - n]
    want = []
    for i, t in enumerate(at):
        z[t:t + n] = rnd((n, V), i, BF, 2.0)
        idx[t:t + n] = torch.randint(0, V, (n, 2), device=DEV, dtype=torch.int32)
        tl[t:t + n] = rnd((n, 2), i + 9)
        want.append(level_bounds(z[t:t + n], idx[t:t + n], tl[t:t + n], 1.0))
    loss, lse, _ = qt.qt_distill_topk(z, idx, tl, dlogits=z)
    for t, (rl, rs, rz, el, ez, _) in zip(at, want):
        assert worst(loss[t:t + n], rl, el) <= 1.0
        assert worst(z[t:t + n], rz, rounded(rz, ez, BF)) <= 1.0
        assert worst(lse[t:t + n], rs, el + 4 * U * (1 + rs.abs())) <= 1.0
        loss[t:t + n], lse[t:t + n], z[t:t + n] = 0, math.log(V), 0
    # rows without entries: no loss, no gradient, the lse of equal logits
    assert not loss.any() and float((lse - math.log(V)).abs().max()) <= 200 * U
    assert float(z.view(torch.int32).amax()) == 0 == float(z.view(torch.int32).amin())
    del z, want
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,D,F,bits,dtype", [
    (1, 1 << 20, 33, (3, 4), BF),
    (1, 1 << 20, 33, (4, 3), F32),
    (70, 1 << 20, 20, (3, 3), BF),
    (30, 1 << 20, 20, (4, 4), F32),
    (3, 100, 1 << 20, (4, 3), BF),
    (70, 64, 1 << 20, (3, 4), F32),
    (1 << 22, 65, 40, (3, 3), BF),
    ((1 << 21) + 1, 70, 24, (4, 4), F32),
])
def test_longest_axes(T, D, F, bits, dtype):
    # random signs keep the long sums' errors far under SUM of their terms
    room(40)
    say(f"block {T} x {D} x {F} {dtype}")
    (gate, vg), (up, vu) = matrix(F, D, bits[0], 1), matrix(F, D, bits[1], 2)
    x, dh = drawn((T, D), 3, dtype), drawn((T, F), 4, dtype)
    h, pre = qt.qt_ffn_gated(gate, up, x, want_pre=True)
    dx, dsg, dsu = qt.qt_ffn_gated_bwd(gate, up, pre, dh, x)
    wg, wu = dense(gate, vg, D), dense(up, vu, D)
    t = slice(max(0, T - 5000), T)
    rh, g, u, bh, bg, bu = ffn_ref(x[t], wg, wu, "silu", dtype)
    errs = [worst(pre[0, t], g, bg), worst(pre[1, t], u, bu), worst(h[t], rh, bh)]
    dg, du, eg, eu = grads_ref(pre[0, t].double(), pre[1, t].double(), dh[t].double(), "silu")
    ref = dg @ wg + du @ wu
    b = dx_bound([(dg, eg, wg), (du, eu, wu)], dtype, dtype)
    errs.append(worst(dx[t], ref, b + half_step(dtype) * (ref.abs() + b) + 1e-30))
    o = slice(max(0, F - 5000), F)
    dg, du, eg, eu = grads_ref(pre[0, :, o].double(), pre[1, :, o].double(), dh[:, o].double(), "silu")
    X = x.double()
    for got, dy, e, v in ((dsg, dg, eg, vg[o]), (dsu, du, eu, vu[o])):
        bound = scale_grad(SUM * dy.abs() + e, X.abs(), v.abs()) + 1e-30
        errs.append(worst(got[o], scale_grad(dy, X, v), bound))
    say("  error / bound: " + " ".join("%.3f" % e for e in errs))
    assert max(errs) <= 1.0


def test_one_matrix_and_one_tensor_twice():
    w, _ = matrix(128, 128, 3, 1)
    x = rnd((200, 128), 1, BF)
    h, pre = qt.qt_ffn_gated(w, w, x, want_pre=True)
    assert torch.equal(pre[0], pre[1])
    got, want = qt.qt_ffn_gated_bwd(w, w, pre, x, x), qt.qt_ffn_gated_bwd(w, w, pre, x.clone(), x)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,V", [(3, 1), (200, 3), (2, 9000), (130, 9000)])
def test_most_entries_on_few_indices(T, V):
    k = 1024
    z = rnd((T, V), 5, F32, 2.0)
    idx = torch.randint(0, min(V, 3), (T, k), generator=torch.Generator().manual_seed(1))
    idx, tl = idx.to(torch.int32).to(DEV), rnd((T, k), 6)
    loss, lse, dz = qt.qt_distill_topk(z, idx, tl, want_dlogits=True)
    rl, rs, rz, el, ez, gq = level_bounds(z, idx, tl, 1.0)
    # an index's p is a sum of up to 1024 in a row, at most 1 in all
    assert worst(loss, rl, el) <= 1.0 and worst(dz, rz, rounded(rz, ez + k * U, F32)) <= 1.0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_widest_rows(dtype):
    # 2^31 - 1 logits, all 0 but the last thousand; f32 sums of 2^31 terms: each
    # thread adds 32768 of them, 32 at a time (1024 additions in a row), then
    # the 256 chunks are joined
    room(40)
    T, V, n = 2, (1 << 31) - 1, 1000
    say(f"loss {T} x {V} {dtype}")
    z = torch.zeros((T, V), dtype=dtype, device=DEV)
    z[1, -n:] = rnd((n,), 3, dtype, 3.0) + 20
    idx = torch.tensor([[0, V - 1, V - 2], [V - 1, 5, V - 3]], dtype=torch.int32, device=DEV)
    tl = rnd((2, 3), 4)
    loss, lse, _ = qt.qt_distill_topk(z, idx, tl)
    rest = torch.tensor([math.log(V), math.log(V - n)], dtype=torch.float64, device=DEV)
    tail = torch.logsumexp(torch.cat([z[1, -n:].double(), rest[1:]]), 0)
    rs = torch.stack([rest[0], tail])
    p = torch.softmax(tl.double(), 1)
    zi = torch.stack([z[r][idx[r].long()] for r in range(T)]).double()
    rl = (p * (p.log() - zi + rs[:, None])).sum(1)
    e = (1024 + 256 + 64) * U + 8 * U * 32
    assert worst(lse, rs, torch.full_like(rs, e)) <= 1.0
    assert worst(loss, rl, torch.full_like(rl, 2 * e)) <= 1.0
    rz = torch.exp(zi - rs[:, None]) - p
    middle = torch.exp(-rs)
    qt.qt_distill_topk_bwd(z, idx, tl, lse, dlogits=z)
    got = torch.stack([z[r][idx[r].long()] for r in range(T)])
    assert worst(got, rz, rounded(rz, e + 16 * U, dtype)) <= 1.0
    assert worst(z[:, V // 2], middle, rounded(middle, middle * (2 * e + 64 * U), dtype)) <= 1.0
    del z
    torch.cuda.empty_cache()


# ------------------------------------------------------------------ workspaces
@pytest.mark.parametrize("T,dtype", [(1, F32), (20, BF), (70, BF), (70, F32), (700, BF)])
def test_what_a_workspace_held_does_not_matter(T, dtype):
    # of exactly the size asked for, full of NaN, and reused by the next call
    D, F, V = 700, 520, 9001
    (gate, _), (up, _) = matrix(F, D, 3, 1), matrix(F, D, 4, 2)
    x, dh, z = rnd((T, D), 1, dtype), rnd((T, F), 2, dtype), rnd((T, V), 3, dtype)
    idx = torch.randint(0, V, (T, 9), generator=torch.Generator().manual_seed(4))
    idx, tl = idx.to(torch.int32).to(DEV), rnd((T, 9), 5)
    xt = qt.QT_BF16 if dtype == BF else qt.QT_F32
    sizes = [qt.qt_ffn_gated_workspace_bytes(T, D, F, xt),
             qt.qt_ffn_gated_bwd_workspace_bytes(T, D, F, xt),
             qt.qt_matmul_bwd_workspace_bytes(T, D, F, xt),
             qt.qt_distill_topk_workspace_bytes(T, V, xt)]
    buf = torch.full((max(sizes) + 256,), 0xFF, dtype=torch.uint8, device=DEV)

    def run(ws):
        h, pre = qt.qt_ffn_gated(gate, up, x, want_pre=True, workspace=ws(0))
        return [h, pre, *qt.qt_ffn_gated_bwd(gate, up, pre, dh, x, workspace=ws(1)),
                *qt.qt_matmul_bwd(gate, dh, x, workspace=ws(2)),
                *qt.qt_distill_topk(z, idx, tl, want_dlogits=True, workspace=ws(3))]

    want = run(lambda n: None)
    for _ in range(2):
        got = run(lambda n: buf[:max(sizes[n], 16)])
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert (buf[max(sizes):] == 0xFF).all(), "wrote past the workspace"


def test_gradient_in_place_in_a_graph():
    for T, V, dtype in ((4, 300, F32), (3, 40000, BF), (140, 9000, BF)):
        z, out = rnd((T, V), 1, dtype), torch.empty((T, V), dtype=dtype, device=DEV)
        idx = torch.randint(0, V, (T, 9), generator=torch.Generator().manual_seed(4))
        idx, tl = idx.to(torch.int32).to(DEV), rnd((T, 9), 5)

        def run():
            loss, lse, _ = qt.qt_distill_topk(out, idx, tl, dlogits=out)
            return loss, lse

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            out.copy_(z)
            run()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            captured = run()
        for r in range(3):
            z.copy_(rnd((T, V), 10 + r, dtype))
            want = qt.qt_distill_topk(z, idx, tl, want_dlogits=True)
            out.copy_(z)
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip((*captured, out), want):
                assert torch.equal(a, b), f"T={T} V={V}: replay {r} differs"
