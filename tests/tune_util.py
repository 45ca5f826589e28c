"""Plain 64-bit forms of the tuning operators and the bounds their tests use
(elementary torch operations on the device the inputs are on)."""
import math

import torch

import dequant_matmul_int3_amd as qt
import workloads
from tests.gpu_util import DEV


def quantized(O, I, bits, seed):
    """(packed, scales, bits) on the device and the codes [O, G, 64] (padded) in f64."""
    W = torch.from_numpy(workloads.generic_weights(O, I, seed=seed)).to(DEV)
    if bits == 3:
        s, c, _ = qt.qt_quantize_g64(W, want_grid_idx=False)
        p = qt.qt_pack_i3(c)
    else:
        s, c, _ = qt.qt_quantize_g64_i4(W, want_grid_idx=False)
        p = qt.qt_pack_i4(c)
    v = torch.nn.functional.pad(c.double(), (0, s.shape[1] * 64 - I)).view(O, -1, 64)
    return (p, s, bits), v


def dense(w, v, I):
    return (v * w[1].double()[..., None]).reshape(v.shape[0], -1)[:, :I]


def act64(z, act):
    """act(z) and act'(z)."""
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    k = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * k * (z + 0.044715 * z ** 3))
    ds = s * torch.sigmoid(-2 * k * (z + 0.044715 * z ** 3)) * 2 * k * (1 + 3 * 0.044715 * z ** 2)
    return z * s, s + z * ds


def half_step(dtype):
    """A rounding to dtype is off by at most this, relative to the value."""
    return torch.finfo(dtype).eps / 2


# f32 sums of exact products: the multiply kernels' bound, relative to the sum
# of the terms' magnitudes
SUM = 1e-5


def ffn_ref(x, wg, wu, act, dtype):
    """h, g, u and bounds of their errors: g and u are off by SUM of sum |w x|;
    |act'| <= 1.13 for both activations."""
    X = x.double()
    g, u = X @ wg.t(), X @ wu.t()
    ag, au = X.abs() @ wg.abs().t(), X.abs() @ wu.abs().t()
    a, _ = act64(g, act)
    bg, bu = SUM * ag, SUM * au
    h = a * u
    # the activation's own f32 operations: a few roundings of a and of the product
    bh = (1.13 * bg + 1e-6 * a.abs()) * (u.abs() + bu) + a.abs() * bu
    return h, g, u, bh + half_step(dtype) * (h.abs() + bh) + 1e-30, bg + 1e-30, bu + 1e-30


def grads_ref(g, u, dh, act):
    """dg, du from f32 pre-activations, with bounds of their f32 evaluation:
    act' is a sum of two terms of magnitude at most 1.2 and |z| sigmoid'."""
    a, da = act64(g, act)
    dg, du = dh * u * da, dh * a
    return dg, du, 2e-6 * (dh * u).abs() * (2 + g.abs()), 2e-6 * du.abs()


def dx_bound(parts, dtype, out_dtype):
    """parts: (dy, bound of dy, w) per matrix.  bf16 calls: dy is rounded once to
    f16 and s v twice (the scale, then the product)."""
    r = half_step(torch.float16) if dtype == torch.bfloat16 else 0.0
    b = 0
    for dy, e, w in parts:
        b = b + (e * (1 + r) + dy.abs() * ((1 + r) ** 3 - 1 + SUM)) @ w.abs() * (1 + r)
    return b


def scale_grad(dy, x, v):
    O, G, _ = v.shape
    dw = torch.nn.functional.pad(dy.t().contiguous() @ x, (0, G * 64 - x.shape[1]))
    return (dw.view(O, G, 64) * v).sum(-1)


def worst(got, ref, bound):
    """Largest error over its bound (inf where got is not finite but ref is)."""
    d = (got.double() - ref).abs() / bound
    return float(torch.nan_to_num(d, nan=math.inf).max())


def distill_ref(z, idx, tl, tau, gloss=None):
    """loss, lse, dlogits in f64 for rows whose inputs are finite or -inf."""
    T, V = z.shape
    z = z.double() / tau
    lse = torch.logsumexp(z, 1)
    live = (idx >= 0) & (idx < V)
    t = (tl.double() / tau).masked_fill(~live, -math.inf)
    mass = (t > -math.inf).any(1)
    p = torch.where(mass[:, None], torch.softmax(t, 1), torch.zeros_like(t))
    p = torch.where(live, p, torch.zeros_like(p))
    at = torch.where(live, idx, torch.zeros_like(idx)).long()
    lp = torch.where(p > 0, torch.log(torch.where(p > 0, p, torch.ones_like(p))),
                     torch.zeros_like(p))
    diff = lp - z.gather(1, at) + lse[:, None]
    loss = tau * tau * torch.where(p > 0, p * diff, torch.zeros_like(p)).sum(1)
    q = torch.where(mass[:, None], torch.exp(z - lse[:, None]), torch.zeros_like(z))
    P = torch.zeros_like(z)
    P.index_put_((torch.arange(T, device=z.device)[:, None].expand_as(at), at), p, accumulate=True)
    g = torch.ones(T, dtype=torch.float64, device=z.device) if gloss is None else gloss.double()
    g = (tau * g)[:, None]
    return loss, lse, torch.where(mass[:, None], g * (q - P), torch.zeros_like(z)), q, P, g
