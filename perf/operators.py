"""The operators that tune a quantized feed-forward block, as cases to measure.

Four paths of a program that serves or tunes group-scaled int3 / int4 weights:

* `ffn`     the gated feed-forward block's first half, h = act(Wg x) * (Wu x),
            on packed weights (serving: one token, a small batch, a prompt);
* `tune`    that block's training step: the forward pass that keeps the
            pre-activations, then the gradients of the input and of both
            projections' group scales;
* `linear`  the backward pass of one quantized linear layer (the output head,
            the down projection): the gradients of its input and scales;
* `distill` the loss that drives the tuning, KL from a teacher's top logits to
            the student's softmax, with the gradient of the student's logits,
            in one call where the gradient of the loss is known beforehand and
            in two where it is not.

The plain forms below are elementary torch operations in 32 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
GROUP = 64


# --------------------------------------------------------------------- cases
def _ffn(name, T, D, F, bits, act, dtype):
    return {"name": name, "kind": "ffn", "T": T, "D": D, "F": F, "gate_bits": bits[0],
            "up_bits": bits[1], "act": act, "dtype": dtype}


def _tune(name, T, D, F, bits, act, dtype):
    return dict(_ffn(name, T, D, F, bits, act, dtype), kind="tune")


def _linear(name, T, D, O, bits, dtype, ydtype):
    return {"name": name, "kind": "linear", "T": T, "D": D, "O": O, "bits": bits, "dtype": dtype,
            "ydtype": ydtype}


def _distill(name, T, V, pad, k, tau, dtype, fused):
    return {"name": name, "kind": "distill", "T": T, "V": V, "pad": pad, "k": k, "tau": tau,
            "dtype": dtype, "fused": fused}


def listed():
    return [
        # one token through an expert-sized block: the latency of a decode step
        _ffn("ffn-1-token", 1, 7168, 2048, (3, 3), "silu", "f32"),
        # one token through a dense block: the weights' stream bounds it
        _ffn("ffn-1-token-wide", 1, 7168, 18432, (3, 3), "silu", "bf16"),
        # a small decode batch, mixed bits per projection
        _ffn("ffn-12-tokens", 12, 7168, 18432, (4, 3), "silu", "bf16"),
        # a prompt
        _ffn("ffn-prompt", 512, 7168, 18432, (3, 3), "silu", "bf16"),
        # a ragged chunk in f32: a short last group of inputs, odd feature count
        _ffn("ffn-ragged-f32", 77, 7200, 2049, (3, 4), "gelu", "f32"),
        # a tuning step over a batch of calibration tokens
        _tune("tune-large", 4096, 5120, 17408, (3, 3), "silu", "bf16"),
        # a small one: few tokens, an expert-sized block, mixed bits
        _tune("tune-small", 200, 7168, 2048, (4, 3), "gelu", "bf16"),
        # the output head's gradients: f32 logits' gradient, bf16 inputs, odd vocabulary
        _linear("linear-head", 1024, 2048, 50257, 4, "bf16", "f32"),
        # one expert-sized projection in f32
        _linear("linear-f32", 96, 7168, 2048, 3, "f32", "f32"),
        # the loss over a large vocabulary, the gradient formed in the same call
        _distill("distill-large", 2048, 131072, 0, 64, 2.0, "bf16", True),
        # a short ragged batch: few rows, odd vocabulary in padded rows
        _distill("distill-short", 7, 50257, 47, 16, 1.0, "f32", True),
        # loss and gradient apart, as a gradient that comes from further on needs it
        _distill("distill-apart", 1024, 32000, 0, 128, 1.5, "bf16", False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("ffn", "ffn", "tune", "linear", "distill", "distill"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    bits = (rng.choice((3, 4)), rng.choice((3, 4)))
    act = rng.choice(("silu", "gelu"))
    if kind == "distill":
        T, V = _log(rng, 1, 2048), _log(rng, 500, 131072)
        return {"kind": kind, "T": T, "V": V, "pad": rng.choice((0, 0, 1, 63)),
                "k": min(V, _log(rng, 1, 256)), "tau": rng.choice((1.0, 1.5, 2.0)),
                "dtype": dtype, "fused": rng.random() < 0.5}
    # widths of every residue: mostly whole groups of inputs, some ragged
    D = _log(rng, 128, 7168)
    D = D if rng.random() < 0.3 else max(128, D // 64 * 64)
    if kind == "linear":
        return {"kind": kind, "T": _log(rng, 1, 2048), "D": D, "O": _log(rng, 64, 18432),
                "bits": bits[0], "dtype": dtype,
                "ydtype": "f32" if dtype == "f32" else rng.choice(("bf16", "f32"))}
    most = 4096 if kind == "ffn" else 2048
    return {"kind": kind, "T": _log(rng, 1, most), "D": D, "F": _log(rng, 64, 18432),
            "gate_bits": bits[0], "up_bits": bits[1], "act": act, "dtype": dtype}


# -------------------------------------------------------------------- inputs
def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _pack(codes, bits):
    """Codes [O, G, 64] -> packed bytes: int3-g64 planes or int4 nibbles."""
    O, G, _ = codes.shape
    if bits == 4:
        u = (codes + 8).view(O, G, 32, 2)
        return (u[..., 0] | (u[..., 1] << 4)).to(torch.uint8).reshape(-1)
    u = codes + 4
    lo = ((u & 3).view(O, G, 16, 4) << torch.tensor([0, 2, 4, 6], device=DEV)).sum(-1)
    hi = ((u >> 2).view(O, G, 8, 8) << torch.arange(8, device=DEV)).sum(-1)
    return torch.cat([lo, hi], -1).to(torch.uint8).reshape(-1)


def _weights(gen, O, I, bits):
    """A quantized matrix [O x I]: N(0, 0.02) weights with 0.5 % outliers of
    N(0, 0.5), rounded to the group's absmax scale -> (packed, scales)."""
    G = -(-I // GROUP)
    w = torch.randn((O, I), generator=gen, device=DEV) * 0.02
    out = torch.rand((O, I), generator=gen, device=DEV) < 0.005
    w = torch.where(out, w * 25.0, w)
    w = torch.nn.functional.pad(w, (0, G * GROUP - I)).view(O, G, GROUP)
    half = 4 if bits == 3 else 8
    s = w.abs().amax(-1) / half
    q = torch.round(w / torch.where(s > 0, s, torch.ones_like(s))[..., None])
    return _pack(q.clamp(-half, half - 1).to(torch.int32), bits), s.contiguous()


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + 17)
    st = {"case": case}
    T = case["T"]

    def normal(shape, std, dtype):
        return (torch.randn(shape, generator=gen, device=DEV) * std).to(_dt(dtype))

    if case["kind"] in ("ffn", "tune"):
        D, F = case["D"], case["F"]
        st["gate"] = (*_weights(gen, F, D, case["gate_bits"]), case["gate_bits"])
        st["up"] = (*_weights(gen, F, D, case["up_bits"]), case["up_bits"])
        st["X"] = normal((T, D), 1.0, case["dtype"])
        if case["kind"] == "tune":
            st["dH"] = normal((T, F), 0.01, case["dtype"])
    elif case["kind"] == "linear":
        st["w"] = (*_weights(gen, case["O"], case["D"], case["bits"]), case["bits"])
        st["X"] = normal((T, case["D"]), 1.0, case["dtype"])
        st["dY"] = normal((T, case["O"]), 0.01, case["ydtype"])
    else:
        V, k = case["V"], case["k"]
        z = torch.randn((T, V), generator=gen, device=DEV) * 2.5
        # the teacher agrees with the student up to noise; its largest k logits are kept
        t = z + torch.randn((T, V), generator=gen, device=DEV)
        top, idx = torch.topk(t, k, dim=1)
        del t
        # some rows keep fewer than k entries, some (padding tokens) keep none
        keep = torch.randint(1, k + 1, (T, 1), generator=gen, device=DEV)
        full = torch.rand((T, 1), generator=gen, device=DEV) < 0.8
        none = torch.rand((T, 1), generator=gen, device=DEV) < 0.05
        keep = torch.where(full, torch.full_like(keep, k), keep)
        keep = torch.where(none, torch.zeros_like(keep), keep)
        live = torch.arange(k, device=DEV)[None, :] < keep
        st["idx"] = torch.where(live, idx, torch.full_like(idx, -1)).to(torch.int32)
        st["tlogits"] = top.contiguous()
        rows = torch.zeros((T, V + case["pad"]), dtype=_dt(case["dtype"]), device=DEV)
        rows[:, :V] = z.to(rows.dtype)
        st["logits"] = rows[:, :V]  # rows of a padded vocabulary
        st["gloss"] = torch.rand((T,), generator=gen, device=DEV) / T
    return st


# --------------------------------------------------------------- plain forms
def _codes(packed, scales, bits):
    """Packed bytes -> codes [O, G, 64] as f32."""
    O, G = scales.shape
    b = packed.view(O, G, -1).to(torch.int32)
    if bits == 4:
        return (torch.stack([b & 15, b >> 4], -1).reshape(O, G, 64) - 8).float()
    two = torch.arange(0, 8, 2, device=b.device, dtype=torch.int32)
    one = torch.arange(0, 8, 1, device=b.device, dtype=torch.int32)
    lo = ((b[..., :16, None] >> two) & 3).reshape(O, G, 64)
    hi = ((b[..., 16:, None] >> one) & 1).reshape(O, G, 64)
    return (lo + 4 * hi - 4).float()


def _dense(w, I):
    """(packed, scales, bits) -> the [O x I] f32 matrix that it denotes."""
    c = _codes(*w)
    return (c * w[1][..., None]).view(c.shape[0], -1)[:, :I]


def _act(z, act):
    """The activation and its derivative, in z's type."""
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    th = torch.tanh(c * (z + 0.044715 * z * z * z))
    return (0.5 * z * (1.0 + th),
            0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * z * z))


def _scale_grad(dy, x, w):
    """sum over t of dy[t, o] * sum over j of v[o, 64 g + j] x[t, 64 g + j], f32 [O x G]."""
    c = _codes(*w)
    O, G, _ = c.shape
    dw = torch.nn.functional.pad(dy.t() @ x, (0, G * GROUP - x.shape[1]))
    return (dw.view(O, G, GROUP) * c).sum(-1)


def _plain_ffn(st):
    case = st["case"]
    x = st["X"].float()
    g = x @ _dense(st["gate"], case["D"]).t()
    u = x @ _dense(st["up"], case["D"]).t()
    return (_act(g, case["act"])[0] * u).to(st["X"].dtype)


def _plain_tune(st):
    case, dt = st["case"], st["X"].dtype
    x, dh = st["X"].float(), st["dH"].float()
    wg, wu = _dense(st["gate"], case["D"]), _dense(st["up"], case["D"])
    g, u = x @ wg.t(), x @ wu.t()
    a, da = _act(g, case["act"])
    dg, du = dh * u * da, dh * a
    return {"h": (a * u).to(dt), "dx": (dg @ wg + du @ wu).to(dt),
            "dgate_scales": _scale_grad(dg, x, st["gate"]),
            "dup_scales": _scale_grad(du, x, st["up"])}


def _plain_linear(st):
    case = st["case"]
    x, dy = st["X"].float(), st["dY"].float()
    return {"dx": (dy @ _dense(st["w"], case["D"])).to(st["X"].dtype),
            "dscales": _scale_grad(dy, x, st["w"])}


def _plain_distill(st):
    case = st["case"]
    tau, idx = case["tau"], st["idx"].long()
    z = st["logits"].float() / tau
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    s = e.sum(1, keepdim=True)
    lse = m + torch.log(s)
    live = idx >= 0
    t = torch.where(live, st["tlogits"] / tau, torch.full_like(st["tlogits"], -math.inf))
    some = live.any(1, keepdim=True)
    tm = torch.where(some, t.amax(1, keepdim=True), torch.zeros_like(m))
    te = torch.exp(t - tm)
    ts = torch.where(some, te.sum(1, keepdim=True), torch.ones_like(m))
    p = te / ts
    at = idx.clamp(min=0)
    lp = (t - tm) - torch.log(ts)
    terms = p * (lp - (z.gather(1, at) - lse))
    loss = tau * tau * torch.where(p > 0, terms, torch.zeros_like(p)).sum(1)
    q = torch.where(some, e / s, torch.zeros_like(e))
    dz = (tau * st["gloss"])[:, None] * q.scatter_add(1, at, -p)
    return {"loss": loss, "lse": lse[:, 0], "dlogits": dz.to(st["logits"].dtype)}


def run(state):
    case = state["case"]
    kind = case["kind"]
    if own:
        import dequant_matmul_int3_amd as qt
        if kind == "ffn":
            return qt.qt_ffn_gated(state["gate"], state["up"], state["X"], act=case["act"])
        if kind == "tune":
            h, pre = qt.qt_ffn_gated(state["gate"], state["up"], state["X"], act=case["act"],
                                     want_pre=True)
            dx, dgs, dus = qt.qt_ffn_gated_bwd(state["gate"], state["up"], pre, state["dH"],
                                               state["X"], act=case["act"])
            return {"h": h, "dx": dx, "dgate_scales": dgs, "dup_scales": dus}
        if kind == "linear":
            dx, ds = qt.qt_matmul_bwd(state["w"], state["dY"], state["X"])
            return {"dx": dx, "dscales": ds}
        if case["fused"]:
            loss, lse, dz = qt.qt_distill_topk(state["logits"], state["idx"], state["tlogits"],
                                               tau=case["tau"], gloss=state["gloss"],
                                               want_dlogits=True)
        else:
            loss, lse, _ = qt.qt_distill_topk(state["logits"], state["idx"], state["tlogits"],
                                              tau=case["tau"])
            dz = qt.qt_distill_topk_bwd(state["logits"], state["idx"], state["tlogits"], lse,
                                        state["gloss"], tau=case["tau"])
        return {"loss": loss, "lse": lse, "dlogits": dz}
    if kind == "ffn":
        return _plain_ffn(state)
    if kind == "tune":
        return _plain_tune(state)
    if kind == "linear":
        return _plain_linear(state)
    return _plain_distill(state)


# ------------------------------------------------------------ work and truth
def _wbytes(O, I, bits):
    return O * -(-I // GROUP) * ((24 if bits == 3 else 32) + 4)


def work(case):
    T, kind = case["T"], case["kind"]
    e = 2 if case["dtype"] == "bf16" else 4
    if kind in ("ffn", "tune"):
        D, F = case["D"], case["F"]
        w = _wbytes(F, D, case["gate_bits"]) + _wbytes(F, D, case["up_bits"])
        if kind == "ffn":
            return {"bytes": w + T * (D + F) * e, "flops": 4 * T * D * F}
        # in: weights, X, dH; out: H, dX and the scales' gradients
        return {"bytes": w + T * (2 * D + 2 * F) * e + 2 * F * -(-D // GROUP) * 4,
                "flops": 12 * T * D * F}
    if kind == "linear":
        D, O = case["D"], case["O"]
        ye = 2 if case["ydtype"] == "bf16" else 4
        return {"bytes": _wbytes(O, D, case["bits"]) + 2 * T * D * e + T * O * ye
                + O * -(-D // GROUP) * 4, "flops": 4 * T * D * O}
    return {"bytes": T * (2 * case["V"] * e + case["k"] * 8 + 12), "flops": 5 * T * case["V"]}


def _dense64(w, I):
    """The same matrix from the format's words alone, in 64 bits."""
    packed, scales, bits = w
    O, G = scales.shape
    j = torch.arange(64, device=packed.device)
    b = packed.view(O, G, -1)
    if bits == 4:
        v = ((b[:, :, j // 2] >> (4 * (j % 2)).to(torch.uint8)) & 15).to(torch.int16) - 8
    else:
        lo = (b[:, :, j // 4] >> (2 * (j % 4)).to(torch.uint8)) & 3
        hi = (b[:, :, 16 + j // 8] >> (j % 8).to(torch.uint8)) & 1
        v = (lo | (hi << 2)).to(torch.int16) - 4
    v = v.double()
    return (v * scales.double()[:, :, None]).view(O, G * 64)[:, :I], v


def _act64(z, act):
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    # 0.5 (1 + tanh y) = sigmoid(2 y)
    y2 = 2.0 * np.sqrt(2.0 / np.pi) * (z + 0.044715 * z ** 3)
    s = torch.sigmoid(y2)
    return z * s, s + z * s * torch.sigmoid(-y2) * 2.0 * np.sqrt(2.0 / np.pi) * (
        1.0 + 3.0 * 0.044715 * z ** 2)


def _scale_grad64(dy, x, v):
    O, G, _ = v.shape
    dw = torch.nn.functional.pad(dy.t().contiguous() @ x, (0, G * 64 - x.shape[1]))
    return torch.mul(dw.view(O, G, 64), v).sum(2)


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind in ("ffn", "tune"):
        x = st["X"].double()
        wg, vg = _dense64(st["gate"], case["D"])
        wu, vu = _dense64(st["up"], case["D"])
        g, u = x @ wg.t(), x @ wu.t()
        a, da = _act64(g, case["act"])
        if kind == "ffn":
            return a * u
        dh = st["dH"].double()
        dg, du = u * dh * da, a * dh
        return {"h": a * u, "dx": torch.addmm(dg @ wg, du, wu),
                "dgate_scales": _scale_grad64(dg, x, vg),
                "dup_scales": _scale_grad64(du, x, vu)}
    if kind == "linear":
        w, v = _dense64(st["w"], case["D"])
        dy = st["dY"].double()
        return {"dx": dy @ w, "dscales": _scale_grad64(dy, st["X"].double(), v)}
    tau, T = case["tau"], case["T"]
    z = st["logits"].double() / tau
    lse = torch.logsumexp(z, 1)
    live = st["idx"] >= 0
    t = (st["tlogits"].double() / tau).masked_fill(~live, -math.inf)
    p = torch.softmax(t, 1).nan_to_num(0.0)  # a row without entries has no mass
    at = st["idx"].long().clamp(min=0)
    lt = torch.log_softmax(t, 1).masked_fill(~live, 0.0)
    loss = tau * tau * (p * (lt - torch.gather(z, 1, at) + lse[:, None])).sum(1)
    dz = torch.exp(z - lse[:, None]) * live.any(1)[:, None]
    row = torch.arange(T, device=dz.device)[:, None].expand_as(at)
    dz.index_put_((row.reshape(-1), at.reshape(-1)), -p.reshape(-1), accumulate=True)
    return {"loss": loss, "lse": lse, "dlogits": dz * (tau * st["gloss"].double())[:, None]}
