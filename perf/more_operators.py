"""The operators of a decode step, as cases to measure.

Three paths of a program that serves a network whose weights and key-value
cache are group-scaled integers:

* `fill`  a chunk of a prompt: its keys and values are quantized into the pages
          of the cache, then the context so far is read back for the chunk's
          own attention;
* `step`  one new token per sequence: its key and value are quantized into the
          cache, then its query attends over the sequence's pages;
* `moe`   the expert layer for a few tokens.

The plain forms below are elementary torch operations in 32 bits (in 64 where a
quotient is rounded to a code).
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 64


# --------------------------------------------------------------------- cases
def _fill(name, T, ctx, heads, dim, page, kbits, vbits, dtype):
    return {"name": name, "kind": "fill", "T": T, "ctx": ctx, "heads": heads, "dim": dim,
            "page": page, "kbits": kbits, "vbits": vbits, "dtype": dtype}


def _step(name, B, ctx, ragged, heads, per, dim, page, kbits, vbits, window, dtype):
    return {"name": name, "kind": "step", "B": B, "ctx": ctx, "ragged": ragged, "heads": heads,
            "per": per, "dim": dim, "page": page, "kbits": kbits, "vbits": vbits,
            "window": window, "dtype": dtype}


def _moe(name, T, E, k, D, F, bits, act, dtype):
    return {"name": name, "kind": "moe", "T": T, "E": E, "k": k, "D": D, "F": F, "gate_bits": bits[0],
            "up_bits": bits[1], "down_bits": bits[2], "act": act, "dtype": dtype}


def listed():
    return [
        # a short turn of a chat appended to a short context: f32, a short last group
        _fill("fill-turn", 37, 301, 2, 80, 16, 8, 8, "f32"),
        # a chunk of a long prompt, keys at 8 bits and values at 4
        _fill("fill-chunk", 4096, 16384, 8, 128, 64, 8, 4, "bf16"),
        # one user, a short context: the latency of a step
        _step("step-1-short", 1, 700, False, 8, 4, 128, 16, 8, 8, 0, "bf16"),
        # one user, a long document: one sequence has to fill the card
        _step("step-1-long", 1, 131072, False, 8, 8, 128, 64, 4, 4, 0, "bf16"),
        # a batch of users at every stage of their contexts, some slots empty
        _step("step-batch", 64, 8192, True, 8, 4, 128, 64, 8, 4, 0, "bf16"),
        # one key-value head for 24 wide query heads
        _step("step-one-head", 24, 12000, True, 1, 24, 256, 128, 8, 8, 0, "bf16"),
        # f32, a key-value head per query head, odd width, a sliding window, pages of 48
        _step("step-window-f32", 5, 6001, True, 12, 1, 100, 48, 4, 8, 1500, "f32"),
        # one token through the expert layer
        _moe("moe-1", 1, 128, 8, 7168, 2048, (3, 3, 3), "silu", "bf16"),
        # the same from f32 inputs, up projection at other bits
        _moe("moe-1-f32", 1, 128, 8, 7168, 2048, (4, 3, 4), "silu", "f32"),
        # a small batch: most pairs have an expert of their own
        _moe("moe-12", 12, 128, 8, 7168, 2048, (3, 3, 3), "silu", "bf16"),
        # small ragged experts in f32: short last groups on both sides
        _moe("moe-5-ragged", 5, 60, 4, 1000, 333, (4, 4, 3), "gelu", "f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("fill", "step", "step", "step", "moe", "moe"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if kind == "moe":
        T, E = _log(rng, 1, 16), _log(rng, 4, 256)
        k = min(E, rng.choice((1, 2, 4, 6, 8)))
        D = _log(rng, 128, 7168)
        F = _log(rng, 64, 2048)
        if rng.random() < 0.6:
            D, F = max(128, D // 64 * 64), max(64, F // 64 * 64)
        # as many expert weights as the largest listed case has at most
        T = max(1, min(T, 12 * 8 * 7168 * 2048 // (k * D * F)))
        E = max(k, min(E, 128 * 7168 * 2048 // (D * F)))
        return {"kind": kind, "T": T, "E": E, "k": k, "D": D, "F": F,
                "gate_bits": rng.choice((3, 4)), "up_bits": rng.choice((3, 4)),
                "down_bits": rng.choice((3, 4)), "act": rng.choice(("silu", "silu", "gelu")),
                "dtype": dtype}
    case = {"kind": kind, "heads": _log(rng, 1, 16),
            "dim": rng.choice((64, 80, 96, 128, 128, 192, 256, _log(rng, 16, 256))),
            "page": 16 * _log(rng, 1, 16), "kbits": rng.choice((4, 8)), "vbits": rng.choice((4, 8)),
            "dtype": dtype}
    wide = case["heads"] * -(-case["dim"] // GROUP) * GROUP
    if kind == "fill":
        case["ctx"] = min(_log(rng, 1, 32768), 16384 * 1024 // wide)
        case["T"] = _log(rng, 1, case["ctx"])
        return case
    case["ctx"] = min(_log(rng, 1, 131072), 131072 * 1024 // wide)
    case["B"] = min(_log(rng, 1, 128), max(1, 32 * 8192 * 1024 // (wide * case["ctx"])))
    case["ragged"] = case["B"] > 1 and rng.random() < 0.7
    case["per"] = rng.choice((1, 2, 4, 5, 8, 16, 24))
    case["window"] = rng.choice((0, 0, 0, _log(rng, 1, case["ctx"])))
    return case


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
    q = u.view(O, G, 16, 4)
    lo = (q[..., 0] & 3) | (q[..., 1] & 3) << 2 | (q[..., 2] & 3) << 4 | (q[..., 3] & 3) << 6
    h = (u >> 2).view(O, G, 8, 8)
    hi = h[..., 0] | h[..., 1] << 1 | h[..., 2] << 2 | h[..., 3] << 3
    hi = hi | h[..., 4] << 4 | h[..., 5] << 5 | h[..., 6] << 6 | h[..., 7] << 7
    return torch.cat([lo, hi], -1).to(torch.uint8).reshape(-1)


def _experts(gen, E, O, I, bits):
    """E quantized matrices [O x I]: N(0, 0.02) weights with 0.5 % outliers of
    N(0, 0.5), rounded to the group's absmax scale -> (packed [E, bytes],
    scales [E, O, G], bits)."""
    G = -(-I // GROUP)
    half = 4 if bits == 3 else 8
    packed = torch.empty((E, O * G * (24 if bits == 3 else 32)), dtype=torch.uint8, device=DEV)
    scales = torch.empty((E, O, G), dtype=torch.float32, device=DEV)
    for e in range(E):
        w = torch.randn((O, I), generator=gen, device=DEV) * 0.02
        w = torch.where(torch.rand((O, I), generator=gen, device=DEV) < 0.005, w * 25.0, w)
        w = torch.nn.functional.pad(w, (0, G * GROUP - I)).view(O, G, GROUP)
        s = w.abs().amax(-1) / half
        q = torch.round(w / torch.where(s > 0, s, torch.ones_like(s))[..., None])
        packed[e] = _pack(q.clamp(-half, half - 1).to(torch.int32), bits)
        scales[e] = s
    return packed, scales, bits


def _lengths(case, gen):
    """Tokens of each sequence, the new one included: spread evenly up to ctx,
    the first one whole; every ninth slot of a ragged batch is empty."""
    B, ctx = case["B"], case["ctx"]
    if not case["ragged"]:
        return torch.full((B,), ctx, dtype=torch.int32, device=DEV)
    n = [0 if b % 9 == 8 else ctx - (b * ctx) // B for b in range(B)]
    at = torch.randperm(B, generator=gen, device=DEV)
    return torch.tensor(n, dtype=torch.int32, device=DEV)[at]


def _cache(case, gen, pages):
    """Pages holding quantized normal keys and values -> (k, v), each
    (codes [pages, heads, page, bytes], scales [pages, heads, page, G], bits)."""
    H, d, P = case["heads"], case["dim"], case["page"]
    G = -(-d // GROUP)
    both = []
    # keys have some large channels, as keys do
    loud = 1.0 + 7.0 * (torch.rand((H, 1, d), generator=gen, device=DEV) < 0.03)
    for bits, std in ((case["kbits"], loud), (case["vbits"], torch.ones_like(loud))):
        codes = torch.empty((pages, H, P, G * 8 * bits), dtype=torch.uint8, device=DEV)
        scales = torch.empty((pages, H, P, G), dtype=torch.float32, device=DEV)
        some = max(1, (1 << 25) // (H * P * G * GROUP))
        for p in range(0, pages, some):
            x = torch.randn((min(some, pages - p), H, P, d), generator=gen, device=DEV) * std
            c, s = _quantize(x.to(_dt(case["dtype"])), bits)
            scales[p:p + some] = s
            codes[p:p + some] = _octets(c, bits) if both else _rows(c, bits)
        both.append((codes, scales, bits))
    return both[0], both[1]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed * 7919 + 23)
    st = {"case": case}
    dt = _dt(case["dtype"])

    def normal(shape, std=1.0):
        return (torch.randn(shape, generator=gen, device=DEV) * std).to(dt)

    if case["kind"] == "moe":
        T, E, D, F = case["T"], case["E"], case["D"], case["F"]
        st["gate"] = _experts(gen, E, F, D, case["gate_bits"])
        st["up"] = _experts(gen, E, F, D, case["up_bits"])
        st["down"] = _experts(gen, E, D, F, case["down_bits"])
        st["X"] = normal((T, D))
        st["logits"] = torch.randn((T, E), generator=gen, device=DEV)
        return st
    H, d, P, ctx = case["heads"], case["dim"], case["page"], case["ctx"]
    B = case["B"] if case["kind"] == "step" else 1
    wide = -(-ctx // P)  # pages of the longest sequence
    st["k"], st["v"] = _cache(case, gen, B * wide + 3)
    table = torch.randperm(B * wide + 3, generator=gen, device=DEV)[:B * wide].view(B, wide).int()
    if case["kind"] == "step":
        st["lens"] = _lengths(case, gen)
        last = (st["lens"].long() - 1)[:, None]
        page = table.long().gather(1, last.clamp(min=0) // P)
        slot = torch.where(last < 0, torch.full_like(last, -1), page * P + last % P)[:, 0]
        Hq = H * case["per"]
        # one projection's output: queries, keys and values of a token side by side
        rows = normal((B, (Hq + 2 * H) * d))
        st["Q"] = rows[:, :Hq * d].view(B, Hq, d)
        st["K"] = rows[:, Hq * d:(Hq + H) * d].view(B, H, d)
        st["V"] = rows[:, (Hq + H) * d:].view(B, H, d)
        st["table"] = table
    else:
        T = case["T"]
        slot = table[0].long()[:, None] * P + torch.arange(P, device=DEV)
        slot = slot.reshape(-1)[:ctx]
        st["read"] = slot.int()
        slot = slot[ctx - T:].clone()
        slot[torch.rand((T,), generator=gen, device=DEV) < 0.01] = -1  # padding
        rows = normal((T, 2 * H * d))
        st["K"], st["V"] = rows[:, :H * d].view(T, H, d), rows[:, H * d:].view(T, H, d)
    st["slots"] = slot.int().contiguous()
    return st


# --------------------------------------------------------------- plain forms
def _quantize(x, bits):
    """x [..., d] -> codes [..., G * 64] (0 past d) as int32, scales [..., G] f32:
    the value of largest magnitude takes the code -8 or -128 exactly."""
    d = x.shape[-1]
    G, half = -(-d // GROUP), 1 << (bits - 1)
    x = torch.nn.functional.pad(x.float(), (0, G * GROUP - d)).view(*x.shape[:-1], G, GROUP)
    top = x.gather(-1, x.abs().argmax(-1, keepdim=True))
    s = top * (-1.0 / half)
    q = x.double() / torch.where(s != 0, s, torch.ones_like(s)).double()
    q = torch.round(q).clamp(-half, half - 1).to(torch.int32)
    return q.view(*q.shape[:-2], G * GROUP), s[..., 0]


def _rows(c, bits):
    """Codes [..., n] -> bytes [..., n * bits / 8], value after value."""
    u = c + (1 << (bits - 1))
    if bits == 8:
        return u.to(torch.uint8)
    u = u.view(*u.shape[:-1], -1, 2)
    return (u[..., 0] | u[..., 1] << 4).to(torch.uint8)


def _unrows(b, bits):
    b = b.to(torch.int32)
    if bits == 4:
        b = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    return b - (1 << (bits - 1))


def _blocks(codes, bits):
    """A view of a page's bytes as blocks of eight tokens, [pages, H, block, pair of tokens, token
    of the pair, group, 4 values of the group, byte]."""
    n, H, P, w = codes.shape
    shape = (n, H, P // 8, w * 8 // (bits * GROUP), 16, 4)
    if bits == 8:
        return codes.view(*shape, 2, 4).permute(0, 1, 2, 5, 6, 3, 4, 7)
    return codes.view(*shape, 2, 2).permute(0, 1, 2, 5, 7, 3, 4, 6)  # a pair's bytes alternate


def _octets(c, bits):
    """Codes [pages, H, P, 64 G] -> the pages' bytes [pages, H, P, 8 bits G] in blocks."""
    n, H, P, w = c.shape
    codes = torch.empty((n, H, P, w * bits // 8), dtype=torch.uint8, device=c.device)
    _blocks(codes, bits).copy_(_rows(c.view(n, H, P // 8, 4, 2, w // GROUP, 16, 4), bits))
    return codes


def _unoctets(b, bits):
    n, H, P, _ = b.shape
    return _unrows(_blocks(b, bits).reshape(n, H, P, -1), bits)


def _plain_write(st):
    slots = st["slots"].long()
    live = slots >= 0
    slots = slots[live]
    for (codes, scales, bits), new, octets in ((st["k"], st["K"], False), (st["v"], st["V"], True)):
        P = codes.shape[2]
        at, t = slots // P, slots % P
        c, s = _quantize(new[live], bits)
        scales[at, :, t] = s
        b = _rows(c, bits)
        if octets:
            _blocks(codes, bits)[at, :, t // 8, t // 2 % 4, t % 2] = b.view(
                *b.shape[:2], -1, 16, bits // 2)
        else:
            codes[at, :, t] = b


def _values(part, pages, octets, d):
    """The named pages' values [n, H, P, d] in f32."""
    codes, scales, bits = part
    c = (_unoctets if octets else _unrows)(codes[pages], bits).float()
    s = scales[pages]
    return (c.view(*s.shape, GROUP) * s[..., None]).flatten(-2)[..., :d]


def _plain_read(st):
    case, slots = st["case"], st["read"].long()
    P = case["page"]
    pages, at = torch.unique_consecutive(slots // P, return_inverse=True)
    return [_values(st[n], pages, o, case["dim"])[at, :, slots % P].to(st["K"].dtype)
            for n, o in (("k", False), ("v", True))]


def _seen(st, L):
    """Which of L positions each sequence attends to, [B, L]."""
    t, n, w = torch.arange(L, device=DEV)[None, :], st["lens"][:, None], st["case"]["window"]
    seen = t < n
    return seen & (t >= n - w) if w else seen


def _plain_attend(st):
    case = st["case"]
    B, H, per, d, P = case["B"], case["heads"], case["per"], case["dim"], case["page"]
    L = st["table"].shape[1] * P
    pages = st["table"].long().reshape(-1)

    def gathered(part, octets):
        x = _values(part, pages, octets, d).view(B, -1, H, P, d)
        return x.transpose(1, 2).reshape(B, H, L, d)

    seen = _seen(st, L)[:, None, None, :]
    q = st["Q"].float().view(B, H, per, d)
    s = q @ gathered(st["k"], False).transpose(2, 3) * (1.0 / math.sqrt(d))
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(s - m)
    z = e.sum(-1, keepdim=True)
    # values of positions that are not seen do not count, whatever they are
    v = torch.where(seen.transpose(2, 3), gathered(st["v"], True), torch.zeros((), device=DEV))
    out = (e @ v) / torch.where(z > 0, z, torch.ones_like(z))
    return {"out": out.reshape(B, H * per, d).to(st["Q"].dtype),
            "lse": (m + torch.log(z)).reshape(B, H * per)}


def _codes(packed, scales, bits):
    """Packed bytes -> codes [..., G, 64] as f32."""
    b = packed.view(*scales.shape, -1).to(torch.int32)
    if bits == 4:
        return (torch.stack([b & 15, b >> 4], -1).flatten(-2) - 8).float()
    two = torch.arange(0, 8, 2, device=b.device, dtype=torch.int32)
    one = torch.arange(0, 8, 1, device=b.device, dtype=torch.int32)
    lo = ((b[..., :16, None] >> two) & 3).flatten(-2)
    hi = ((b[..., 16:, None] >> one) & 1).flatten(-2)
    return (lo + 4 * hi - 4).float()


def _product(w, e, x):
    """W_e[p] x[p] for every pair p."""
    packed, scales, bits = w
    s = scales[e]
    m = (_codes(packed[e], s, bits) * s[..., None]).flatten(-2)[..., :x.shape[1]]
    return (m @ x[..., None])[..., 0]


def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))


def _plain_moe(st):
    case = st["case"]
    T, k = case["T"], case["k"]
    top, e = torch.sort(st["logits"], dim=1, descending=True, stable=True)
    top, e = top[:, :k], e[:, :k].reshape(-1)
    w = torch.exp(top - top[:, :1])
    w = w / w.sum(1, keepdim=True)
    x = st["X"].float().repeat_interleave(k, 0)
    h = _act(_product(st["gate"], e, x), case["act"]) * _product(st["up"], e, x)
    y = _product(st["down"], e, h).view(T, k, -1)
    return (y * w[..., None]).sum(1).to(st["X"].dtype)


def run(state):
    case = state["case"]
    kind = case["kind"]
    if own:
        import dequant_matmul_int3_amd as qt
        if kind == "moe":
            return qt.qt_moe_decode(state["X"], state["logits"], case["k"], state["gate"],
                                    state["up"], state["down"], act=case["act"])
        qt.qt_kv_write(state["K"], state["V"], state["slots"], state["k"], state["v"])
        if kind == "fill":
            k, v = qt.qt_kv_read(state["read"], state["k"], state["v"], case["dim"],
                                 dtype=state["K"].dtype)
            return {"k": k, "v": v}
        out, lse = qt.qt_attn_decode(state["Q"], state["k"], state["v"], state["table"],
                                     state["lens"], window=case["window"], want_lse=True)
        return {"out": out, "lse": lse}
    if kind == "moe":
        return _plain_moe(state)
    _plain_write(state)
    if kind == "fill":
        k, v = _plain_read(state)
        return {"k": k, "v": v}
    return _plain_attend(state)


# ------------------------------------------------------------ work and truth
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "moe":
        T, E, k, D, F = (case[n] for n in ("T", "E", "k", "D", "F"))

        def rows(O, I, bits):
            return O * -(-I // GROUP) * ((24 if bits == 3 else 32) + 4)

        # an expert is some token's with probability 1 - (1 - k/E)^T
        live = E * (1.0 - (1.0 - k / E) ** T)
        w = rows(F, D, case["gate_bits"]) + rows(F, D, case["up_bits"]) + rows(D, F, case["down_bits"])
        return {"bytes": int(live * w) + T * (2 * D * e + E * 4), "flops": 6 * T * k * D * F}
    H, d = case["heads"], case["dim"]
    token = H * -(-d // GROUP) * (8 * (case["kbits"] + case["vbits"]) + 8)
    if case["kind"] == "fill":
        T, R = case["T"], case["ctx"]
        return {"bytes": 2 * (T + R) * H * d * e + (T + R) * token, "flops": (4 * T + 2 * R) * H * d}
    B, Hq, ctx = case["B"], H * case["per"], case["ctx"]
    n = [ctx] * B
    if case["ragged"]:
        n = [0 if b % 9 == 8 else ctx - (b * ctx) // B for b in range(B)]
    seen = sum(min(x, case["window"] or x) for x in n)
    return {"bytes": B * (2 * Hq * d * e + 2 * H * d * e + Hq * 4 + token) + seen * token,
            "flops": 4 * seen * Hq * d}


def _dense64(w, e, n):
    """Expert e's matrix from the format's words alone, in 64 bits."""
    packed, scales, bits = w
    b, s = packed[e], scales[e].double()
    b = b.view(*s.shape, -1)
    j = torch.arange(64, device=b.device)
    if bits == 4:
        v = ((b[..., j // 2] >> (4 * (j % 2)).to(torch.uint8)) & 15).to(torch.int16) - 8
    else:
        lo = (b[..., j // 4] >> (2 * (j % 4)).to(torch.uint8)) & 3
        hi = (b[..., 16 + j // 8] >> (j % 8).to(torch.uint8)) & 1
        v = (lo | hi << 2).to(torch.int16) - 4
    return torch.mul(v.double(), s[..., None]).reshape(s.shape[0], -1)[:, :n]


def _act64(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    return z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))


def _nearest64(x, bits):
    """The values that x [T, H, d] is held as, in 64 bits."""
    T, H, d = x.shape
    half = 2 ** (bits - 1)
    out = torch.empty((T, H, d), dtype=torch.float64, device=x.device)
    for g in range(0, d, GROUP):
        y = x[..., g:g + GROUP].double()
        hi, lo = y.amax(-1, keepdim=True), y.amin(-1, keepdim=True)
        # of two values of one magnitude and different signs the first one counts
        first_hi, first_lo = y.argmax(-1, keepdim=True), y.argmin(-1, keepdim=True)
        up = (hi > -lo) | ((hi == -lo) & (first_hi < first_lo))
        s = torch.where(up, hi, lo) / -half
        v = torch.where(s == 0, torch.zeros_like(y), y / s).round().clamp(-half, half - 1)
        out[..., g:g + GROUP] = v * s
    return out


def _held64(part, octets, page, t, d):
    """Values of the tokens t of the pages named (two index arrays of one shape) in 64 bits,
    byte by byte from the layout: [..., H, d]."""
    codes, scales, bits = part
    n, H, P, w = codes.shape
    G, W = scales.shape[3], bits // 2
    j = torch.arange(d, device=codes.device)
    if octets:
        # the byte of value j of token t, counted from the page's first
        t = t[..., None]
        byte = (t // 8 * G * 16 + j // 64 * 16 + j % 64 // 4) * 8 * W
        byte = byte + (t % 8 * 4 + j % 4 if bits == 8 else t % 8 // 2 * 4 + j % 4 // 2 * 2 + t % 2)
        t = t[..., 0]
    else:
        byte = t[..., None] * w + j * bits // 8
    b = codes.view(n, H, P * w)[page[..., None, None], torch.arange(H, device=codes.device)[:, None],
                                byte[..., None, :]]
    if bits == 4:
        b = (b >> (4 * (j % 2)).to(torch.uint8)) & 15
    s = scales[page, :, t].double()
    return (b.to(torch.int16) - 2 ** (bits - 1)).double() * s[..., j // 64]


def exact(case, seed):
    st = prepare(case, seed)
    kind = case["kind"]
    if kind == "moe":
        T, k, D, F = case["T"], case["k"], case["D"], case["F"]
        out = torch.zeros((T, D), dtype=torch.float64, device=DEV)
        logits = st["logits"].double().cpu()
        x = st["X"].double()
        users = {}
        for t in range(T):
            best = sorted(range(case["E"]), key=lambda e: (-float(logits[t, e]), e))[:k]
            w = torch.softmax(logits[t, best], 0)
            for e, p in zip(best, w.tolist()):
                users.setdefault(e, []).append((t, p))
        for e, who in users.items():
            t = torch.tensor([a for a, _ in who], device=DEV)
            p = torch.tensor([b for _, b in who], dtype=torch.float64, device=DEV)
            xe = x[t]
            h = _act64(xe @ _dense64(st["gate"], e, D).t(), case["act"])
            h = h * (xe @ _dense64(st["up"], e, D).t())
            out.index_add_(0, t, (h @ _dense64(st["down"], e, F).t()) * p[:, None])
        return out
    H, d, P = case["heads"], case["dim"], case["page"]
    slots = st["slots"].long()
    new = [_nearest64(st[n], st[m][2]) for n, m in (("K", "k"), ("V", "v"))]
    if kind == "fill":
        read = st["read"].long()
        got = [_held64(st[m], o, read // P, read % P, d) for m, o in (("k", False), ("v", True))]
        T = case["T"]
        wrote = (slots >= 0)[:, None, None]
        for g, x in zip(got, new):
            g[-T:] = torch.where(wrote, x, g[-T:])
        return {"k": got[0], "v": got[1]}
    B, per = case["B"], case["per"]
    out = torch.zeros((B, H, per, d), dtype=torch.float64, device=DEV)
    lse = torch.full((B, H, per), -math.inf, dtype=torch.float64, device=DEV)
    q = st["Q"].double().view(B, H, per, d)
    for b, n in enumerate(st["lens"].tolist()):
        if n == 0:
            continue
        pos = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device=DEV)
        page = st["table"][b].long()[pos // P]
        k, v = (_held64(st[m], o, page, pos % P, d) for m, o in (("k", False), ("v", True)))
        k[-1], v[-1] = new[0][b], new[1][b]
        s = q[b] @ k.permute(1, 2, 0).contiguous() / math.sqrt(d)
        out[b] = torch.softmax(s, -1) @ v.transpose(0, 1).contiguous()
        lse[b] = torch.logsumexp(s, -1)
    return {"out": out.view(B, H * per, d), "lse": lse.view(B, H * per)}
