"""Plain 64-bit forms of the quantized key-value cache, its attention and the
few-token expert layer, and the bounds their tests use (elementary torch
operations on the device the inputs are on)."""
import math

import torch

U = 2.0 ** -24  # half a step of f32 at 1


def groups(d):
    return -(-d // 64)


def quantize(x, bits):
    """x [..., d] -> (codes [..., G, 64] int64, scales [..., G] f32) by the
    definition: quotients in 64 bits, where f32 operands never meet a tie by rounding."""
    d, half = x.shape[-1], 2 ** (bits - 1)
    G = groups(d)
    x = torch.nn.functional.pad(x.float(), (0, 64 * G - d)).view(*x.shape[:-1], G, 64)
    m = torch.zeros_like(x[..., 0])
    for j in range(64):  # the first of equals stays
        m = torch.where(x[..., j].abs() > m.abs(), x[..., j], m)
    s = -m / half
    q = torch.where(s[..., None] == 0, torch.zeros_like(x, dtype=torch.float64),
                    x.double() / s.double()[..., None])
    v = torch.round(q).clamp(-half, half - 1).nan_to_num(0.0).long()
    bad = ~torch.isfinite(x).all(-1)
    return torch.where(bad[..., None], torch.zeros_like(v), v), \
        torch.where(bad, torch.full_like(s, math.nan), s)


def value(codes, scales, d):
    return (codes.double() * scales.double()[..., None]).flatten(-2)[..., :d]


def _places(bits, octets, t, G, device):
    """(byte within its (page, head), shift) of the codes [G, 64] of page tokens t [n]."""
    t = t[:, None, None]
    g = torch.arange(G, device=device)[:, None]
    j = torch.arange(64, device=device)[None, :]
    if not octets:
        row = t * (G * 8 * bits) + g * 8 * bits
        return (row + j, 0 * j) if bits == 8 else (row + j // 2, 4 * (j % 2) + 0 * g)
    block = ((t // 8 * G + g) * 16 + j // 4) * 4 * bits
    if bits == 8:
        return block + 4 * (t % 8) + j % 4, 0 * j
    return block + 4 * (t % 8 // 2) + 2 * (j % 4 // 2) + t % 2, 4 * (j % 2) + 0 * g


def store(part, octets, slots, codes, scales):
    """codes [T, H, G, 64], scales [T, H, G] into the slots [T] >= 0 of a cache
    part, byte by byte."""
    buf, sc, bits = part
    n, H, P, G = sc.shape
    page, t = slots.long() // P, slots.long() % P
    flat = buf.view(n, H, -1)
    byte, shift = _places(bits, octets, t, G, buf.device)
    u = codes + 2 ** (bits - 1)
    sc[page, :, t] = scales
    mask = 2 ** bits - 1
    # the two codes of an int4 byte one after the other
    for par in ((0, 1) if bits == 4 else (0,)):
        sel = slice(par, None, 2) if bits == 4 else slice(None)
        for h in range(H):
            b = byte[..., sel]
            old = flat[page[:, None, None], h, b].long()
            sh = shift[..., sel].expand_as(b)
            new = (old & ~(mask << sh)) | (u[:, h, :, sel] << sh)
            flat[page[:, None, None], h, b] = new.to(torch.uint8)


def fetch(part, octets, slots):
    """(codes [T, H, G, 64], scales [T, H, G]) of slots [T] >= 0."""
    buf, sc, bits = part
    n, H, P, G = sc.shape
    page, t = slots.long() // P, slots.long() % P
    byte, shift = _places(bits, octets, t, G, buf.device)
    flat = buf.view(n, H, -1)
    b = flat[page[:, None, None, None], torch.arange(H, device=buf.device)[None, :, None, None],
             byte[:, None]].long()
    u = (b >> shift) & (2 ** bits - 1)
    return u - 2 ** (bits - 1), sc[page, :, t]


def attend(q, kc, ks, vc, vs, scale, f32, kbits, vbits):
    """One sequence: q [Hq, d], codes [n, H, G, 64], scales [n, H, G] of the
    positions that count -> out [Hq, d], lse [Hq] in 64 bits and bounds of the
    kernel's errors before the rounding of out."""
    Hq, d = q.shape
    n, H, G, _ = kc.shape
    per = Hq // H
    Q = torch.nn.functional.pad(q.double(), (0, 64 * G - d)).view(H, per, 1, G * 64)
    k = value(kc, ks, 64 * G).permute(1, 0, 2)[:, None]  # [H, 1, n, d]
    v = value(vc, vs, 64 * G).permute(1, 0, 2)
    s = scale * (Q * k).sum(-1)  # [H, per, n]
    # the products' sums: 64 exact terms a group and G of them, in any order,
    # each of magnitude |q| (|v| + 16) s where codes are offset by 8 and taken
    # out again, |q v| s elsewhere (f32 inputs in three pieces: three times the
    # additions)
    off = 16.0 if kbits == 4 and not f32 else 0.0
    mag = (kc.double().abs() + off) * ks.double().abs()[..., None]
    mag = mag.flatten(-2).permute(1, 0, 2)[:, None]
    es = U * (3 * 64 + G + 8) * abs(scale) * (Q.abs() * mag).sum(-1)
    es = es + 4 * U * s.abs()
    p = torch.softmax(s, -1)
    out = p @ v[:, :, :] if n else torch.zeros((H, per, 64 * G), dtype=torch.float64, device=q.device)
    lse = torch.logsumexp(s, -1) if n else torch.full((H, per), -math.inf, dtype=torch.float64,
                                                      device=q.device)
    if n == 0:
        return out.view(Hq, -1)[:, :d], lse.view(Hq), torch.zeros(Hq, d, device=q.device).double(), \
            torch.zeros(Hq, device=q.device).double()
    e = es.amax(-1)  # relative error of every probability, and of their sum
    rel = torch.expm1(2 * e) + 16 * U
    offv = 16.0 if vbits == 4 and not f32 else 0.0
    magv = ((vc.double().abs() + offv) * vs.double().abs()[..., None]).flatten(-2).permute(1, 0, 2)
    pm = p @ magv
    pieces = 0.0 if f32 else 2.0 ** -16
    adds = U * (n / 8 + 200)
    bo = (2 * rel + pieces + adds)[..., None] * pm
    bl = e + adds + 8 * U * lse.abs()
    return out.view(Hq, -1)[:, :d], lse.view(Hq), bo.view(Hq, -1)[:, :d], bl.view(Hq)
