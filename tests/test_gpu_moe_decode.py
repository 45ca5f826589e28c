"""The expert layer for a few tokens on the GPU against its 64-bit definition,
within bounds derived from its roundings."""
import math

import pytest
import torch

import dequant_matmul_int3_amd as qt
from tests.gpu_util import DEV, say
from tests.tune_util import SUM, act64, dense, half_step, quantized, worst

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def experts(E, O, I, bits, seed):
    """((packed [E, bytes], scales [E, O, G], bits), [dense f64 per expert])."""
    w, v = quantized(E * O, I, bits, seed)
    s = w[1].view(E, O, -1).contiguous()
    m = dense(w, v, I).view(E, O, I)
    return (w[0].view(E, -1), s, bits), m


def reference(X, logits, k, g, u, d, act, dtype):
    """out in 64 bits, and the bound of the kernel's error: group sums in f32
    (SUM of the terms' magnitudes, as the multiply kernels), h in two pieces of
    bf16 (2^-17) or exactly, f32 routing weights (exp and a quotient: 2^-21)."""
    T, E = logits.shape
    out = torch.zeros(T, X.shape[1], dtype=torch.float64, device=DEV)
    bound = torch.zeros_like(out)
    x = X.double()
    for t in range(T):
        lg = logits[t].double().tolist()
        top = sorted(range(E), key=lambda e: (-lg[e], e))[:k]
        w = torch.softmax(torch.tensor([lg[e] for e in top], dtype=torch.float64), 0).tolist()
        for p, e in zip(w, top):
            if p == 0.0:
                continue
            zg, zu = g[e] @ x[t], u[e] @ x[t]
            bg, bu = SUM * (g[e].abs() @ x[t].abs()), SUM * (u[e].abs() @ x[t].abs())
            a, _ = act64(zg, act)
            h = a * zu
            bh = (1.13 * bg + 1e-6 * a.abs()) * (zu.abs() + bu) + a.abs() * bu
            bh = bh + (2.0 ** -17 if dtype == torch.bfloat16 else 0.0) * (h.abs() + bh)
            out[t] += p * (d[e] @ h)
            mag = d[e].abs() @ h.abs()
            bound[t] += p * (d[e].abs() @ bh + (SUM + 2.0 ** -21 + k * 2.0 ** -23) * mag)
    return out, bound + half_step(dtype) * (out.abs() + bound) + 1e-30


CASES = [  # T, E, k, D, F
    (1, 4, 2, 128, 64), (1, 128, 8, 512, 256), (2, 7, 7, 64, 64), (16, 8, 2, 256, 128),
    (16, 2, 2, 200, 70), (5, 60, 4, 1000, 333), (9, 130, 3, 65, 1), (3, 512, 32, 1, 65),
    (13, 1, 1, 2100, 40), (8, 16, 1, 640, 320), (4, 300, 6, 330, 450),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits,act", [((3, 3, 3), "silu"), ((4, 3, 4), "gelu"), ((3, 4, 3), "silu"),
                                      ((4, 4, 4), "silu")])
@pytest.mark.parametrize("T,E,k,D,F", CASES)
def test_against_definition(T, E, k, D, F, bits, act, dtype):
    say(f"moe T={T} E={E} k={k} D={D} F={F} {bits} {act} {dtype}")
    gen = torch.Generator(device=DEV).manual_seed(T * 100 + E)
    gate, g = experts(E, F, D, bits[0], 1)
    up, u = experts(E, F, D, bits[1], 2)
    down, d = experts(E, D, F, bits[2], 3)
    X = torch.randn((T, D), generator=gen, device=DEV).to(DT[dtype])
    logits = torch.randn((T, E), generator=gen, device=DEV)
    out = qt.qt_moe_decode(X, logits, k, gate, up, down, act=act)
    ref, bound = reference(X, logits, k, g, u, d, act, DT[dtype])
    assert worst(out, ref, bound) <= 1
    assert torch.equal(out, qt.qt_moe_decode(X, logits, k, gate, up, down, act=act))


def small(T=6, E=12, k=3, D=256, F=192, dtype=torch.float32, bits=(3, 4, 3), seed=5):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    w = [experts(E, *s, b, i) for i, (s, b) in
         enumerate(zip(((F, D), (F, D), (D, F)), bits))]
    X = torch.randn((T, D), generator=gen, device=DEV).to(dtype)
    logits = torch.randn((T, E), generator=gen, device=DEV)
    return X, logits, k, [m for m, _ in w], [v for _, v in w]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_and_masked_logits(dtype):
    """Equal logits (of either zero) take the lower expert first; -inf has no
    weight; every token may choose the same experts."""
    X, logits, k, w, v = small(T=16, dtype=DT[dtype])
    logits[0] = 0.0
    logits[1, ::2], logits[1, 1::2] = -0.0, 0.0
    logits[2, 4:] = -math.inf
    logits[3, 1:] = -math.inf
    logits[4] = torch.finfo(torch.float32).min
    logits[4, 7] = 1.0
    logits[5:] = logits[5]
    out = qt.qt_moe_decode(X, logits, k, *w)
    ref, bound = reference(X, logits, k, *v, "silu", DT[dtype])
    assert worst(out, ref, bound) <= 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_do_not_mix(dtype):
    """A token whose inputs overflow or are not numbers leaves the others as they are."""
    X, logits, k, w, _ = small(T=7, E=5, dtype=DT[dtype])
    out = qt.qt_moe_decode(X, logits, k, *w)
    Y = X.clone()
    Y[2], Y[5, 3] = math.inf, math.nan
    got = qt.qt_moe_decode(Y, logits, k, *w)
    keep = [0, 1, 3, 4, 6]
    assert torch.equal(got[keep], out[keep])
    assert not got[2].isfinite().any() and got[5].isnan().any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_streams(dtype):
    """Enough weights and tokens for the full layer's launches: the same
    definition, with equal and masked logits among them, from a workspace of the
    exact size full of NaN; rows at odd addresses and GELU keep the two launches."""
    T, E, k, D, F = 16, 64, 8, 1024, 1536
    X, logits, k, w, v = small(T, E, k, D, F, DT[dtype])
    logits[0] = 0.0
    logits[1, ::2], logits[1, 1::2] = -0.0, 0.0
    logits[2, 9:] = -math.inf
    logits[5:8] = logits[5]
    need = qt.qt_moe_decode_workspace_bytes(T, k, E, D, F, qt.QT_BF16 if dtype == "bf16" else qt.QT_F32)
    assert need >= qt.qt_moe_layer_workspace_bytes(T, k, E, D, F)
    ws = torch.full((need // 4 + 8,), math.nan, device=DEV)
    out = qt.qt_moe_decode(X, logits, k, *w, workspace=ws[4:4 + need // 4])
    assert ws[:4].isnan().all() and ws[4 + need // 4:].isnan().all()
    ref, bound = reference(X, logits, k, *v, "silu", DT[dtype])
    assert worst(out, ref, bound) <= 1
    assert torch.equal(out, qt.qt_moe_decode(X, logits, k, *w))
    if dtype == "f32":
        assert torch.equal(out, qt.qt_moe_layer(X, logits, k, *w))
    room = torch.empty(X.numel() + 1, dtype=X.dtype, device=DEV)
    Xu = room[1:].view(X.shape)
    Xu.copy_(X)
    assert worst(qt.qt_moe_decode(Xu, logits, k, *w), ref, bound) <= 1
    ref, bound = reference(X, logits, k, *v, "gelu", DT[dtype])
    assert worst(qt.qt_moe_decode(X, logits, k, *w, act="gelu"), ref, bound) <= 1
    Y = X.clone()
    Y[2], Y[5, 3] = math.inf, math.nan
    got = qt.qt_moe_decode(Y, logits, k, *w)
    keep = [t for t in range(T) if t not in (2, 5)]
    assert torch.equal(got[keep], out[keep])
    assert not got[2].isfinite().any() and got[5].isnan().any()


def test_agrees_with_the_layer_of_five_launches():
    X, logits, k, w, _ = small(T=9, E=20, k=4, D=256, F=128)
    a = qt.qt_moe_decode(X, logits, k, *w)
    b = qt.qt_moe_layer(X, logits, k, *w)
    assert float((a - b).norm() / b.norm()) < 2e-6


def test_unaligned_rows():
    """Rows at their elements' alignment only."""
    for dtype in (torch.bfloat16, torch.float32):
        X, logits, k, w, _ = small(D=256, dtype=dtype)
        ref = qt.qt_moe_decode(X, logits, k, *w)
        room = torch.empty(X.numel() + 1, dtype=dtype, device=DEV)
        room2 = torch.full((X.numel() + 2,), math.nan, dtype=dtype, device=DEV)
        Xu = room[1:].view(X.shape)
        Xu.copy_(X)
        out = room2[1:-1].view(X.shape)
        qt.qt_moe_decode(Xu, logits, k, *w, out=out)
        assert torch.equal(out, ref) and room2[0].isnan() and room2[-1].isnan()


def test_workspace_of_the_size_asked_for():
    X, logits, k, w, _ = small()
    ref = qt.qt_moe_decode(X, logits, k, *w)
    need = qt.qt_moe_decode_workspace_bytes(6, k, 12, 256, 192, qt.QT_F32)
    assert need % 4 == 0
    pad = torch.full((need // 4 + 64,), math.nan, device=DEV)
    ws = pad[32:32 + need // 4]
    assert torch.equal(qt.qt_moe_decode(X, logits, k, *w, workspace=ws), ref)
    assert pad[:32].isnan().all() and pad[32 + need // 4:].isnan().all()
    with pytest.raises(qt.QtError, match="workspace"):
        qt.qt_moe_decode(X, logits, k, *w, workspace=ws[:-4])
    with pytest.raises(qt.QtError):
        qt.qt_moe_decode(X[:1].expand(17, 256).contiguous(),
                         logits[:1].expand(17, 12).contiguous(), k, *w)


def test_captured_and_replayed():
    X, logits, k, w, v = small(dtype=torch.bfloat16)
    Xs, ls, out = X.clone(), logits.clone(), torch.empty_like(X)
    qt.qt_moe_decode(Xs, ls, k, *w, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qt.qt_moe_decode(Xs, ls, k, *w, out=out)
    for i in range(4):
        Xs.copy_(X.roll(i, 0) * (i + 1))
        ls.copy_(logits.roll(i, 1))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, qt.qt_moe_decode(Xs, ls, k, *w))


def test_two_streams_at_once():
    calls = [small(T=t, seed=t, dtype=torch.bfloat16) for t in (1, 16)]
    ref = [qt.qt_moe_decode(X, lg, k, *w) for X, lg, k, w, _ in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        outs = [qt.qt_moe_decode(X, lg, k, *w, stream=s)
                for (X, lg, k, w, _), s in zip(calls, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))
