"""The expert layer for a few tokens where its roundings show."""
import math

import pytest
import torch

import dequant_matmul_int3_amd as qt
from tests.gpu_util import DEV, say
from tests.serve_util import U
from tests.test_gpu_moe_decode import DT, experts
from tests.tune_util import act64, worst

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits,act", [(3, "silu"), (4, "silu"), (3, "gelu"), (4, "gelu")])
@pytest.mark.parametrize("E", [1, 16])
def test_activations_are_held_exactly(E, bits, act, dtype):
    """One input that is not zero, one feature, one expert a token (alone or shared): an
    output is the product of six numbers.  Besides its own rounding, in U = 2^-24: gate
    and up two each, the activation's last operations sixteen, its product one, three
    pieces scaled and added six, the weight (exp(0) / exp(0), exact) and the sum one:
    less than 32.  The activation is z / (1 + e^-y), y = z or 2 sqrt(2/pi) (z + 0.044715 z^3):
    an error of y counts 1 - sigmoid(y) times, and y errs by six roundings of its own and
    three times the two of z: 12 U |y|."""
    say(f"exact activation E={E} {bits} {act} {dtype}")
    T, D, F = 16, 4096, 1
    gen = torch.Generator(device=DEV).manual_seed(E + bits)
    (gate, g), (up, u), (down, d) = (experts(E, *s, bits, i)
                                     for i, s in enumerate(((F, D), (F, D), (D, F))))
    logits = torch.zeros(T, E, device=DEV)
    at = torch.arange(T, device=DEV) % E
    logits[torch.arange(T, device=DEV), at] = 1.0
    # the input at which the token's gate and up are furthest from zero
    j = (g[at, 0].abs() * u[at, 0].abs()).argmax(-1)
    X = torch.zeros(T, D, device=DEV)
    X[torch.arange(T, device=DEV), j] = 20.0 + 10.0 * torch.rand(T, generator=gen, device=DEV)
    X = X.to(DT[dtype])
    out = qt.qt_moe_decode(X, logits, 1, gate, up, down, act=act)
    x = X.double().gather(1, j[:, None])[:, 0]
    z = g[at, 0, j] * x
    a, _ = act64(z, act)
    y = z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    ref = (a * u[at, 0, j] * x)[:, None] * d[at, :, 0]
    bound = (32 + 12 * y.abs() * torch.sigmoid(-y))[:, None] * U * ref.abs() + 1e-30
    if dtype == "bf16":
        bound = bound + torch.exp2(torch.floor(torch.log2(ref.abs().clamp_min(1e-30))) - 8)
    assert worst(out, ref, bound) <= 1


@pytest.mark.parametrize("T,E,k,D,F", [(16, 48, 8, 1024, 1536), (8, 64, 6, 2048, 1408)])
def test_bf16_calls_take_the_faster_launches(T, E, k, D, F):
    """Streams of 1 to 2 * 10^9 bytes times tokens, where the full layer's launches are
    the faster ones of either type: the layer's outputs, rounded once."""
    say(f"long bf16 T={T} E={E} k={k} D={D} F={F}")
    gen = torch.Generator(device=DEV).manual_seed(T)
    w = []
    for rows, cols in ((F, D), (F, D), (D, F)):
        n = rows * (cols // 64)
        packed = torch.randint(0, 256, (E, 24 * n), generator=gen, device=DEV, dtype=torch.uint8)
        w.append((packed, 0.01 + 0.01 * torch.rand((E, rows, cols // 64), generator=gen, device=DEV), 3))
    X = torch.randn((T, D), generator=gen, device=DEV).bfloat16()
    logits = torch.randn((T, E), generator=gen, device=DEV)
    layer = qt.qt_moe_layer(X.float(), logits, k, *w).bfloat16()
    assert torch.equal(qt.qt_moe_decode(X, logits, k, *w), layer)
