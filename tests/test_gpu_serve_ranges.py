"""The cache and its attention at the ends of their values' ranges: offsets of int4
values taken out exactly, values near the largest and the smallest numbers under
scores that rise, groups below the normal numbers."""
import math

import pytest
import torch

import dequant_matmul_int3_amd as qt
from tests import serve_util as su
from tests.gpu_util import DEV, say
from tests.test_gpu_serve import DT, check, gen, normal
from tests.tune_util import worst

pytestmark = pytest.mark.gpu


def filled(P, H, d, kb, vb, k_codes, k_scales, v_codes, v_scales):
    """A cache of one run of pages holding the codes [n, H, G, 64] and scales [n, H, G]
    of positions 0 .. n - 1, with a page table of `wide` pages."""
    n = k_codes.shape[0]
    pages = -(-n // P)
    k, v = qt.qt_kv_cache(pages, P, H, d, kb, vb, device=DEV)
    slots = torch.arange(n, device=DEV)
    su.store(k, False, slots, k_codes, k_scales)
    su.store(v, True, slots, v_codes, v_scales)
    return k, v


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kb,vb", [(4, 4), (8, 4), (8, 8)])
@pytest.mark.parametrize("d,wide", [(64, 16), (128, 60), (128, 400), (256, 16)])
@pytest.mark.parametrize("short", [True, False])
def test_codes_of_zero_give_zero(short, d, wide, kb, vb, dtype):
    """Values with the code 0 at every position come out as 0, whatever their group's
    scales s, 1 <= s < 2.  Scores are equal: a probability is a power of two, a
    value's weight its scale.  With scales of 16 bits, 256 of them times the offset 8
    stay below 2^24 of their steps of 8 * 2^-15: exact in f32 in any order, and what
    is taken out again is what was put in.  Otherwise both sums err by U = 2^-24 of
    8 sum s, which is below 16 n, for each of at most n / 8 + 200 additions."""
    say(f"zeros {short} d={d} wide={wide} k{kb} v{vb} {dtype}")
    g, P, H, n = gen(d + wide), 16, 2, 256
    G = su.groups(d)
    half = 2 ** (vb - 1)
    kc = torch.randint(-8, 8, (n, H, G, 64), generator=g, device=DEV)
    vc = torch.randint(-half, half, (n, H, G, 64), generator=g, device=DEV)
    vc[..., ::3] = 0
    vs = 1.0 + torch.rand((n, H, G), generator=g, device=DEV)
    if short:
        vs = (vs.view(torch.int32) & ~0xFF).view(torch.float32)
    k, v = filled(P, H, d, kb, vb, kc, torch.ones_like(vs), vc, vs)
    table = torch.full((1, wide), -1, dtype=torch.int32, device=DEV)
    table[0, :n // P] = torch.arange(n // P, device=DEV)
    lens = torch.tensor([n], device=DEV, dtype=torch.int32)
    Q = torch.zeros(1, 3 * H, d, device=DEV, dtype=DT[dtype])
    out = qt.qt_attn_decode(Q, k, v, table, lens)
    at = torch.arange(d, device=DEV) % 64 % 3 == 0
    exact = short or vb == 8 or dtype == "f32"  # no offset there
    assert out[..., at].abs().max() <= (0.0 if exact else 2 * su.U * (n / 8 + 200) * 16)
    assert out[..., ~at].any(-1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kb,vb", [(4, 4), (8, 8)])
@pytest.mark.parametrize("power", [120, 0, -90])
@pytest.mark.parametrize("d,n", [(64, 250), (128, 600), (128, 3000), (256, 700)])
def test_values_of_any_magnitude_under_rising_scores(d, n, power, kb, vb, dtype):
    """Every position's score is above the one's before it, 22 powers of two from
    the first to the last; values lie around 2^power.  The outputs are means of the
    values: they exist whatever the sums on the way."""
    say(f"rising d={d} n={n} 2^{power} k{kb} v{vb} {dtype}")
    g, P, H = gen(n + power), 32, 2
    G = su.groups(d)
    kc = torch.zeros((n, H, G, 64), dtype=torch.long, device=DEV)
    kc[:, :, 0, 0] = -2
    ks = torch.zeros((n, H, G), device=DEV)
    ks[..., 0] = -0.5 * torch.linspace(0, 22 * math.log(2), n, device=DEV)[:, None]
    vc, vs = su.quantize(normal(g, n, H, d) * 2.0 ** power, vb)
    k, v = filled(P, H, d, kb, vb, kc, ks, vc, vs)
    table = torch.arange(-(-n // P), device=DEV, dtype=torch.int32)[None].contiguous()
    lens = torch.tensor([n], device=DEV, dtype=torch.int32)
    Q = torch.zeros(1, 2 * H, d, device=DEV, dtype=DT[dtype])
    Q[..., 0] = 1.0
    out, lse = qt.qt_attn_decode(Q, k, v, table, lens, scale=1.0, want_lse=True)
    assert out.isfinite().all()
    # in units of 2^power, so that the bounds' absolute part stays below them
    small = 2.0 ** -power
    unit = (v[0], v[1] * small, vb)
    check(Q, k, unit, table, lens, ((out.double() * small).to(DT[dtype]), lse), scale=1.0)


@pytest.mark.parametrize("kb,vb", [(4, 4), (8, 4), (8, 8)])
@pytest.mark.parametrize("d,wide", [(64, 16), (128, 60), (128, 400), (200, 16)])
def test_one_position_is_rounded_once(d, wide, kb, vb):
    """A sequence of one position: the output is s v, rounded to bf16 once.  The
    probability is a power of two; the product's three terms and, at 4 bits, what the
    offset 8 takes out leave 4 U of 15 s (8 bits: of |s v|) besides, U = 2^-24, the
    quotient 2 U of |s v|."""
    say(f"one position d={d} wide={wide} k{kb} v{vb}")
    g, P, H, B = gen(d + wide), 16, 4, 40
    G, half = su.groups(d), 2 ** (vb - 1)
    kc = torch.randint(-8, 8, (B * P, H, G, 64), generator=g, device=DEV)
    vc = torch.randint(-half, half, (B * P, H, G, 64), generator=g, device=DEV)
    vs = torch.exp(3 * normal(g, B * P, H, G))
    k, v = filled(P, H, d, kb, vb, kc, normal(g, B * P, H, G), vc, vs)
    table = torch.full((B, wide), -1, dtype=torch.int32, device=DEV)
    table[:, 0] = torch.arange(B, device=DEV)
    lens = torch.ones(B, device=DEV, dtype=torch.int32)
    out = qt.qt_attn_decode(normal(g, B, 2 * H, d).bfloat16(), k, v, table, lens)
    ref = su.value(vc, vs, d)[::P].repeat_interleave(2, 1)
    step = vs[::P].double().repeat_interleave(64, -1)[..., :d].repeat_interleave(2, 1)
    half_ulp = torch.exp2(torch.floor(torch.log2(ref.abs().clamp_min(1e-30))) - 8)
    bound = half_ulp + su.U * (4 * (15 * step if vb == 4 else ref.abs()) + 2 * ref.abs())
    assert worst(out, ref, bound) <= 1


def test_one_part_is_read_alone():
    """Keys or values alone, and given tensors of either type beside no other."""
    g, R, H, d = gen(6), 70, 2, 96
    k, v = qt.qt_kv_cache(3, 32, H, d, 8, 4, device=DEV)
    x = normal(g, 96, H, d)
    qt.qt_kv_write(x, x, torch.arange(96, device=DEV, dtype=torch.int32), k, v)
    slots = torch.randint(-3, 99, (R,), generator=g, device=DEV, dtype=torch.int32)
    both = qt.qt_kv_read(slots, k, v, d, dtype=torch.float32)
    K, none = qt.qt_kv_read(slots, k, v, d, dtype=torch.float32, parts="k")
    assert none is None and torch.equal(K, both[0])
    none, V = qt.qt_kv_read(slots, k, v, d, parts="v")
    assert none is None and torch.equal(V, both[1].bfloat16())
    for dtype in (torch.float32, torch.bfloat16):
        for i in (0, 1):
            mine = torch.full((R, H, d), math.nan, device=DEV, dtype=dtype)
            got = qt.qt_kv_read(slots, k, v, d, **{"KV"[i]: mine})
            assert got[i] is mine
            assert all(torch.equal(a, b.to(dtype)) for a, b in zip(got, both))
            mine.fill_(math.nan)
            got = qt.qt_kv_read(slots, k, v, d, parts="kv"[i], **{"KV"[i]: mine},
                                stream=torch.cuda.current_stream())
            assert got[i] is mine and got[1 - i] is None and torch.equal(mine, both[i].to(dtype))
    with pytest.raises(ValueError, match="not read"):
        qt.qt_kv_read(slots, k, v, d, K=mine, parts="v")
    with pytest.raises(ValueError, match="parts"):
        qt.qt_kv_read(slots, k, v, d, parts="")
    with pytest.raises(ValueError, match="V must be"):
        qt.qt_kv_read(slots, k, v, d, K=mine, V=mine.float())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bits", [4, 8])
def test_groups_below_the_normal_numbers(bits, dtype):
    """Groups from the smallest subnormal number to 2^-95: codes and scales bit for
    bit, and what is read back."""
    g = gen(bits)
    T, H, d = 55 * 16, 2, 128
    power = torch.arange(-149, -94, device=DEV).repeat_interleave(16).double()
    x = (2.0 * torch.rand((T, H, d), generator=g, device=DEV, dtype=torch.float64) - 1.0)
    x[:, :, 1::5] *= 2.0 ** -3
    x = (x * 2.0 ** (power[:, None, None] + torch.randint(0, 3, (T, H, 1), generator=g, device=DEV)))
    x = x.float().to(DT[dtype])
    slots = torch.randperm(T, generator=g, device=DEV).int()
    k, v = qt.qt_kv_cache(T // 16, 16, H, d, bits, bits, device=DEV)
    qt.qt_kv_write(x, x, slots, k, v)
    c, s = su.quantize(x.cpu(), bits)
    # a group of zeros has the scale of its first one, whose sign s = -m / h turns
    zero = (x == 0).view(T, H, 2, 64).all(-1).cpu()
    s = torch.where(zero, -x.float().cpu()[:, :, ::64], s)
    assert (s != 0).any() and (s.abs() < 2.0 ** -126).any()
    for part, octets in ((k, False), (v, True)):
        gc, gs = su.fetch(part, octets, slots)
        assert torch.equal(gs.cpu().view(torch.int32), s.view(torch.int32))
        assert torch.equal(gc.cpu(), c)
    ref = su.value(c, s, d).float()
    for y in qt.qt_kv_read(slots, k, v, d, dtype=torch.float32):
        assert torch.equal(y.cpu(), ref)
