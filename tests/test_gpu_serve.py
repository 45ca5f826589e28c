"""The quantized key-value cache and its attention on the GPU against 64-bit
references (serve_util.py): bit-exact codes and scales, and attention within
bounds derived from its roundings."""
import math

import pytest
import torch

import dequant_matmul_int3_amd as qt
from tests import serve_util as su
from tests.gpu_util import DEV, say
from tests.tune_util import half_step, worst

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def cache(n, P, H, d, kb, vb, g, fill=None):
    """A cache of quantized normal values (or of bytes `fill` and NaN scales),
    stored by the reference."""
    k, v = qt.qt_kv_cache(n, P, H, d, kb, vb, device=DEV)
    if fill is not None:
        for c, s, _ in (k, v):
            c.fill_(fill)
            s.fill_(math.nan)
        return k, v
    slots = torch.arange(n * P, device=DEV)
    for part, octets in ((k, False), (v, True)):
        c, s = su.quantize(normal(g, n * P, H, d), part[2])
        su.store(part, octets, slots, c, s)
    return k, v


# ------------------------------------------------------------ write and read
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kb,vb", [(4, 8), (8, 4)])
@pytest.mark.parametrize("T,H,d,P", [(1, 1, 1, 16), (5, 3, 7, 16), (33, 2, 64, 48), (19, 1, 65, 16),
                                     (130, 4, 128, 64), (40, 5, 200, 32), (16, 2, 256, 16)])
def test_write_and_read(T, H, d, P, kb, vb, dtype):
    say(f"write T={T} H={H} d={d} P={P} k{kb} v{vb} {dtype}")
    g = gen(T * 1000 + d)
    n = -(-T // P) + 3
    k, v = cache(n, P, H, d, kb, vb, g, fill=0xA5)
    before = [t.clone() for t in (k[0], k[1], v[0], v[1])]
    # rows of a projection, at an odd distance; every scale of magnitudes
    rows = normal(g, T, 2 * H * d + 3) * torch.exp(4 * normal(g, T, 1))
    rows = rows.to(DT[dtype])
    K, V = rows[:, 1:1 + H * d].view(T, H, d), rows[:, 1 + H * d:1 + 2 * H * d].view(T, H, d)
    K[0, 0] = 0.0                          # a group of zeros
    V[T // 2, H - 1, -1] = -V[T // 2, H - 1].abs().max()  # equal magnitudes
    slots = torch.randperm(n * P, generator=g, device=DEV)[:T].int()
    if T > 4:
        slots[1], slots[3] = -1, n * P     # padding, and past the cache
    qt.qt_kv_write(K, V, slots, k, v)
    live = (slots >= 0) & (slots < n * P)
    for part, x, octets, old in ((k, K, False, before[:2]), (v, V, True, before[2:])):
        c, s = su.quantize(x[live], part[2])
        want = (old[0].clone(), old[1].clone(), part[2])
        su.store(want, octets, slots[live], c, s)
        assert torch.equal(part[0], want[0])  # the bytes, those of other slots among them
        assert torch.equal(part[1].view(torch.int32), want[1].view(torch.int32))
    for out_t in (torch.float32, torch.bfloat16):
        some = torch.cat([slots, slots[:1], slots.flip(0)])
        Kr, Vr = qt.qt_kv_read(some, k, v, d, dtype=out_t)
        ok = (some >= 0) & (some < n * P)
        for part, got, octets in ((k, Kr, False), (v, Vr, True)):
            ref = torch.zeros(some.numel(), H, d, device=DEV, dtype=torch.float64)
            ref[ok] = su.value(*su.fetch(part, octets, some[ok]), d)
            # s v is one rounding of the exact product: to f32, or through it to bf16
            assert torch.equal(got, ref.float().to(out_t))


@pytest.mark.parametrize("T,H,d", [(4099, 2, 128), (2731, 3, 70), (16384, 1, 64), (1025, 16, 33)])
def test_many_tokens(T, H, d):
    """Calls large enough for four tokens a thread, a number of them that four
    does not divide among them, with padding, and slots of either order."""
    say(f"many T={T} H={H} d={d}")
    g = gen(T)
    P = 64
    n = -(-T // P) + 1
    k, v = cache(n, P, H, d, 8, 4, g, fill=0x5A)
    old = [t.clone() for t in (k[0], k[1], v[0], v[1])]
    K, V = normal(g, T, H, d).bfloat16(), normal(g, T, H, d).bfloat16()
    slots = torch.arange(T, device=DEV, dtype=torch.int32).flip(0).contiguous()
    slots[::7] = -1
    slots[5], slots[T - 1] = n * P, -(1 << 31)
    qt.qt_kv_write(K, V, slots, k, v)
    live = (slots >= 0) & (slots < n * P)
    for part, x, octets, was in ((k, K, False, old[:2]), (v, V, True, old[2:])):
        c, s = su.quantize(x[live], part[2])
        want = (was[0].clone(), was[1].clone(), part[2])
        su.store(want, octets, slots[live], c, s)
        assert torch.equal(part[0], want[0])
        assert torch.equal(part[1].view(torch.int32), want[1].view(torch.int32))
    for out_t in (torch.float32, torch.bfloat16):
        got = qt.qt_kv_read(slots, k, v, d, dtype=out_t)
        for part, y, x, octets in ((k, got[0], K, False), (v, got[1], V, True)):
            ref = torch.zeros(T, H, d, device=DEV, dtype=torch.float64)
            ref[live] = su.value(*su.quantize(x[live], part[2]), d)
            assert torch.equal(y, ref.float().to(out_t))


def test_read_one_of_two():
    k, v = cache(3, 16, 2, 96, 8, 4, gen(5))
    slots = torch.tensor([47, 0, 13], device=DEV, dtype=torch.int32)
    K, V = qt.qt_kv_read(slots, k, v, 96, dtype=torch.float32)
    K2 = torch.empty_like(K)
    a = (*[t.data_ptr() for t in (slots,)], 3, k[0].data_ptr(), k[1].data_ptr(), 8, v[0].data_ptr(),
         v[1].data_ptr(), 4, 3, 16, 2, 96)
    s = torch.cuda.current_stream().cuda_stream
    assert qt.lib().qt_kv_read(*a, K2.data_ptr(), None, 0, s) == 0
    V2 = torch.empty_like(V)
    assert qt.lib().qt_kv_read(*a, None, V2.data_ptr(), 0, s) == 0
    assert torch.equal(K, K2) and torch.equal(V, V2)


@pytest.mark.parametrize("bits", [4, 8])
def test_rounding_at_ties(bits):
    """f32 quotients that round onto a tie take the neighbour that the exact
    quotient is nearest to."""
    g, half = gen(bits), 2 ** (bits - 1)
    T = 4096
    m = 1.0 + torch.rand(T, generator=g, device=DEV)
    x = torch.zeros(T, 1, 64, device=DEV)
    x[:, 0, 0] = m
    j = torch.randint(-half, half - 1, (T, 63), generator=g, device=DEV)
    tie = ((j.double() + 0.5) * (-m.double() / half)[:, None]).float()
    step = torch.randint(-2, 3, (T, 63), generator=g, device=DEV)
    x[:, 0, 1:] = (tie.view(torch.int32) + step.int()).view(torch.float32)
    k, v = qt.qt_kv_cache(T // 16, 16, 1, 64, bits, bits, device=DEV)
    slots = torch.arange(T, device=DEV, dtype=torch.int32)
    qt.qt_kv_write(x, x, slots, k, v)
    c, s = su.quantize(x, bits)
    for part, octets in ((k, False), (v, True)):
        gc, gs = su.fetch(part, octets, slots)
        assert torch.equal(gc, c) and torch.equal(gs, s)


def test_values_that_are_not_finite_stay_in_their_group():
    x = normal(gen(3), 4, 2, 128)
    x[0, 0, 3], x[1, 1, 70], x[2, 0, 127] = math.nan, math.inf, -math.inf
    x[3] = 2.0 ** -140  # below the normal numbers
    k, v = qt.qt_kv_cache(1, 16, 2, 128, 4, 8, device=DEV)
    slots = torch.arange(4, device=DEV, dtype=torch.int32)
    qt.qt_kv_write(x, x, slots, k, v)
    for part, octets, got in ((k, False, 0), (v, True, 1)):
        c, s = su.quantize(x[:3], part[2])
        gc, gs = su.fetch(part, octets, slots[:3])
        assert torch.equal(gc, c) and torch.equal(gs.view(torch.int32), s.view(torch.int32))
        r = qt.qt_kv_read(slots, k, v, 128, dtype=torch.float32)[got]
        assert r[0, 0, :64].isnan().all() and r[0, 0, 64:].isfinite().all()
        assert r[1, 1, 64:].isnan().all() and r[1, 1, :64].isfinite().all()
        assert r[2, 0, 64:].isnan().all() and r[3].isfinite().all()


# ----------------------------------------------------------------- attention
def check(Q, k, v, table, lens, got, window=0, scale=None, f32=None):
    out, lse = got
    B, Hq, d = Q.shape
    f32 = Q.dtype == torch.float32
    scale = d ** -0.5 if scale is None else scale
    P, pages = k[1].shape[2], k[1].shape[0]
    for b in range(B):
        n = max(0, min(int(lens[b]), table.shape[1] * P))
        pos = torch.arange(max(0, n - window) if window else 0, n, device=DEV)
        page = table[b].long()[pos // P]
        ok = (page >= 0) & (page < pages)
        slots = (page * P + pos % P)[ok]
        kc, ks = su.fetch(k, False, slots)
        vc, vs = su.fetch(v, True, slots)
        ref, rl, bo, bl = su.attend(Q[b], kc, ks, vc, vs, scale, f32, k[2], v[2])
        if slots.numel() == 0:
            assert not out[b].any() and (lse[b] == -math.inf).all(), b
            continue
        eo = worst(out[b], ref, bo + half_step(out.dtype) * (ref.abs() + bo) + 1e-30)
        el = worst(lse[b], rl, bl + half_step(torch.float32) * rl.abs() + 1e-30)
        assert eo <= 1 and el <= 1, (b, n, eo, el)


def tables(B, wide, g, spare=2):
    t = torch.randperm(B * wide + spare, generator=g, device=DEV)[:B * wide]
    return t.view(B, wide).int()


EDGES = [0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 300]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kb,vb", [(4, 4), (8, 8), (4, 8), (8, 4)])
@pytest.mark.parametrize("H,per,d,P,window", [(2, 4, 128, 16, 0), (1, 1, 64, 48, 0),
                                              (3, 2, 100, 64, 40), (2, 16, 192, 32, 0),
                                              (1, 40, 256, 16, 33), (2, 17, 7, 112, 0)])
def test_attention_edges(H, per, d, P, window, kb, vb, dtype):
    say(f"attention H={H} per={per} d={d} P={P} w={window} k{kb} v{vb} {dtype}")
    g = gen(d + 7 * kb + vb)
    B, wide = len(EDGES), -(-300 // P)
    k, v = cache(B * wide + 2, P, H, d, kb, vb, g)
    table = tables(B, wide, g)
    lens = torch.tensor(EDGES, device=DEV, dtype=torch.int32)
    rows = normal(g, B, H * per * d + 5).to(DT[dtype])
    Q = rows[:, 2:2 + H * per * d].view(B, H * per, d)
    got = qt.qt_attn_decode(Q, k, v, table, lens, window=window, want_lse=True)
    check(Q, k, v, table, lens, got, window)
    # without lse, and into given tensors: the same
    out = torch.full_like(got[0], math.nan)
    assert qt.qt_attn_decode(Q, k, v, table, lens, window=window, out=out) is out
    assert torch.equal(out, got[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,per,d,P,kb,vb,lens,window,scale",
                         [(2, 8, 128, 64, 4, 4, [9000, 1, 4097, 0], 0, None),
                          (1, 20, 80, 16, 8, 4, [5000], 0, 0.5),
                          (4, 1, 256, 128, 8, 8, [3000, 2999], 700, None),
                          (1, 3, 64, 32, 4, 8, [20011], 0, -0.1)])
def test_attention_in_chunks(H, per, d, P, kb, vb, lens, window, scale, dtype):
    say(f"chunks {lens} d={d} k{kb} v{vb} {dtype}")
    g = gen(sum(lens))
    B, wide = len(lens), -(-max(lens) // P)
    assert qt.qt_attn_decode_workspace_bytes(B, H * per, H, d, wide, P, window) > 0
    k, v = cache(B * wide + 2, P, H, d, kb, vb, g)
    table = tables(B, wide, g)
    lens = torch.tensor(lens, device=DEV, dtype=torch.int32)
    Q = normal(g, B, H * per, d).to(DT[dtype])
    got = qt.qt_attn_decode(Q, k, v, table, lens, scale=scale, window=window, want_lse=True)
    check(Q, k, v, table, lens, got, window, scale)
    again = qt.qt_attn_decode(Q, k, v, table, lens, scale=scale, window=window, want_lse=True)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kb,vb", [(4, 4), (8, 8), (4, 8), (8, 4)])
@pytest.mark.parametrize("H,per,d,P,window", [(2, 3, 128, 16, 0), (1, 7, 64, 48, 0),
                                              (2, 16, 100, 32, 990), (1, 33, 24, 64, 500)])
def test_attention_in_one_block(H, per, d, P, window, kb, vb, dtype):
    """Short contexts that one block takes, without a second launch."""
    say(f"one block H={H} per={per} d={d} P={P} w={window} k{kb} v{vb} {dtype}")
    g = gen(d + 5 * kb + vb)
    lens = torch.tensor([1024 // P * P, 1000, 257, 256, 33, 0], device=DEV, dtype=torch.int32)
    B, wide = 6, (2048 if window else 1024) // P
    if window:
        lens[1] = 2000
    assert qt.qt_attn_decode_workspace_bytes(B, H * per, H, d, wide, P, window) == 0
    k, v = cache(B * wide + 2, P, H, d, kb, vb, g)
    table = tables(B, wide, g)
    Q = normal(g, B, H * per, d).to(DT[dtype])
    got = qt.qt_attn_decode(Q, k, v, table, lens, window=window, want_lse=True)
    check(Q, k, v, table, lens, got, window)
    again = qt.qt_attn_decode(Q, k, v, table, lens, window=window, want_lse=True)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("kb,vb", [(4, 4), (8, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_memory_that_does_not_count(kb, vb, dtype):
    """Slots past a sequence's end hold NaN scales, some pages do not exist,
    lengths pass the table or are negative; what counts is attended to."""
    g = gen(11)
    H, per, d, P, wide = 2, 3, 128, 16, 80
    k, v = cache(4 * wide, P, H, d, kb, vb, g)
    table = torch.arange(4 * wide, device=DEV, dtype=torch.int32).view(4, wide)
    table[0, 1], table[0, 5], table[2, 0] = -1, 4 * wide, 1 << 30
    table[3, :] = -7                      # no page at all
    lens = torch.tensor([1000, 9999, -3, 40], device=DEV, dtype=torch.int32)
    for part in (k, v):
        part[1][62, :, 8:] = math.nan     # past position 1000 of sequence 0
        part[1][63:wide] = math.inf
        part[1][2 * wide:] = math.nan     # sequences 2 and 3 have none
    Q = normal(g, 4, H * per, d).to(DT[dtype])
    got = qt.qt_attn_decode(Q, k, v, table, lens, want_lse=True)
    check(Q, k, v, table, lens, got)
    assert got[0][:2].isfinite().all() and not got[0][2:].any()
    # and what counts and is not a number says so, for its sequence alone
    part = k if kb == 4 else v
    part[1][wide + 3, 1, 5] = math.nan
    bad = qt.qt_attn_decode(Q, k, v, table, lens)
    assert bad[1, per:].isnan().any() and torch.equal(bad[0], got[0][0])
    assert torch.equal(bad[1, :per], got[0][1, :per])


def test_large_scores():
    """Scores far apart: the maximum moves from tile to tile, the smallest
    probabilities vanish."""
    g = gen(21)
    H, d, P, n = 1, 64, 32, 2000
    k, v = cache(64, P, H, d, 8, 8, g)
    table = torch.arange(64, device=DEV, dtype=torch.int32)[None]
    lens = torch.tensor([n], device=DEV, dtype=torch.int32)
    ramp = torch.linspace(-1, 1, 64 * P, device=DEV).view(64, 1, P, 1)
    for sign in (1.0, -1.0):
        k[1].copy_(sign * 0.05 * ramp.expand_as(k[1]))
        for dtype in (torch.bfloat16, torch.float32):
            Q = (3 * normal(g, 1, 4, d)).to(dtype)
            got = qt.qt_attn_decode(Q, k, v, table, lens, scale=2.0, want_lse=True)
            check(Q, k, v, table, lens, got, scale=2.0)


def test_cache_past_32_bits():
    """Pages whose bytes lie past 2^32: written, read and attended to."""
    P, H, d, n = 64, 8, 256, 36000        # 4.7 GB of 8-bit codes
    free = torch.cuda.mem_get_info()[0]
    assert free > 16 << 30
    k, v = (tuple((torch.empty((n, H, P, 256), dtype=torch.uint8, device=DEV),
                   torch.empty((n, H, P, 4), dtype=torch.float32, device=DEV), 8)) for _ in "kv")
    g = gen(9)
    T = 150
    pages = torch.tensor([n - 1, 3, n - 5], device=DEV)
    pos = torch.arange(T, device=DEV)
    slots = (pages[pos // P] * P + pos % P).int()
    K, V = normal(g, T, H, d).bfloat16(), normal(g, T, H, d).bfloat16()
    qt.qt_kv_write(K, V, slots, k, v)
    Kr, Vr = qt.qt_kv_read(slots, k, v, d, dtype=torch.float32)
    assert torch.equal(Kr.double(), su.value(*su.quantize(K, 8), d))
    assert torch.equal(Vr.double(), su.value(*su.quantize(V, 8), d))
    lens = torch.tensor([T], device=DEV, dtype=torch.int32)
    Q = normal(g, 1, 2 * H, d).bfloat16()
    table = pages.int()[None]
    got = qt.qt_attn_decode(Q, k, v, table, lens, want_lse=True)
    check(Q, k, v, table, lens, got)


def test_write_then_attend_step_by_step():
    """Tokens come one at a time and each attends to those before it, by two
    calls on one stream; a captured step replays for the next tokens."""
    g = gen(31)
    H, per, d, P, B, n = 2, 3, 96, 16, 3, 37
    k, v = cache(B * 3, P, H, d, 8, 4, g, fill=0xFF)
    table = tables(B, 3, g, spare=0)
    K, V, Q = (normal(g, n, B, h, d).bfloat16() for h in (H, H, H * per))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    kin, vin, qin = torch.empty_like(K[0]), torch.empty_like(V[0]), torch.empty_like(Q[0])
    slots = torch.empty(B, dtype=torch.int32, device=DEV)
    lens = torch.empty(B, dtype=torch.int32, device=DEV)
    out = torch.empty_like(qin)
    lse = torch.empty(B, H * per, device=DEV)

    def step():
        qt.qt_kv_write(kin, vin, slots, k, v)
        qt.qt_attn_decode(qin, k, v, table, lens, out=out, lse=lse)

    graph = None
    for t in range(n):
        with torch.cuda.stream(st):
            kin.copy_(K[t]), vin.copy_(V[t]), qin.copy_(Q[t])
            slots.copy_(table[:, t // P] * P + t % P)
            lens.fill_(t + 1)
            if t < 5:
                step()
            elif graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=st):
                    step()
            if graph is not None:
                graph.replay()
        torch.cuda.synchronize()
        check(qin, k, v, table, lens, (out, lse))
        # the newest position is what was written
        Kr, _ = qt.qt_kv_read(slots, k, v, d, dtype=torch.float32)
        assert torch.equal(Kr.double(), su.value(*su.quantize(K[t], 8), d))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_decode_step(dtype):
    """What a decoder calls for its next tokens, together: the projection's keys
    and values into the cache, attention, the expert layer on what comes out, and
    the context read back; on a stream of its own, eager and replayed."""
    from tests.test_gpu_moe_decode import experts
    g = gen(71)
    B, H, per, P, d, E, F = 5, 2, 3, 32, 64, 9, 100
    D, wide, t = H * per * d, 60, DT[dtype]
    k, v = cache(B * wide, P, H, d, 8, 4, g)
    table = tables(B, wide, g, spare=0)
    lens = torch.tensor([1, 700, 1900, 64, 1], device=DEV, dtype=torch.int32)
    w = [experts(E, *s, b, i)[0] for i, (s, b) in
         enumerate((((F, D), 3), ((F, D), 4), ((D, F), 3)))]
    logits = torch.empty(B, E, device=DEV)
    rows = torch.empty(B, D + 2 * H * d, device=DEV, dtype=t)  # a fused projection's
    st = torch.cuda.Stream()

    def step():
        pos = (lens - 1).long()
        slots = (table[torch.arange(B, device=DEV), pos // P] * P + pos % P).int()
        kv = rows[:, D:].view(B, 2 * H, d)
        qt.qt_kv_write(kv[:, :H], kv[:, H:], slots, k, v)
        att = qt.qt_attn_decode(rows[:, :D].view(B, H * per, d), k, v, table, lens, want_lse=True)
        y = qt.qt_moe_decode(att[0].view(B, D), logits, 2, *w)
        back = qt.qt_kv_read(slots, k, v, d, dtype=torch.float32)
        lens.add_(1)
        return (*att, y, *back)

    def fill(i):
        rows.copy_(normal(gen(100 + i), *rows.shape))
        logits.copy_(normal(gen(200 + i), B, E))

    def fresh():
        lens.copy_(torch.tensor([1, 700, 1900, 64, 1], device=DEV, dtype=torch.int32))

    eager = []
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for i in range(4):
            fill(i)
            before = lens.clone()
            out = step()
            check(rows[:, :D].view(B, H * per, d), k, v, table, before, out[:2])
            for got, kv, bits, s in ((out[3], 0, 8, H), (out[4], H, 4, H)):
                x = rows[:, D:].view(B, 2 * H, d)[:, kv:kv + s]
                assert torch.equal(got, su.value(*su.quantize(x, bits), d).float())
            assert out[2].isfinite().all() and out[2].any()
            eager.append([o.clone() for o in out])
        fresh()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            out = step()
        fresh()
        for i in range(4):
            fill(i)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, eager[i]):
                assert torch.equal(a, b)
            normal(g, 1000).sum().item()  # the program's own work between replays


def test_a_stream_and_queries_of_others():
    """A call on a stream given as an object or a number, from another current
    one; queries that are every second sequence of a larger tensor."""
    g = gen(81)
    H, per, d, P, B = 2, 2, 40, 16, 3
    k, v = cache(B * 100, P, H, d, 4, 4, g)
    table = tables(B, 100, g, 0)
    lens = torch.tensor([1600, 3, 900], device=DEV, dtype=torch.int32)
    Q = normal(g, 2 * B, H * per, d)[::2]
    ref = qt.qt_attn_decode(Q.contiguous(), k, v, table, lens)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for s in (st, st.cuda_stream):
        got = qt.qt_attn_decode(Q, k, v, table, lens, stream=s)
        st.synchronize()
        assert torch.equal(got, ref)
    with pytest.raises(ValueError, match="contiguous tokens"):
        qt.qt_attn_decode(Q.transpose(0, 1), k, v, table, lens)
    with pytest.raises(ValueError, match="contiguous"):
        qt.qt_attn_decode(Q, k, v, table.t().contiguous().t(), lens)
    with pytest.raises(ValueError, match="device tensors"):
        qt.qt_attn_decode(Q, k, v, table, lens.cpu())


def test_workspace_of_the_size_asked_for():
    """A workspace full of NaN and of exactly the size; one too small is refused."""
    g = gen(41)
    H, per, d, P, wide = 2, 5, 80, 16, 200
    k, v = cache(wide, P, H, d, 8, 8, g)
    table = torch.arange(wide, device=DEV, dtype=torch.int32)[None].contiguous()
    Q = normal(g, 1, H * per, d)
    need = qt.qt_attn_decode_workspace_bytes(1, H * per, H, d, wide, P, 0)
    assert need > 0
    pad = torch.full((need // 4 + 64,), math.nan, device=DEV)
    ws = pad[16:16 + need // 4]
    for n in (3200, 1, 1500, 0):
        lens = torch.tensor([n], device=DEV, dtype=torch.int32)
        pad.fill_(math.nan)
        out, lse = qt.qt_attn_decode(Q, k, v, table, lens, want_lse=True, workspace=ws)
        check(Q, k, v, table, lens, (out, lse))
        assert pad[:16].isnan().all() and pad[16 + need // 4:].isnan().all()
    with pytest.raises(qt.QtError, match="workspace"):
        qt.qt_attn_decode(Q, k, v, table, lens, workspace=ws[:-1])


def test_two_streams_at_once():
    g = gen(51)
    H, per, d, P, wide = 2, 4, 128, 64, 100
    k, v = cache(2 * wide, P, H, d, 4, 8, g)
    table = tables(2, wide, g, 0)
    lens = torch.tensor([6400, 5000], device=DEV, dtype=torch.int32)
    Q = normal(g, 2, H * per, d).bfloat16()
    ref = [qt.qt_attn_decode(Q[i:i + 1], k, v, table[i:i + 1], lens[i:i + 1]) for i in (0, 1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        outs = [qt.qt_attn_decode(Q[i:i + 1], k, v, table[i:i + 1], lens[i:i + 1],
                                  stream=streams[i]) for i in (0, 1)]
        torch.cuda.synchronize()
        assert torch.equal(outs[0], ref[0]) and torch.equal(outs[1], ref[1])


def test_empty_tensors_and_sizes_are_refused():
    k, v = qt.qt_kv_cache(2, 16, 2, 64, 8, 8, device=DEV)
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    with pytest.raises(qt.QtError):
        qt.qt_kv_read(none, k, v, 64)
    with pytest.raises(qt.QtError):
        qt.qt_attn_decode(torch.zeros(1, 3, 64, device=DEV), k, v,
                          torch.zeros(1, 2, dtype=torch.int32, device=DEV),
                          torch.ones(1, dtype=torch.int32, device=DEV))
