// The quantized key-value cache: rows quantized into slots of its pages, and
// read back.
//
// Per (token, head, group of 64): m = the value of largest magnitude (the
// first of equals), s = -m / h with h = 8 or 128 (a power of two: exact but where s
// is below the normal numbers, where it is rounded to the nearest), v =
// clamp(nearest integer to x / s, ties to even, -h, h - 1).  Where s is exact m
// itself takes the code -h.
//
// Layout of a (page, head): key rows are one token after the other, int4 as
// the int4-g64 format (nibble j % 2 of byte j / 2), int8 byte j = v + 128.
// Values are laid out for the attention's second product, whose operands hold
// eight tokens of one value: blocks of eight tokens, in them group, then the
// group's 16 columns of four values, then the column's 8 x 4 codes: int8 byte
// 4 t + i, int4 byte 4 (t / 2) + 2 (i / 2) + t % 2 with value i in nibble
// i % 2 (the bytes of a pair of tokens alternate, so that a byte mask leaves
// both tokens' codes of one value next to each other).
//
// Memory bounds both where there is enough of it (16384 tokens of 8 x 128, 8 and 4
// bits, are read in 26 us: 95 MB, 3.6 TB/s; one access for four tokens' values
// in place of eight changes nothing), small calls their launch.
#include "serve.h"

namespace qt {
namespace {

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;

struct RwArgs {
    KvCache c;
    KvRows r;
    const int32_t* slots;
    int64_t T;        // tokens of the call
    int64_t t0;       // first row of units of this launch
    int32_t units;    // of 16 lanes: rows of units * heads * groups
    void *K, *V;      // read: outputs (null: not wanted)
    FastDiv hg, g, page;  // heads * groups, groups, page
    bool vec;         // read: four values of a head may be stored at once
};

// this lane's 16-lane row, rotated by N
template <int N>
__device__ __forceinline__ uint32_t ror16(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + N, 0xF, 0xF, false);
}
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = max(v, ror16<8>(v));
    v = max(v, ror16<4>(v));
    v = max(v, ror16<2>(v));
    return max(v, ror16<1>(v));
}

// The scale of a group whose lane holds values 4 c .. 4 c + 3 in x: a key of
// magnitude above, place and sign below finds the first of the largest.  A
// value that is not finite makes the scale NaN.
__device__ __forceinline__ float group_scale(const float (&x)[4], int c, int half) {
    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) best = max(best, __float_as_uint(x[i]) & 0x7FFFFFFFu);
    best = max16(best);
    uint32_t who = 0;  // 128 - 2 place, less one for a negative value
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = __float_as_uint(x[i]);
        if ((b & 0x7FFFFFFFu) == best) who = max(who, 128u - 2 * (4 * c + i) - (b >> 31));
    }
    who = max16(who);
    const float m = __uint_as_float(best);
    if (best >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    const float s = m / (float)half;  // exact, or rounded once to a subnormal number
    return who & 1 ? s : -s;
}

// clamp(nearest integer to x / s, ties to even), inv = 1 / s to a few units in
// the last place: the product is off by less than one, and the remainder,
// exact in one FMA where it is near half of s, tells which side it is on.
__device__ __forceinline__ int code_of(float x, float s, float inv, int half) {
    float q = rintf(x * inv);
    const float r2 = 2.0f * __builtin_fmaf(-q, s, x);
    const bool odd = (int)q & 1;
    if (fabsf(r2) > fabsf(s) || (fabsf(r2) == fabsf(s) && odd))
        q += (r2 < 0.0f) == (s < 0.0f) ? 1.0f : -1.0f;
    return min(max((int)q, -half), half - 1);
}
struct Unit {
    int64_t t;  // row of units: its tokens are TOK t ..
    int h, g;
};
__device__ __forceinline__ Unit unit_of(const RwArgs& a, uint32_t u) {
    const uint32_t t = a.hg.div(u), w = u - t * a.hg.d, h = a.g.div(w);
    return Unit{a.t0 + t, (int)h, (int)(w - h * a.g.d)};
}

// byte of this lane's four key codes in their (page, head), and of its value
// codes: int8 four bytes, int4 two bytes (keys: next to each other, values:
// two apart)
__device__ __forceinline__ int64_t k_byte(const KvCache& c, int t, int g, int col) {
    return ((int64_t)t * c.groups + g) * 8 * c.kbits + col * (c.kbits / 2);
}
__device__ __forceinline__ int64_t v_byte(const KvCache& c, int t, int g, int col) {
    const int64_t blk = (((int64_t)(t >> 3) * c.groups + g) * 16 + col) * (4 * c.vbits);
    return blk + (c.vbits == 8 ? 4 * (t & 7) : 4 * ((t & 7) >> 1) + (t & 1));
}

// TOK tokens of a unit, one after the other in the call: all their loads go out
// before the first is used (a wave of one token's group spends its life
// waiting: the write of 4096 tokens of 8 x 128 takes 16 us with one, 14.6 with four).
template <bool BF16, bool VEC, int TOK>
__global__ __launch_bounds__(256) void kv_write_kernel(RwArgs a) {
    const int tid = threadIdx.x, col = tid & 15;
    const uint32_t u = blockIdx.x * 16 + (tid >> 4);
    if (u >= (uint32_t)a.units) return;  // whole 16-lane rows
    const Unit n = unit_of(a, u);
    const bool val = blockIdx.y == 1;
    const int d0 = n.g * kGroup + 4 * col;
    const int64_t ld = val ? a.r.ldv : a.r.ldk;
    const void* src = val ? a.r.V : a.r.K;
    int32_t slot[TOK];
    float x[TOK][4];
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        const int64_t t = n.t * TOK + k, tc = min(t, a.T - 1);
        slot[k] = a.slots[tc];
        if (t >= a.T) slot[k] = -1;
        const int64_t row = tc * ld + (int64_t)n.h * a.c.dim;
        if constexpr (VEC) {  // four values lie wholly inside or outside the head
            const bool in = d0 < a.c.dim;
            const int64_t p = row + (in ? d0 : 0);
            if constexpr (BF16) {
                const u32x2_t w =
                    *reinterpret_cast<const u32x2_t*>(static_cast<const uint16_t*>(src) + p);
                x[k][0] = __uint_as_float(w.x << 16);
                x[k][1] = __uint_as_float(w.x & 0xFFFF0000u);
                x[k][2] = __uint_as_float(w.y << 16);
                x[k][3] = __uint_as_float(w.y & 0xFFFF0000u);
            } else {
                const f32x4_t w =
                    *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(src) + p);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[k][i] = w[i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) x[k][i] = in ? x[k][i] : 0.0f;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bool in = d0 + i < a.c.dim;
                const int64_t p = row + (in ? d0 + i : 0);
                if constexpr (BF16)
                    x[k][i] =
                        __uint_as_float((uint32_t)static_cast<const uint16_t*>(src)[p] << 16);
                else
                    x[k][i] = static_cast<const float*>(src)[p];
                x[k][i] = in ? x[k][i] : 0.0f;
            }
        }
    }
    const int bits = val ? a.c.vbits : a.c.kbits, half = 1 << (bits - 1);
    const int64_t rows = (int64_t)a.c.page * a.c.groups;  // (token, group) pairs of a (page, head)
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        const float s = group_scale(x[k], col, half);
        // tiny groups are quantized 2^60 times as large: 1 / s may overflow, or s be
        // no normal number
        const float up = fabsf(s) < 0x1p-100f ? 0x1p60f : 1.0f;
        const float inv = __builtin_amdgcn_rcpf(s * up);
        const bool any = fabsf(s) > 0.0f;  // neither 0 nor NaN
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = (uint32_t)((any ? code_of(x[k][i] * up, s * up, inv, half) : 0) + half);
        if (slot[k] < 0 || slot[k] >= a.c.pages * a.c.page) continue;
        const uint32_t pi = a.page.div((uint32_t)slot[k]);
        const int64_t ph = (int64_t)pi * a.c.heads + n.h;
        const int t = (int)((uint32_t)slot[k] - pi * a.page.d);
        uint8_t* dst = val ? a.c.vc + ph * rows * 8 * bits + v_byte(a.c, t, n.g, col)
                           : a.c.kc + ph * rows * 8 * bits + k_byte(a.c, t, n.g, col);
        if (bits == 8) {
            *reinterpret_cast<uint32_t*>(dst) = w[0] | w[1] << 8 | w[2] << 16 | w[3] << 24;
        } else if (val) {
            dst[0] = (uint8_t)(w[0] | w[1] << 4);
            dst[2] = (uint8_t)(w[2] | w[3] << 4);
        } else {
            *reinterpret_cast<uint16_t*>(dst) =
                (uint16_t)(w[0] | w[1] << 4 | w[2] << 8 | w[3] << 12);
        }
        if (col == 0) (val ? a.c.vs : a.c.ks)[ph * rows + (int64_t)t * a.c.groups + n.g] = s;
    }
}

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
__device__ __forceinline__ uint32_t pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)a, (__bf16)b});
}

template <bool BF16, int TOK>
__global__ __launch_bounds__(256) void kv_read_kernel(RwArgs a) {
    const int tid = threadIdx.x, col = tid & 15;
    const uint32_t u = blockIdx.x * 16 + (tid >> 4);
    if (u >= (uint32_t)a.units) return;
    const Unit n = unit_of(a, u);
    const bool val = blockIdx.y == 1;
    void* const out = val ? a.V : a.K;
    if (!out) return;
    const int bits = val ? a.c.vbits : a.c.kbits, half = 1 << (bits - 1);
    const int64_t rows = (int64_t)a.c.page * a.c.groups;
    const int d0 = n.g * kGroup + 4 * col;
    bool there[TOK];
    float s[TOK];
    uint32_t b[TOK];
    int32_t slot[TOK];
#pragma unroll
    for (int k = 0; k < TOK; ++k) slot[k] = a.slots[min(n.t * TOK + k, a.T - 1)];
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        there[k] = slot[k] >= 0 && slot[k] < a.c.pages * a.c.page;
        const uint32_t sl = there[k] ? (uint32_t)slot[k] : 0u, pi = a.page.div(sl);
        const int64_t ph = (int64_t)pi * a.c.heads + n.h;
        const int t = (int)(sl - pi * a.page.d);
        const uint8_t* src = val ? a.c.vc + ph * rows * 8 * bits + v_byte(a.c, t, n.g, col)
                                 : a.c.kc + ph * rows * 8 * bits + k_byte(a.c, t, n.g, col);
        s[k] = (val ? a.c.vs : a.c.ks)[ph * rows + (int64_t)t * a.c.groups + n.g];
        if (bits == 8)
            b[k] = *reinterpret_cast<const uint32_t*>(src);
        else if (val)
            b[k] = (uint32_t)src[0] | (uint32_t)src[2] << 8;
        else
            b[k] = *reinterpret_cast<const uint16_t*>(src);
    }
    if (d0 >= a.c.dim) return;
#pragma unroll
    for (int k = 0; k < TOK; ++k) {
        const int64_t t = n.t * TOK + k;
        if (t >= a.T) break;
        const int64_t at = (t * a.c.heads + n.h) * a.c.dim + d0;
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int w = (int)((b[k] >> (bits * i)) & (2u * half - 1u));
            y[i] = there[k] ? (float)(w - half) * s[k] : 0.0f;
        }
        if (a.vec) {
            if constexpr (BF16)
                *reinterpret_cast<u32x2_t*>(static_cast<__bf16*>(out) + at) =
                    u32x2_t{pair(y[0], y[1]), pair(y[2], y[3])};
            else
                *reinterpret_cast<f32x4_t*>(static_cast<float*>(out) + at) =
                    f32x4_t{y[0], y[1], y[2], y[3]};
            continue;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (d0 + i >= a.c.dim) break;
            if constexpr (BF16)
                static_cast<__bf16*>(out)[at + i] = (__bf16)y[i];
            else
                static_cast<float*>(out)[at + i] = y[i];
        }
    }
}

// Launches over ranges of units of at most 2^27 (2^31 threads).  Four tokens a
// unit where that still leaves every CU some blocks.
constexpr int kTok = 4;
template <typename F>
hipError_t over_tokens(RwArgs& a, int64_t T, F launch) {
    const int64_t hg = (int64_t)a.c.heads * a.c.groups;
    a.hg = FastDiv::of((uint32_t)hg);
    a.g = FastDiv::of((uint32_t)a.c.groups);
    a.page = FastDiv::of((uint32_t)a.c.page);
    a.T = T;
    const bool many = T * hg >= 16 * 256 * kTok;
    const int64_t rows = many ? (T + kTok - 1) / kTok : T;
    const int64_t most = std::max<int64_t>(1, (int64_t(1) << 27) / hg);
    for (int64_t t0 = 0; t0 < rows; t0 += most) {
        a.t0 = t0;
        a.units = (int32_t)(std::min(most, rows - t0) * hg);
        launch(dim3((unsigned)((a.units + 15) / 16), 2), many);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <bool BF16, bool VEC>
void run_write(const RwArgs& a, dim3 grid, bool many, hipStream_t s) {
    if (many)
        kv_write_kernel<BF16, VEC, kTok><<<grid, 256, 0, s>>>(a);
    else
        kv_write_kernel<BF16, VEC, 1><<<grid, 256, 0, s>>>(a);
}
template <bool BF16>
void run_read(const RwArgs& a, dim3 grid, bool many, hipStream_t s) {
    if (many)
        kv_read_kernel<BF16, kTok><<<grid, 256, 0, s>>>(a);
    else
        kv_read_kernel<BF16, 1><<<grid, 256, 0, s>>>(a);
}

}  // namespace

hipError_t launch_kv_write(const KvCache& c, const KvRows& r, const int32_t* slots, int64_t T,
                           hipStream_t s) {
    RwArgs a{};
    a.c = c;
    a.r = r;
    a.slots = slots;
    const uintptr_t mask = r.bf16 ? 7 : 15;
    const bool vec = c.dim % 4 == 0 && r.ldk % 4 == 0 && r.ldv % 4 == 0 &&
                     ((reinterpret_cast<uintptr_t>(r.K) | reinterpret_cast<uintptr_t>(r.V)) &
                      mask) == 0;
    return over_tokens(a, T, [&](dim3 grid, bool many) {
        if (r.bf16)
            vec ? run_write<true, true>(a, grid, many, s) : run_write<true, false>(a, grid, many, s);
        else
            vec ? run_write<false, true>(a, grid, many, s)
                : run_write<false, false>(a, grid, many, s);
    });
}

hipError_t launch_kv_read(const KvCache& c, const int32_t* slots, int64_t R, void* K, void* V,
                          bool bf16, hipStream_t s) {
    RwArgs a{};
    a.c = c;
    a.slots = slots;
    a.K = K;
    a.V = V;
    a.vec = c.dim % 4 == 0 &&
            ((reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(V)) & (bf16 ? 7 : 15)) == 0;
    return over_tokens(a, R, [&](dim3 grid, bool many) {
        bf16 ? run_read<true>(a, grid, many, s) : run_read<false>(a, grid, many, s);
    });
}

}  // namespace qt
