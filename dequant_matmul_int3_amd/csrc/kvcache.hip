// The quantized key-value cache: rows quantized into slots of its pages, and
// read back.
//
// Per (token, head, group of 64): m = the value of largest magnitude (the
// first of equals), s = -m / h with h = 8 or 128 (a power of two: exact), v =
// clamp(nearest integer to x / s, ties to even, -h, h - 1).  m itself takes
// the code -h exactly.
//
// Layout of a (page, head): key rows are one token after the other, int4 as
// the int4-g64 format (nibble j % 2 of byte j / 2), int8 byte j = v + 128.
// Values are laid out for the attention's second product, whose operands hold
// eight tokens of one value: blocks of eight tokens, in them group, then the
// group's 16 columns of four values, then the column's 8 x 4 codes: int8 byte
// 4 t + i, int4 byte 4 (t / 2) + 2 (i / 2) + t % 2 with value i in nibble
// i % 2 (the bytes of a pair of tokens alternate, so that a byte mask leaves
// both tokens' codes of one value next to each other).
#include "serve.h"

namespace qt {
namespace {

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;

struct RwArgs {
    KvCache c;
    KvRows r;
    const int32_t* slots;
    int64_t t0;       // first token of this launch
    int32_t units;    // of 16 lanes: tokens of this launch * heads * groups
    void *K, *V;      // read: outputs (null: not wanted)
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
    const float s = m / (float)half;  // exact: a power of two
    return who & 1 ? s : -s;
}

// clamp(nearest integer to x / s).  The rounded quotient can only fall on a
// tie that the true one misses: the remainder, exact in one FMA, tells.
__device__ __forceinline__ int code_of(float x, float s, int half) {
    if (!(s != 0.0f) || s != s) return 0;
    float q = rintf(x / s);
    const float r = __builtin_fmaf(-q, s, x);
    if (2.0f * fabsf(r) > fabsf(s)) q += (r < 0.0f) == (s < 0.0f) ? 1.0f : -1.0f;
    return min(max((int)q, -half), half - 1);
}

struct Unit {
    int64_t t;  // token of the call
    int h, g;
};
__device__ __forceinline__ Unit unit_of(const RwArgs& a, uint32_t u) {
    const uint32_t g = (uint32_t)a.c.groups, hg = (uint32_t)a.c.heads * g;
    const uint32_t t = u / hg, w = u - t * hg;
    return Unit{a.t0 + t, (int)(w / g), (int)(w % g)};
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

template <bool BF16, bool VEC>
__global__ __launch_bounds__(256) void kv_write_kernel(RwArgs a) {
    const int tid = threadIdx.x, col = tid & 15;
    const uint32_t u = blockIdx.x * 16 + (tid >> 4);
    if (u >= (uint32_t)a.units) return;  // whole 16-lane rows
    const Unit n = unit_of(a, u);
    const bool val = blockIdx.y == 1;
    const int32_t slot = a.slots[n.t];
    if (slot < 0 || slot >= a.c.pages * a.c.page) return;
    const int d0 = n.g * kGroup + 4 * col;
    const int64_t at = n.t * (val ? a.r.ldv : a.r.ldk) + (int64_t)n.h * a.c.dim + d0;
    float x[4];
    if constexpr (VEC) {  // four values lie wholly inside or outside the head
        const bool in = d0 < a.c.dim;
        const int64_t p = in ? at : at - 4 * col - n.g * kGroup;
        if constexpr (BF16) {
            const u32x2_t w = *reinterpret_cast<const u32x2_t*>(
                reinterpret_cast<const uint16_t*>(val ? a.r.V : a.r.K) + p);
            x[0] = __uint_as_float(w.x << 16);
            x[1] = __uint_as_float(w.x & 0xFFFF0000u);
            x[2] = __uint_as_float(w.y << 16);
            x[3] = __uint_as_float(w.y & 0xFFFF0000u);
        } else {
            const f32x4_t w = *reinterpret_cast<const f32x4_t*>(
                reinterpret_cast<const float*>(val ? a.r.V : a.r.K) + p);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = w[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = in ? x[i] : 0.0f;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = d0 + i < a.c.dim;
            const int64_t p = in ? at + i : at - d0;
            if constexpr (BF16)
                x[i] = __uint_as_float(
                    (uint32_t)reinterpret_cast<const uint16_t*>(val ? a.r.V : a.r.K)[p] << 16);
            else
                x[i] = reinterpret_cast<const float*>(val ? a.r.V : a.r.K)[p];
            x[i] = in ? x[i] : 0.0f;
        }
    }
    const int bits = val ? a.c.vbits : a.c.kbits, half = 1 << (bits - 1);
    const float s = group_scale(x, col, half);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)(code_of(x[i], s, half) + half);
    const uint32_t page = (uint32_t)a.c.page;
    const int64_t ph = (int64_t)((uint32_t)slot / page) * a.c.heads + n.h;
    const int t = (int)((uint32_t)slot % page);
    const int64_t row = (int64_t)page * a.c.groups;  // (token, group) pairs of a (page, head)
    uint8_t* dst = val ? a.c.vc + ph * row * 8 * bits + v_byte(a.c, t, n.g, col)
                       : a.c.kc + ph * row * 8 * bits + k_byte(a.c, t, n.g, col);
    if (bits == 8) {
        *reinterpret_cast<uint32_t*>(dst) = w[0] | w[1] << 8 | w[2] << 16 | w[3] << 24;
    } else if (val) {
        dst[0] = (uint8_t)(w[0] | w[1] << 4);
        dst[2] = (uint8_t)(w[2] | w[3] << 4);
    } else {
        *reinterpret_cast<uint16_t*>(dst) = (uint16_t)(w[0] | w[1] << 4 | w[2] << 8 | w[3] << 12);
    }
    if (col == 0) (val ? a.c.vs : a.c.ks)[ph * row + (int64_t)t * a.c.groups + n.g] = s;
}

template <bool BF16>
__global__ __launch_bounds__(256) void kv_read_kernel(RwArgs a) {
    const int tid = threadIdx.x, col = tid & 15;
    const uint32_t u = blockIdx.x * 16 + (tid >> 4);
    if (u >= (uint32_t)a.units) return;
    const Unit n = unit_of(a, u);
    const bool val = blockIdx.y == 1;
    void* const out = val ? a.V : a.K;
    if (!out) return;
    const int32_t slot = a.slots[n.t];
    const bool there = slot >= 0 && slot < a.c.pages * a.c.page;
    const int bits = val ? a.c.vbits : a.c.kbits, half = 1 << (bits - 1);
    const uint32_t page = (uint32_t)a.c.page, sl = there ? (uint32_t)slot : 0u;
    const int64_t ph = (int64_t)(sl / page) * a.c.heads + n.h;
    const int t = (int)(sl % page);
    const int64_t row = (int64_t)page * a.c.groups;
    const uint8_t* src = val ? a.c.vc + ph * row * 8 * bits + v_byte(a.c, t, n.g, col)
                             : a.c.kc + ph * row * 8 * bits + k_byte(a.c, t, n.g, col);
    const float s = (val ? a.c.vs : a.c.ks)[ph * row + (int64_t)t * a.c.groups + n.g];
    int w[4];
    if (bits == 8) {
        const uint32_t b = *reinterpret_cast<const uint32_t*>(src);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (int)((b >> (8 * i)) & 255u);
    } else {
        const uint32_t b = val ? (uint32_t)src[0] | (uint32_t)src[2] << 8
                               : (uint32_t)*reinterpret_cast<const uint16_t*>(src);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (int)((b >> (4 * i)) & 15u);
    }
    const int d0 = n.g * kGroup + 4 * col;
    const int64_t at = (n.t * a.c.heads + n.h) * a.c.dim + d0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (d0 + i >= a.c.dim) break;
        const float x = there ? (float)(w[i] - half) * s : 0.0f;
        if constexpr (BF16)
            static_cast<__bf16*>(out)[at + i] = (__bf16)x;
        else
            static_cast<float*>(out)[at + i] = x;
    }
}

// Launches over ranges of tokens of at most 2^27 units (2^31 threads).
template <typename F>
hipError_t over_tokens(RwArgs& a, int64_t T, F launch) {
    const int64_t hg = (int64_t)a.c.heads * a.c.groups;
    const int64_t most = std::max<int64_t>(1, (int64_t(1) << 27) / hg);
    for (int64_t t0 = 0; t0 < T; t0 += most) {
        a.t0 = t0;
        a.units = (int32_t)(std::min(most, T - t0) * hg);
        launch(dim3((unsigned)((a.units + 15) / 16), 2));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_kv_write(const KvCache& c, const KvRows& r, const int32_t* slots, int64_t T,
                           hipStream_t s) {
    RwArgs a{c, r, slots, 0, 0, nullptr, nullptr};
    const uintptr_t mask = r.bf16 ? 7 : 15;
    const bool vec = c.dim % 4 == 0 && r.ldk % 4 == 0 && r.ldv % 4 == 0 &&
                     ((reinterpret_cast<uintptr_t>(r.K) | reinterpret_cast<uintptr_t>(r.V)) &
                      mask) == 0;
    return over_tokens(a, T, [&](dim3 grid) {
        if (r.bf16)
            vec ? kv_write_kernel<true, true><<<grid, 256, 0, s>>>(a)
                : kv_write_kernel<true, false><<<grid, 256, 0, s>>>(a);
        else
            vec ? kv_write_kernel<false, true><<<grid, 256, 0, s>>>(a)
                : kv_write_kernel<false, false><<<grid, 256, 0, s>>>(a);
    });
}

hipError_t launch_kv_read(const KvCache& c, const int32_t* slots, int64_t R, void* K, void* V,
                          bool bf16, hipStream_t s) {
    RwArgs a{c, {}, slots, 0, 0, K, V};
    return over_tokens(a, R, [&](dim3 grid) {
        bf16 ? kv_read_kernel<true><<<grid, 256, 0, s>>>(a)
             : kv_read_kernel<false><<<grid, 256, 0, s>>>(a);
    });
}

}  // namespace qt
