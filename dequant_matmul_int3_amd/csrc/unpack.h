// Device-side unpacking of int3-g64 and grouped int4 codes into bf16 or f32
// matrix operands, shared by the feed-forward block and the backward passes.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tune.h"

namespace qt {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;

// The packed words of one 16-code quarter of a group: int3 has its 16 low
// pairs in a and its 16 high bits in half `q & 1` of b; int4 has codes 0..7
// in a and 8..15 in b.
struct Quarter {
    uint32_t a, b;
};

// int3: u = v + 4 of the quarter's codes, one per byte: word 0 holds codes
// 0 1 4 5, word 1 codes 2 3 6 7, word 2 codes 8 9 12 13, word 3 codes
// 10 11 14 15.  hsel picks the quarter's two high-plane bytes (0x0C010C00 for
// even quarters, 0x0C030C02 for odd ones) into bytes 0 and 2; one shift-or
// then spreads nibble b to byte b, so that bit i of byte b is the high bit of
// code 4b+i.
__device__ __forceinline__ void unpack_i3(uint32_t L, uint32_t hw, uint32_t hsel,
                                          uint32_t (&w)[4]) {
    const uint32_t b = __builtin_amdgcn_perm(0u, hw, hsel);
    const uint32_t t = (b | (b << 4)) & 0x0F0F0F0Fu;
    const uint32_t f0 = (L & 0x03030303u) | ((t << 2) & 0x04040404u);
    const uint32_t f1 = ((L >> 2) & 0x03030303u) | ((t << 1) & 0x04040404u);
    const uint32_t f2 = ((L >> 4) & 0x03030303u) | (t & 0x04040404u);
    const uint32_t f3 = ((L >> 6) & 0x03030303u) | ((t >> 1) & 0x04040404u);
    // byte b of f_i is code 4b+i
    w[0] = __builtin_amdgcn_perm(f1, f0, 0x05010400u);
    w[1] = __builtin_amdgcn_perm(f3, f2, 0x05010400u);
    w[2] = __builtin_amdgcn_perm(f1, f0, 0x07030602u);
    w[3] = __builtin_amdgcn_perm(f3, f2, 0x07030602u);
}
__device__ __forceinline__ uint32_t high_sel(int q) { return (q & 1) ? 0x0C030C02u : 0x0C010C00u; }

// v/16 of the two's-complement nibble in the low four bits of byte B of t.  The
// conversion is the compiler's: in inline assembly it would miss the waits kept between
// a matrix instruction and the next write of its accumulator's registers.
template <int B>
__device__ __forceinline__ float nibble(uint32_t t) {
    return __builtin_amdgcn_cvt_off_f32_i4((t >> (8 * B)) & 0xFFu);
}
// The eight codes of an int4 word as v/16, in order.
__device__ __forceinline__ void unpack_i4(uint32_t w, float (&v)[8]) {
    uint32_t t = w ^ 0x88888888u;
    asm("" : "+v"(t));  // one exclusive or and one shift for all bytes, which are selected
    uint32_t h = t >> 4;
    asm("" : "+v"(h));
    v[0] = nibble<0>(t);
    v[1] = nibble<0>(h);
    v[2] = nibble<1>(t);
    v[3] = nibble<1>(h);
    v[4] = nibble<2>(t);
    v[5] = nibble<2>(h);
    v[6] = nibble<3>(t);
    v[7] = nibble<3>(h);
}

// What the exact operand's products are multiplied by, beside the scale: the
// int4 codes enter as v/16.
__device__ __forceinline__ float code_unit(int bits) { return bits == 3 ? 1.0f : 16.0f; }

// Codes 0..7 and 8..15 of a quarter as exact bf16 (v for int3, v/16 for
// int4).  int3: a byte table maps u to the FP8 (E4M3) encoding of v/256
// (|v| <= 3 are subnormals, -4 the smallest normal) and the packed conversion
// with the scale 2^8 gives bf16(v), two codes per instruction.
__device__ __forceinline__ void exact_quarter(const Quarter& qd, int q, int bits, u32x4_t& lo8,
                                              u32x4_t& hi8) {
    if (bits == 3) {
        uint32_t w[4];
        unpack_i3(qd.a, qd.b, high_sel(q), w);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __builtin_amdgcn_perm(0x06040200u, 0x82848688u, w[i]);
#define QT_CV(u, HI) \
    __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, 256.0f, HI))
        lo8 = u32x4_t{QT_CV(w[0], false), QT_CV(w[1], false), QT_CV(w[0], true), QT_CV(w[1], true)};
        hi8 = u32x4_t{QT_CV(w[2], false), QT_CV(w[3], false), QT_CV(w[2], true), QT_CV(w[3], true)};
#undef QT_CV
    } else {
        float a[8], b[8];
        unpack_i4(qd.a, a);
        unpack_i4(qd.b, b);
        // the low halves are zero: the high halves are the bf16 values
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo8[i] = __builtin_amdgcn_perm(__float_as_uint(a[2 * i + 1]), __float_as_uint(a[2 * i]),
                                           0x07060302u);
            hi8[i] = __builtin_amdgcn_perm(__float_as_uint(b[2 * i + 1]), __float_as_uint(b[2 * i]),
                                           0x07060302u);
        }
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)a, (__bf16)b});
}

// The same codes times s in f16.  int3: a byte table gives f16(v), whose low
// byte is zero, and a packed product multiplies two codes by f16(s).  int4: the
// f16 word 0x6400 | u is 1024 + u and 0x5400 | u at bits 4..7 is 64 + u, both
// exact, and a packed subtraction leaves v = u - 8.  Two roundings of 2^-12.
__device__ __forceinline__ void scaled_quarter_f16(const Quarter& qd, int q, int bits, float s,
                                                   u32x4_t& lo8, u32x4_t& hi8) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    const h2 s2 = {(_Float16)s, (_Float16)s};
    auto mul = [&](uint32_t pair) {
        return __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2, pair) * s2);
    };
    if (bits == 3) {
        uint32_t w[4];
        unpack_i3(qd.a, qd.b, high_sel(q), w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // high bytes of f16(v), u = 0..3: c4 c2 c0 bc, u = 4..7: 00 3c 40 42
            const uint32_t hb = __builtin_amdgcn_perm(0x42403C00u, 0xBCC0C2C4u, w[i]);
            w[i] = hb;
        }
        auto lo = [&](uint32_t hb) { return mul(__builtin_amdgcn_perm(hb, hb, 0x010C000Cu)); };
        auto hi = [&](uint32_t hb) { return mul(__builtin_amdgcn_perm(hb, hb, 0x030C020Cu)); };
        lo8 = u32x4_t{lo(w[0]), lo(w[1]), hi(w[0]), hi(w[1])};
        hi8 = u32x4_t{lo(w[2]), lo(w[3]), hi(w[2]), hi(w[3])};
    } else {
        const h2 lo_off = {(_Float16)1032.0f, (_Float16)1032.0f};
        const h2 hi_off = {(_Float16)72.0f, (_Float16)72.0f};
        auto word = [&](uint32_t W, u32x4_t& o) {
            // nibbles n of the word in pairs (n, n + 4): 04 15 26 37
            const uint32_t W8 = W >> 8;
            uint32_t p[4];
            p[0] = __builtin_bit_cast(
                uint32_t, (__builtin_bit_cast(h2, (W & 0x000F000Fu) | 0x64006400u) - lo_off) * s2);
            p[1] = __builtin_bit_cast(
                uint32_t, (__builtin_bit_cast(h2, (W & 0x00F000F0u) | 0x54005400u) - hi_off) * s2);
            p[2] = __builtin_bit_cast(
                uint32_t, (__builtin_bit_cast(h2, (W8 & 0x000F000Fu) | 0x64006400u) - lo_off) * s2);
            p[3] = __builtin_bit_cast(
                uint32_t, (__builtin_bit_cast(h2, (W8 & 0x00F000F0u) | 0x54005400u) - hi_off) * s2);
            o = u32x4_t{__builtin_amdgcn_perm(p[1], p[0], 0x05040100u),
                        __builtin_amdgcn_perm(p[3], p[2], 0x05040100u),
                        __builtin_amdgcn_perm(p[1], p[0], 0x07060302u),
                        __builtin_amdgcn_perm(p[3], p[2], 0x07060302u)};
        };
        word(qd.a, lo8);
        word(qd.b, hi8);
    }
}

// The same products in f32 (one rounding).
__device__ __forceinline__ void scaled_quarter_f32(const Quarter& qd, int q, int bits, float s,
                                                   float (&v)[16]) {
    if (bits == 3) {
        uint32_t w[4];
        unpack_i3(qd.a, qd.b, high_sel(q), w);
        // codes in word order: 0 1 4 5 | 2 3 6 7 | 8 9 12 13 | 10 11 14 15
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const int j = 8 * (i >> 1) + 2 * (i & 1) + (b & 1) + 4 * (b >> 1);
                v[j] = ((float)((w[i] >> (8 * b)) & 0xFFu) - 4.0f) * s;
            }
    } else {
        float a[8], b[8];
        unpack_i4(qd.a, a);
        unpack_i4(qd.b, b);
        const float s16 = 16.0f * s;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = a[i] * s16;
            v[8 + i] = b[i] * s16;
        }
    }
}

// Three bf16 pieces that sum to x exactly (x's leading 8, next 8 and last 8
// significand bits), as bf16 bit patterns; exact for |x| >= 2^-110.
__device__ __forceinline__ void split3(float x, uint32_t& h, uint32_t& m, uint32_t& l) {
    const float hf = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
    const float r1 = x - hf;
    const float mf = __uint_as_float(__float_as_uint(r1) & 0xFFFF0000u);
    const float lf = r1 - mf;
    h = __float_as_uint(hf) >> 16;
    m = __float_as_uint(mf) >> 16;
    l = __float_as_uint(lf) >> 16;
}

// Row h of the four 16-lane rows takes element r of in[h]: the 4x4 transpose
// of four registers over the rows.
__device__ __forceinline__ void transpose_rows(uint32_t (&v)[4]) {
    const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    v[0] = c[0];
    v[1] = c[1];
    v[2] = d[0];
    v[3] = d[1];
}

// One lane's whole group of a row.  Where the four lane rows of a wave hold
// four consecutive groups of the same 16 matrix rows, quarters() exchanges
// them: lane row h gets quarter h of all four groups.
template <int BITS>
struct RowGroup;
template <>
struct RowGroup<3> {
    u32x2_t w[3];
    __device__ __forceinline__ void load(const uint8_t* __restrict__ p) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            w[i] = reinterpret_cast<const u32x2_t*>(p)[i];
    }
    __device__ __forceinline__ void quarters(Quarter (&q)[4]) const {
        uint32_t a[4] = {w[0].x, w[0].y, w[1].x, w[1].y};
        uint32_t b[4] = {w[2].x, w[2].x, w[2].y, w[2].y};
        transpose_rows(a);
        transpose_rows(b);
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = Quarter{a[j], b[j]};
    }
};
template <>
struct RowGroup<4> {
    u32x4_t w[2];
    __device__ __forceinline__ void load(const uint8_t* __restrict__ p) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = reinterpret_cast<const u32x4_t*>(p)[i];
    }
    __device__ __forceinline__ void quarters(Quarter (&q)[4]) const {
        uint32_t a[4] = {w[0].x, w[0].z, w[1].x, w[1].z};
        uint32_t b[4] = {w[0].y, w[0].w, w[1].y, w[1].w};
        transpose_rows(a);
        transpose_rows(b);
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = Quarter{a[j], b[j]};
    }
};

// The weights of one 16-row tile for a walk over the groups, four at a time:
// load(g) issues the loads of groups g .. g+3 (one per lane row; past the row
// a valid group is read), take() exchanges what the last load brought, so that
// word j of lane row h is quarter h of group g + j.  Lanes with `second` set
// read the second matrix; B1 and B2 are the matrices' bits.
template <int B1, int B2>
struct RowFeed {
    static constexpr int kBytes1 = B1 == 3 ? kGroupBytes : kGroupBytesI4;
    static constexpr int kBytes2 = B2 == 3 ? kGroupBytes : kGroupBytesI4;
    const uint8_t* p;
    const float* s;
    int G, h;
    bool second, four;  // this lane's matrix; whether its groups are int4
    RowGroup<B1> r;  // B1 == B2
    u32x2_t w[4];           // else: both formats' groups in 8-byte pieces
    float rs;
    Quarter q[4];
    uint32_t sc[4];

    __device__ __forceinline__ void init(const QMat& a, const QMat& b, bool sec, int64_t row,
                                         int G_, int h_) {
        second = sec;
        four = (sec ? B2 : B1) == 4;
        G = G_;
        h = h_;
        p = sec ? b.packed + row * G * kBytes2 : a.packed + row * G * kBytes1;
        s = (sec ? b.scales : a.scales) + row * G;
    }
    __device__ __forceinline__ void load(int g) {
        const int64_t i = g + h < G ? g + h : G - 1;
        if constexpr (B1 == B2) {
            r.load(p + i * kBytes1);
        } else {
            // no branch: an int3 group's fourth piece repeats its third
            const u32x2_t* d =
                reinterpret_cast<const u32x2_t*>(p + i * (second ? kBytes2 : kBytes1));
#pragma unroll
            for (int k = 0; k < 4; ++k)
                w[k] = d[k == 3 && !four ? 2 : k];
        }
        rs = s[i];
    }
    __device__ __forceinline__ void take() {
        if constexpr (B1 == B2) {
            r.quarters(q);
        } else {
            uint32_t a[4] = {w[0].x, four ? w[1].x : w[0].y, four ? w[2].x : w[1].x,
                             four ? w[3].x : w[1].y};
            uint32_t b[4] = {four ? w[0].y : w[2].x, four ? w[1].y : w[2].x,
                             four ? w[2].y : w[2].y, four ? w[3].y : w[2].y};
            transpose_rows(a);
            transpose_rows(b);
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = Quarter{a[j], b[j]};
        }
        const float u = rs * (second ? code_unit(B2) : code_unit(B1));
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[j] = __float_as_uint(u);
        transpose_rows(sc);
    }
    __device__ __forceinline__ void exact(int j, int qn, u32x4_t& lo8, u32x4_t& hi8) const {
        if constexpr (B1 == B2) {
            exact_quarter(q[j], qn, B1, lo8, hi8);
        } else {
            u32x4_t l4, h4;
            exact_quarter(q[j], qn, 3, lo8, hi8);
            exact_quarter(q[j], qn, 4, l4, h4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lo8[i] = four ? l4[i] : lo8[i];
                hi8[i] = four ? h4[i] : hi8[i];
            }
        }
    }
    // the scale times what the exact operand's codes are multiplied by
    __device__ __forceinline__ float scale(int j) const { return __uint_as_float(sc[j]); }
};

// Consecutive block ids run on different XCDs (8 of them, each with its own
// L2): the ids are remapped so that every XCD takes a contiguous range.
__device__ __forceinline__ int64_t xcd_range(int64_t lin, int64_t n) {
    const int64_t x = lin & 7, q = n >> 3, r = n & 7;
    return x * q + (x < r ? x : r) + (lin >> 3);
}

// ------------------------------------------------------------- activations
// act 0: silu(z) = z / (1 + e^-z).  act 1: gelu(z) = z/2 (1 + tanh y) with
// y = sqrt(2/pi) (z + 0.044715 z^3), which is z / (1 + e^(-2y)).
__device__ __forceinline__ void act_gate(float z, int act, float& sig, float& slope) {
    float x = z;
    slope = 1.0f;
    if (act == 1) {
        const float k = 1.5957691216057308f;  // 2 sqrt(2/pi)
        x = k * (z + 0.044715f * z * z * z);
        slope = k * (1.0f + 3.0f * 0.044715f * z * z);
    }
    sig = 1.0f / (1.0f + expf(-x));
}
__device__ __forceinline__ float act_value(float z, int act) {
    float s, sl;
    act_gate(z, act, s, sl);
    return z * s;
}
// The gradients of h = act(g) u: dg = dh u act'(g), du = dh act(g).  Where
// the sigmoid is 0 the derivative is 0 (the slope may have overflowed).
__device__ __forceinline__ void act_grads(float g, float u, float dh, int act, float& dg,
                                          float& du) {
    float s, sl;
    act_gate(g, act, s, sl);
    const float r = s * (1.0f - s);
    const float da = s + (r != 0.0f ? g * sl * r : 0.0f);
    dg = dh * u * da;
    du = dh * (g * s);
}

}  // namespace
}  // namespace qt
