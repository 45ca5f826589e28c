// Device-side unpacking of int3-g64 and grouped int4 codes into bf16 or f32
// matrix operands, shared by the feed-forward block and the backward passes.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

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

// Quarter q of group `grp` (24 or 32 bytes, 4-byte aligned).
__device__ __forceinline__ Quarter load_quarter(const uint8_t* __restrict__ grp, int q, int bits) {
    Quarter r;
    if (bits == 3) {
        r.a = *reinterpret_cast<const uint32_t*>(grp + 4 * q);
        r.b = *reinterpret_cast<const uint32_t*>(grp + 16 + 4 * (q >> 1));
    } else {
        const u32x2_t w = *reinterpret_cast<const u32x2_t*>(grp + 8 * q);
        r.a = w.x;
        r.b = w.y;
    }
    return r;
}

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

// v/16 of the two's-complement nibble in the low four bits of byte B of t.
template <int B>
__device__ __forceinline__ float nibble(uint32_t t) {
    float r;
    if constexpr (B == 0)
        asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0"
            : "=v"(r) : "v"(t));
    else if constexpr (B == 1)
        asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1"
            : "=v"(r) : "v"(t));
    else if constexpr (B == 2)
        asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2"
            : "=v"(r) : "v"(t));
    else
        asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3"
            : "=v"(r) : "v"(t));
    return r;
}
// The eight codes of an int4 word as v/16, in order.
__device__ __forceinline__ void unpack_i4(uint32_t w, float (&v)[8]) {
    const uint32_t t = w ^ 0x88888888u, h = t >> 4;
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

// The same codes times the group's scale s, each product rounded once to
// bf16.  int3 has eight possible products per group: bf16(s), bf16(2s),
// bf16(3s), bf16(4s) and their negatives, whose high and low bytes make two
// byte tables.
__device__ __forceinline__ void scaled_quarter(const Quarter& qd, int q, int bits, float s,
                                               u32x4_t& lo8, u32x4_t& hi8) {
    if (bits == 3) {
        uint32_t w[4];
        unpack_i3(qd.a, qd.b, high_sel(q), w);
        const uint32_t p12 = bf16_pair(s, 2.0f * s), p34 = bf16_pair(3.0f * s, 4.0f * s);
        // entries u = 0..3 are -4s -3s -2s -s, u = 4..7 are 0 s 2s 3s
        const uint32_t lo_n = __builtin_amdgcn_perm(p34, p12, 0x00020406u);
        const uint32_t hi_n = __builtin_amdgcn_perm(p34, p12, 0x01030507u) ^ 0x80808080u;
        const uint32_t lo_p = __builtin_amdgcn_perm(p34, p12, 0x0402000Cu);
        const uint32_t hi_p = __builtin_amdgcn_perm(p34, p12, 0x0503010Cu);
        uint32_t d[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t hi = __builtin_amdgcn_perm(hi_p, hi_n, w[i]);
            const uint32_t lo = __builtin_amdgcn_perm(lo_p, lo_n, w[i]);
            d[i][0] = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
            d[i][1] = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
        }
        lo8 = u32x4_t{d[0][0], d[1][0], d[0][1], d[1][1]};
        hi8 = u32x4_t{d[2][0], d[3][0], d[2][1], d[3][1]};
    } else {
        float a[8], b[8];
        unpack_i4(qd.a, a);
        unpack_i4(qd.b, b);
        const float s16 = 16.0f * s;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo8[i] = bf16_pair(a[2 * i] * s16, a[2 * i + 1] * s16);
            hi8[i] = bf16_pair(b[2 * i] * s16, b[2 * i + 1] * s16);
        }
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
