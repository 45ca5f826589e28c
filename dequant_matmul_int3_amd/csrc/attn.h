// Attention of one new token per sequence over the quantized paged cache: the
// kernel over a chunk of positions, instantiated for bf16 and f32 calls in a
// source of its own each.
//
//   S_t = scale sum_g sK[t,g] sum_j q_j vK[t,j],  p = softmax(S),
//   out_j = sum_t p_t sV[t,g(j)] vV[t,j]
//
// A block owns a chunk of one sequence's positions for one key-value head and
// up to 16 of its query heads; its four waves take tiles of 32 positions in
// turn, each with an online softmax of its own (running maximum and sum in
// f32), and join them in LDS at the end.  The cache's bytes are read once and
// bound it; both products run on the bf16 matrix cores, whatever the number of
// heads, so that the vector instructions per cache value stay below two.
//
// First product: the keys' codes as 16 x 32 operands (rows are tokens), the
// queries' values as the other (f32 queries as three exact bf16 pieces); each
// group's sum takes its f32 scale afterwards.  Row r of the tile's half s is
// token 8 (r / 4) + 4 s + r % 4: the results of the two halves are then, lane
// by lane, eight consecutive tokens of one head, which is what the second
// product's operand wants: no probability moves between lanes.  It takes p sV
// as two bf16 pieces (three in f32 calls; one alone would add an error as
// large as the output's own rounding) and the values' codes, of which a lane
// loads eight tokens x four values in one piece (the layout of the pages).
//
// bf16 calls take int4 codes as u = v + 8: the nibble is the FP8 (E4M3)
// encoding of u / 512, so a mask and a packed conversion make two operands,
// and the eightfold sums are taken out again (in the keys' product as its
// initial value, in the values' at the end).  f32 calls convert to v itself
// (over a long flat softmax the offset costs more than f32's accuracy).
#pragma once
#include "lds_barrier.h"
#include "serve.h"
#include "unpack.h"
#include "wave_reduce.h"

namespace qt {

// One call's arguments in the kernel; see AttnArgs.
struct AttnKernelArgs {
    AttnArgs a;
    int chunk, splits, tiles;   // tiles: of 16 query heads per key-value head
    uint32_t page_mul, page_sh; // x / page for x < 2^31
    float* part;                // splits > 1: [rows][splits] x (G 64 values, max, sum)
};

hipError_t launch_attn_bf16(const AttnKernelArgs& k, hipStream_t s);
hipError_t launch_attn_f32(const AttnKernelArgs& k, hipStream_t s);

namespace {

constexpr int kAttnWaves = 4;
constexpr int kAttnTile = 32;

// max / sum over the four lanes that share l % 16
__device__ __forceinline__ float quad_max(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const float m = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const uint32_t w = __float_as_uint(m);
    const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quad_sum(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const float m = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const uint32_t w = __float_as_uint(m);
    const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

template <int B>
__device__ __forceinline__ float signed_byte(uint32_t t) {
    float r;
    if constexpr (B == 0)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0"
            : "=v"(r) : "v"(t));
    else if constexpr (B == 1)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1"
            : "=v"(r) : "v"(t));
    else if constexpr (B == 2)
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2"
            : "=v"(r) : "v"(t));
    else
        asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3"
            : "=v"(r) : "v"(t));
    return r;
}
// the high halves of two f32 values as a bf16 pair
__device__ __forceinline__ uint32_t high_pair(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ uint32_t fp8_pair(uint32_t u, bool hi) {
    return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, 512.0f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, 512.0f, false));
}

// What the operand's codes stand for: u = v + 8 (bf16 calls' int4), v / 16
// (f32 calls' int4) or v.
template <int BITS, bool F32>
struct Code {
    static constexpr bool kOffset = BITS == 4 && !F32;
    static constexpr float kUnit = BITS == 4 && F32 ? 16.0f : 1.0f;
};

// Eight key codes as an operand, and which of the eight the operand's value j
// is.
template <bool F32>
__device__ __forceinline__ u32x4_t key_operand4(uint32_t w) {
    if constexpr (F32) {
        float v[8];
        unpack_i4(w, v);
        return u32x4_t{high_pair(v[0], v[1]), high_pair(v[2], v[3]), high_pair(v[4], v[5]),
                       high_pair(v[6], v[7])};
    } else {
        const uint32_t e = w & 0x0F0F0F0Fu, o = (w >> 4) & 0x0F0F0F0Fu;
        return u32x4_t{fp8_pair(e, false), fp8_pair(e, true), fp8_pair(o, false),
                       fp8_pair(o, true)};
    }
}
__device__ __forceinline__ u32x4_t key_operand8(uint32_t lo, uint32_t hi) {
    const uint32_t a = lo ^ 0x80808080u, b = hi ^ 0x80808080u;
    return u32x4_t{high_pair(signed_byte<0>(a), signed_byte<1>(a)),
                   high_pair(signed_byte<2>(a), signed_byte<3>(a)),
                   high_pair(signed_byte<0>(b), signed_byte<1>(b)),
                   high_pair(signed_byte<2>(b), signed_byte<3>(b))};
}
template <int BITS, bool F32>
__device__ __forceinline__ int key_order(int j) {
    return BITS == 4 && !F32 ? (j < 4 ? 2 * j : 2 * j - 7) : j;
}

// The codes of eight tokens x four values as four operands.
template <bool F32>
__device__ __forceinline__ void value_operands4(const u32x4_t& w, u32x4_t (&o)[4]) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {  // a pair of tokens
        if constexpr (F32) {
            const uint32_t t = w[a] ^ 0x88888888u, h = t >> 4;
            o[0][a] = high_pair(nibble<0>(t), nibble<1>(t));
            o[1][a] = high_pair(nibble<0>(h), nibble<1>(h));
            o[2][a] = high_pair(nibble<2>(t), nibble<3>(t));
            o[3][a] = high_pair(nibble<2>(h), nibble<3>(h));
        } else {
            const uint32_t e = w[a] & 0x0F0F0F0Fu, d = (w[a] >> 4) & 0x0F0F0F0Fu;
            o[0][a] = fp8_pair(e, false);
            o[1][a] = fp8_pair(d, false);
            o[2][a] = fp8_pair(e, true);
            o[3][a] = fp8_pair(d, true);
        }
    }
}
__device__ __forceinline__ void value_operands8(const u32x4_t& w0, const u32x4_t& w1,
                                                u32x4_t (&o)[4]) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {
        const uint32_t x = (a < 2 ? w0[2 * a] : w1[2 * a - 4]) ^ 0x80808080u;
        const uint32_t y = (a < 2 ? w0[2 * a + 1] : w1[2 * a - 3]) ^ 0x80808080u;
        o[0][a] = high_pair(signed_byte<0>(x), signed_byte<0>(y));
        o[1][a] = high_pair(signed_byte<1>(x), signed_byte<1>(y));
        o[2][a] = high_pair(signed_byte<2>(x), signed_byte<2>(y));
        o[3][a] = high_pair(signed_byte<3>(x), signed_byte<3>(y));
    }
}

__device__ __forceinline__ f32x4_t mma(const u32x4_t& a, const u32x4_t& b, const f32x4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// What a tile of 32 positions is read into: codes as the operands want them,
// the tile's 32 G scales one after the other over the lanes.
template <int KB, int VB, int G>
struct AttnTile {
    u32x4_t k[2][KB == 8 ? G : (G + 1) / 2];  // int4: two groups a word of four
    u32x4_t v[VB == 8 ? 2 * G : G];
    float sk[(G + 1) / 2], sv[(G + 1) / 2];
};

// Where a tile lies: the (page, head) and place of its halves of 16 positions.
struct AttnPlace {
    int64_t ph[2];
    int at[2];
    bool ok[2];  // the page exists
};

template <int KB, int VB, int G, bool F32>
__global__ __launch_bounds__(64 * kAttnWaves) void attn_decode_kernel(const AttnKernelArgs x) {
    constexpr int NP = F32 ? 3 : 1;   // pieces of a query value
    constexpr int PP = F32 ? 3 : 2;   // pieces of a probability
    constexpr int KROW = G * 8 * KB, W = G * kGroup;
    using KC = Code<KB, F32>;
    using VC = Code<VB, F32>;
    const AttnArgs& a = x.a;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    const int kvh = blockIdx.y / x.tiles, qt = blockIdx.y % x.tiles, b = blockIdx.z;
    const int per = a.q_heads / a.c.heads;
    const int r0 = 16 * qt, nr = min(16, per - r0);  // query heads of this block
    const int64_t row0 = (int64_t)b * a.q_heads + (int64_t)kvh * per + r0;

    // positions lo .. n - 1, this block's from t_begin to t_end
    const int64_t reach = a.table_pages * a.c.page;
    const int n = (int)min<int64_t>(max(a.lens[b], 0), reach);
    const int lo = a.window > 0 && a.window < n ? (int)(n - a.window) : 0;
    const int64_t begin = (lo & ~(kAttnTile - 1)) + (int64_t)blockIdx.x * x.chunk;
    if (begin >= n && blockIdx.x > 0) return;  // the first chunk writes even nothing
    const int t_begin = (int)min<int64_t>(begin, n);
    const int t_end = (int)min<int64_t>(begin + x.chunk, n);

    // ---- queries as operands: column l16 is the head, values 16 g .. of each
    // group in the order that the codes come in
    u32x4_t q[NP][G][2];
    float qoff[G];  // -8 times the group's sum, where the codes are offset
    {
        const int64_t head = (int64_t)kvh * per + r0 + min(l16, nr - 1);
        const int64_t at = (int64_t)b * a.ldq + head * a.c.dim;
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
            float sum = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t p[NP][8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int d = 64 * gr + 16 * g + 8 * h + key_order<KB, F32>(j);
                    const int64_t i = at + min(d, a.c.dim - 1);
                    if constexpr (F32) {
                        float v = static_cast<const float*>(a.Q)[i];
                        v = d < a.c.dim ? v : 0.0f;
                        split3(v, p[0][j], p[NP > 1 ? 1 : 0][j], p[NP > 1 ? 2 : 0][j]);
                    } else {
                        uint32_t v = static_cast<const uint16_t*>(a.Q)[i];
                        p[0][j] = d < a.c.dim ? v : 0u;
                        sum += __uint_as_float(p[0][j] << 16);
                    }
                }
#pragma unroll
                for (int k = 0; k < NP; ++k)
                    q[k][gr][h] = u32x4_t{p[k][0] | p[k][1] << 16, p[k][2] | p[k][3] << 16,
                                          p[k][4] | p[k][5] << 16, p[k][6] | p[k][7] << 16};
            }
            qoff[gr] = KC::kOffset ? -8.0f * quad_sum(sum) : 0.0f;
        }
    }

    // ---- a tile's place (scalar) and its loads
    const int64_t prow = (int64_t)a.c.page * G;  // scales of a (page, head)
    const int32_t* table = a.table + (int64_t)b * a.table_pages;
    const int ka = 8 * (l16 >> 2) + (l16 & 3);  // this lane's key row of half 0
    auto find = [&](int t0) {
        AttnPlace w;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t pos = min((uint32_t)t0 + 16u * h, (uint32_t)reach - 16u);
            const uint32_t pi = (uint32_t)(((uint64_t)pos * x.page_mul) >> 32) >> x.page_sh;
            w.at[h] = (int)(pos - pi * (uint32_t)a.c.page);
            const int32_t id = table[pi];
            w.ok[h] = id >= 0 && id < a.c.pages;
            w.ph[h] = (int64_t)(w.ok[h] ? id : 0) * a.c.heads + kvh;
        }
        return w;
    };
    auto load = [&](const AttnPlace& w, AttnTile<KB, VB, G>& t) {
        // rows of the (page, head) from which token i of the tile is row i
        const int64_t b0 = w.ph[0] * prow + (int64_t)w.at[0] * G;
        const int64_t b1 = w.ph[1] * prow + (int64_t)(w.at[1] - 16) * G;
        const uint8_t* kp = a.c.kc + (l16 < 8 ? b0 : b1) * (8 * KB) + ka * KROW +
                            (KB == 8 ? 16 : 8) * g;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                const uint8_t* p = kp + 4 * h * KROW + 8 * KB * gr;
                if constexpr (KB == 8) {
                    t.k[h][gr] = *reinterpret_cast<const u32x4_t*>(p);
                } else {
                    const u32x2_t z = *reinterpret_cast<const u32x2_t*>(p);
                    t.k[h][gr >> 1][2 * (gr & 1)] = z.x;
                    t.k[h][gr >> 1][2 * (gr & 1) + 1] = z.y;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < (G + 1) / 2; ++i) {
            const int f = min(lane + 64 * i, 32 * G - 1);
            const int64_t at = (f < 16 * G ? b0 : b1) + f;
            t.sk[i] = a.c.ks[at];
            t.sv[i] = a.c.vs[at];
        }
        // blocks of eight tokens; a block's 64 G values are its columns' 16 G words
        const uint8_t* vp = a.c.vc + (g < 2 ? b0 : b1) * (8 * VB) + (8 * g * G * 16 / 8 + l16) * (4 * VB);
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
            const u32x4_t* p = reinterpret_cast<const u32x4_t*>(vp + gr * 16 * (4 * VB));
            if constexpr (VB == 8) {
                t.v[2 * gr] = p[0];
                t.v[2 * gr + 1] = p[1];
            } else {
                t.v[gr] = p[0];
            }
        }
    };

    const float sc = a.scale * 1.4426950408889634f * KC::kUnit;  // powers of two from here on
    float m = -INFINITY, l = 0.0f;  // head l16; l: this lane's tokens
    float voff[G];                  // this lane's sum of p sV, where the codes are offset
    f32x4_t o[G][4];                // heads 4 g .. 4 g + 3, values 64 gr + 4 l16 + i
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
        voff[gr] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[gr][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
    __shared__ __attribute__((aligned(16))) float sl[kAttnWaves][2][32 * G];
    auto step = [&](int t0, const AttnPlace& w, const AttnTile<KB, VB, G>& t) {
        // the scales of this lane's tokens 8 g + j, [j][group] flat
        f32x4_t sk[2 * G], sv[2 * G];
        lds_wave_sync();  // the last tile's are read
#pragma unroll
        for (int i = 0; i < (G + 1) / 2; ++i)
            if (32 * G >= 64 * (i + 1) || lane < 32) {
                sl[wave][0][lane + 64 * i] = t.sk[i];
                sl[wave][1][lane + 64 * i] = t.sv[i];
            }
        lds_wave_sync();
#pragma unroll
        for (int i = 0; i < 2 * G; ++i) {
            sk[i] = *reinterpret_cast<const f32x4_t*>(&sl[wave][0][8 * G * g + 4 * i]);
            sv[i] = *reinterpret_cast<const f32x4_t*>(&sl[wave][1][8 * G * g + 4 * i]);
        }
        float s[8];  // token 8 g + j
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            f32x4_t r[G];
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                const float c = KC::kOffset ? qoff[gr] : 0.0f;
                r[gr] = f32x4_t{c, c, c, c};
                u32x4_t k0, k1;
                if constexpr (KB == 8) {
                    k0 = key_operand8(t.k[h][gr][0], t.k[h][gr][1]);
                    k1 = key_operand8(t.k[h][gr][2], t.k[h][gr][3]);
                } else {
                    k0 = key_operand4<F32>(t.k[h][gr >> 1][2 * (gr & 1)]);
                    k1 = key_operand4<F32>(t.k[h][gr >> 1][2 * (gr & 1) + 1]);
                }
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    r[gr] = mma(k0, q[p][gr][0], r[gr]);
                    r[gr] = mma(k1, q[p][gr][1], r[gr]);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = (4 * h + j) * G;
                float v = sk[at >> 2][at & 3] * r[0][j];
#pragma unroll
                for (int gr = 1; gr < G; ++gr)
                    v = __builtin_fmaf(sk[(at + gr) >> 2][(at + gr) & 3], r[gr][j], v);
                s[4 * h + j] = v * sc;
            }
        }
        if (t0 < lo || t0 + kAttnTile > n || !w.ok[0] || !w.ok[1]) {
            // what is not there counts as nothing, whatever the memory holds
            const bool ok = g < 2 ? w.ok[0] : w.ok[1];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int pos = t0 + 8 * g + j;
                const bool in = ok && pos >= lo && pos < n;
                s[j] = in ? s[j] : -INFINITY;
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    const int at = j * G + gr;
                    sv[at >> 2][at & 3] = in ? sv[at >> 2][at & 3] : 0.0f;
                }
            }
        }
        float mt = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])),
                         fmaxf(fmaxf(s[4], s[5]), fmaxf(s[6], s[7])));
        mt = fmaxf(m, quad_max(mt));
        const float base = mt == -INFINITY ? 0.0f : mt;
        if (__any(mt != m)) {
            const float al = __builtin_amdgcn_exp2f(m - base);
            l *= al;
            float ao[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) ao[j] = __shfl(al, 4 * g + j);
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                voff[gr] *= al;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[gr][i][j] *= ao[j];
            }
            m = mt;
        }
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            p[j] = __builtin_amdgcn_exp2f(s[j] - base);
            l += p[j];
        }
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
            u32x4_t ap[PP];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                float w0 = p[j] * sv[(j * G + gr) >> 2][(j * G + gr) & 3];
                float w1 = p[j + 1] * sv[((j + 1) * G + gr) >> 2][((j + 1) * G + gr) & 3];
                if constexpr (VC::kOffset) voff[gr] += w0 + w1;
#pragma unroll
                for (int k = 0; k < PP; ++k) {
                    if (k + 1 < PP) {
                        ap[k][j >> 1] = high_pair(w0, w1);
                        w0 -= __uint_as_float(__float_as_uint(w0) & 0xFFFF0000u);
                        w1 -= __uint_as_float(__float_as_uint(w1) & 0xFFFF0000u);
                    } else {
                        ap[k][j >> 1] = bf16_pair(w0, w1);
                    }
                }
            }
            u32x4_t bv[4];
            if constexpr (VB == 8)
                value_operands8(t.v[2 * gr], t.v[2 * gr + 1], bv);
            else
                value_operands4<F32>(t.v[gr], bv);
#pragma unroll
            for (int k = 0; k < PP; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[gr][i] = mma(ap[k], bv[i], o[gr][i]);
        }
    };

    {
        // this wave's tiles, the next two in flight meanwhile; past the last
        // one its loads repeat (a loop without branches around its loads)
        constexpr int kHop = kAttnWaves * kAttnTile;
        const int first = t_begin + wave * kAttnTile;
        if (first < t_end) {
            const int last = first + (t_end - 1 - first) / kHop * kHop;
            AttnTile<KB, VB, G> ta, tb, tc;
            AttnPlace pa = find(first), pb = find(min(first + kHop, last)), pc, pn;
            load(pa, ta);
            load(pb, tb);
            pc = find(min(first + 2 * kHop, last));
            for (int t0 = first;; t0 += 3 * kHop) {
                load(pc, tc);
                pn = find(min(t0 + 3 * kHop, last));
                step(t0, pa, ta);
                if (t0 == last) break;
                pa = pn;
                load(pa, ta);
                pn = find(min(t0 + 4 * kHop, last));
                step(t0 + kHop, pb, tb);
                if (t0 + kHop == last) break;
                pb = pn;
                load(pb, tb);
                pn = find(min(t0 + 5 * kHop, last));
                step(t0 + 2 * kHop, pc, tc);
                if (t0 + 2 * kHop == last) break;
                pc = pn;
            }
        }
    }

    // ---- the waves' parts: a common maximum, then sums in wave order
    __shared__ float ml[kAttnWaves][2][16];
    __shared__ __attribute__((aligned(16))) float red[kAttnWaves][16][W];
    l = quad_sum(l);
    if (lane < 16) {
        ml[wave][0][l16] = m;
        ml[wave][1][l16] = l;
    }
#pragma unroll
    for (int gr = 0; gr < G; ++gr) voff[gr] = VC::kOffset ? -8.0f * quad_sum(voff[gr]) : 0.0f;
#pragma unroll
    for (int gr = 0; gr < G; ++gr)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f32x4_t v;
            const float c = VC::kOffset ? __shfl(voff[gr], 4 * g + j) : 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = (o[gr][i][j] + c) * VC::kUnit;
            *reinterpret_cast<f32x4_t*>(&red[wave][4 * g + j][64 * gr + 4 * l16]) = v;
        }
    __syncthreads();
    for (int i = tid; i < nr * (W / 4); i += 64 * kAttnWaves) {
        const int r = i / (W / 4), d = i % (W / 4) * 4;
        float mx = ml[0][0][r];
#pragma unroll
        for (int w = 1; w < kAttnWaves; ++w) mx = fmaxf(mx, ml[w][0][r]);
        const float base = mx == -INFINITY ? 0.0f : mx;
        float sum = 0.0f;
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kAttnWaves; ++w) {
            const float e = __builtin_amdgcn_exp2f(ml[w][0][r] - base);
            sum += e * ml[w][1][r];
            const f32x4_t z = *reinterpret_cast<const f32x4_t*>(&red[w][r][d]);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = __builtin_fmaf(e, z[k], v[k]);
        }
        if (x.splits > 1) {
            float* out = x.part + ((row0 + r) * x.splits + blockIdx.x) * (W + 2);
#pragma unroll
            for (int k = 0; k < 4; ++k) out[d + k] = v[k];
            if (d == 0) {
                out[W] = mx;
                out[W + 1] = sum;
            }
        } else {
            const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;  // a NaN stays one
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (d + k >= a.c.dim) break;
                const float y = v[k] * inv;
                if constexpr (F32)
                    static_cast<float*>(a.out)[(row0 + r) * a.c.dim + d + k] = y;
                else
                    static_cast<__bf16*>(a.out)[(row0 + r) * a.c.dim + d + k] = (__bf16)y;
            }
            if (d == 0 && a.lse) a.lse[row0 + r] = (mx + __log2f(sum)) * 0.6931471805599453f;
        }
    }
}

template <int KB, int VB, bool F32>
hipError_t attn_width(const AttnKernelArgs& k, dim3 grid, hipStream_t s) {
    switch (k.a.c.groups) {
        case 1: attn_decode_kernel<KB, VB, 1, F32><<<grid, 64 * kAttnWaves, 0, s>>>(k); break;
        case 2: attn_decode_kernel<KB, VB, 2, F32><<<grid, 64 * kAttnWaves, 0, s>>>(k); break;
        case 3: attn_decode_kernel<KB, VB, 3, F32><<<grid, 64 * kAttnWaves, 0, s>>>(k); break;
        default: attn_decode_kernel<KB, VB, 4, F32><<<grid, 64 * kAttnWaves, 0, s>>>(k); break;
    }
    return hipGetLastError();
}

template <bool F32>
hipError_t attn_bits(const AttnKernelArgs& k, hipStream_t s) {
    const dim3 grid((unsigned)k.splits, (unsigned)(k.a.c.heads * k.tiles), (unsigned)k.a.B);
    if (k.a.c.kbits == 4)
        return k.a.c.vbits == 4 ? attn_width<4, 4, F32>(k, grid, s) : attn_width<4, 8, F32>(k, grid, s);
    return k.a.c.vbits == 4 ? attn_width<8, 4, F32>(k, grid, s) : attn_width<8, 8, F32>(k, grid, s);
}

}  // namespace
}  // namespace qt
