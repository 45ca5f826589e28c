// Attention of one new token per sequence over the quantized paged cache: the
// kernel over a chunk of positions, instantiated for bf16 and f32 calls in a
// source of its own each.
//
//   S_t = scale sum_g sK[t,g] sum_j q_j vK[t,j],  p = softmax(S),
//   out_j = sum_t p_t sV[t,g(j)] vV[t,j]
//
// A block owns a chunk of one sequence's positions for one key-value head and
// up to 16 of its query heads; its four or eight waves take tiles of 32 positions in
// turn, each with an online softmax of its own (running base and sum in
// f32), and join them in LDS at the end.  The cache's bytes are read once and
// bound it; both products run on the bf16 matrix cores, whatever the number of
// heads, so that the vector instructions per cache value stay below two.
//
// First product: rows are the queries' values (f32 queries as three exact bf16
// pieces), columns the keys' codes of 16 tokens; each group's sum takes its f32
// scale afterwards.  Row 4 g + r is head 4 r + g, so that the scores of up to 4
// heads come in one register of every lane, 8 in two, 16 in four (NR), and the
// softmax's instructions go by the heads there are.  A lane's two columns of a
// tile are tokens 2 c and 2 c + 1: its probabilities, times the values' scales
// and split into three bf16 pieces (exactly: with two, which are 1 to 4 % faster, one
// bf16 output in 100 to 300 rounded the other way than the exact sum), go to LDS as
// pairs and come back as the second product's operand, whose other side is the values' codes:
// a lane loads eight tokens x four values in one piece (the layout of the
// pages).
//
// A wave's scores are taken relative to a base: eight powers of two above the
// largest one at the time, moved when a score passes it; else a tile costs one
// comparison a score.  No probability is above 1, so that no sum is larger than
// the formula's own, and the largest is not below 2^-8.
//
// bf16 calls take int4 codes as u = v + 8: the nibble is the FP8 (E4M3)
// encoding of u / 512, so a mask and a packed conversion make two operands,
// and the eightfold sums are taken out again (in the keys' product as its
// initial value, in the values' at the end).  f32 calls convert to v itself
// (over a long flat softmax the offset costs more than f32's accuracy).
//
// Measured, this kernel alone: one sequence of 131072 positions, 8 heads of 128
// with 8 queries each, 4 bits: 35.7 us (151 MB, 4.2 TB/s); 64 sequences of up to
// 8192, 8 and 4 bits: 88-92 us (401 MB, 4.4 TB/s), where loads and conversions
// alone take 64; about 9 us of a block are its start, first loads and end.
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
    uint32_t rows, items;       // B heads; rows * splits
    FastDiv page;
    bool q_vec;                 // eight query values may be loaded at once
    float* part;                // splits > 1: [rows][splits] x (G 64 values, base, sum, 2 unused)
};

hipError_t launch_attn_bf16(const AttnKernelArgs& k, hipStream_t s);
hipError_t launch_attn_f32(const AttnKernelArgs& k, hipStream_t s);
hipError_t launch_attn_short(const AttnKernelArgs& k, hipStream_t s);  // kAttnMaxWaves waves

namespace {

constexpr int kAttnTile = 32;
static_assert(kAttnMaxChunk <= 64 * kAttnWaves * kAttnTile, "a wave's tiles are kept one a lane");

// max / sum over a 16-lane row
template <int N>
__device__ __forceinline__ float row_ror(float v) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x120 + N, 0xF, 0xF, false));
}
__device__ __forceinline__ float row_max(float v) {
    v = fmaxf(v, row_ror<8>(v));
    v = fmaxf(v, row_ror<4>(v));
    v = fmaxf(v, row_ror<2>(v));
    return fmaxf(v, row_ror<1>(v));
}
__device__ __forceinline__ float row_sum(float v) {
    v += row_ror<8>(v);
    v += row_ror<4>(v);
    v += row_ror<2>(v);
    return v + row_ror<1>(v);
}
// sum over the four lanes that share l % 16
__device__ __forceinline__ float quad_sum(float v) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const float m = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const uint32_t w = __float_as_uint(m);
    const auto b = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Codes as f32, by the compiler: conversions in inline assembly next to matrix
// instructions would miss the waits that it keeps between a matrix result and
// the next write of its registers.
template <int B>
__device__ __forceinline__ float signed_byte(uint32_t t) {
    return (float)(int8_t)(t >> (8 * B));
}
// nibble N of w, less 8
template <int N>
__device__ __forceinline__ float signed_nibble(uint32_t t) {  // t = w ^ 0x88888888
    return (float)((int32_t)(t << (28 - 4 * N)) >> 28);
}
// the high halves of two f32 values as a bf16 pair
__device__ __forceinline__ uint32_t high_pair(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ uint32_t fp8_pair(uint32_t u, bool hi) {
    return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, 512.0f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(u, 512.0f, false));
}

// What the operand's codes stand for: u = v + 8 (bf16 calls' int4) or v.
template <int BITS, bool F32>
struct Code {
    static constexpr bool kOffset = BITS == 4 && !F32;
};

// Eight key codes as an operand, and which of the eight the operand's value j
// is.
template <bool F32>
__device__ __forceinline__ u32x4_t key_operand4(uint32_t w) {
    if constexpr (F32) {
        const uint32_t t = w ^ 0x88888888u;
        return u32x4_t{high_pair(signed_nibble<0>(t), signed_nibble<1>(t)),
                       high_pair(signed_nibble<2>(t), signed_nibble<3>(t)),
                       high_pair(signed_nibble<4>(t), signed_nibble<5>(t)),
                       high_pair(signed_nibble<6>(t), signed_nibble<7>(t))};
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
__device__ __forceinline__ constexpr int key_order(int j) {
    return BITS == 4 && !F32 ? (j < 4 ? 2 * j : 2 * j - 7) : j;
}

// The codes of eight tokens x four values as four operands.
template <bool F32>
__device__ __forceinline__ void value_operands4(const u32x4_t& w, u32x4_t (&o)[4]) {
#pragma unroll
    for (int a = 0; a < 4; ++a) {  // a pair of tokens
        if constexpr (F32) {
            const uint32_t t = w[a] ^ 0x88888888u;
            o[0][a] = high_pair(signed_nibble<0>(t), signed_nibble<2>(t));
            o[1][a] = high_pair(signed_nibble<1>(t), signed_nibble<3>(t));
            o[2][a] = high_pair(signed_nibble<4>(t), signed_nibble<6>(t));
            o[3][a] = high_pair(signed_nibble<5>(t), signed_nibble<7>(t));
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

// What a tile of 32 positions is read into: the codes of keys 2 c and 2 c + 1
// and the scales of these keys and values, all groups; the codes of eight
// values.
template <int KB, int G>
struct KeyTile {
    u32x4_t k[2][KB == 8 ? G : (G + 1) / 2];  // int4: two groups a word of four
    float sk[2 * G], sv[2 * G];
};
template <int VB, int G>
struct ValueTile {
    u32x4_t v[VB == 8 ? 2 * G : G];
};
// n floats, n = 2, 4, 6 or 8, at 8-byte alignment at least
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float (&v)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const f32x4_t w = reinterpret_cast<const f32x4_t*>(p)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * i + j] = w[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const u32x2_t w = reinterpret_cast<const u32x2_t*>(p)[i];
            v[2 * i] = __uint_as_float(w.x);
            v[2 * i + 1] = __uint_as_float(w.y);
        }
    }
}

// Where a tile lies: the (page, head) and place of its halves of 16 positions.
struct AttnPlace {
    int64_t ph[2];
    int at[2];
    bool ok[2];  // the page exists
};

// A row of probabilities in LDS: 32 tokens of a piece, 16 bytes apart in the banks.
constexpr int kProbRow = 32 * 2 + 16;

// Pieces of a probability times a value's scale: all of its 24 bits.
constexpr int kProbPieces = 3;

// A wave's LDS: the probabilities of its tile; at the end its value sums.
template <int G, int NR>
union AttnWaveLds {
    uint8_t probs[G][kProbPieces][4 * NR][kProbRow];
    float red[4 * NR][G * kGroup];
};

// Waves a SIMD at least: two, but where the LDS of a block is more than half a CU's.
constexpr int attn_waves(int G, int NR, bool f32) { return f32 && G == 4 && NR == 4 ? 1 : 2; }

template <int WAVES, int KB, int VB, int G, int NR, bool F32>
__global__ __launch_bounds__(64 * WAVES) __attribute__((amdgpu_waves_per_eu(attn_waves(G, NR, F32)))) void
attn_decode_kernel(const AttnKernelArgs x) {
    constexpr int kHop = WAVES * kAttnTile;  // to a wave's next tile
    constexpr int NP = F32 ? 3 : 1;   // pieces of a query value
    constexpr int PP = kProbPieces;
    constexpr int KROW = G * 8 * KB, W = G * kGroup;
    constexpr bool kWide = G > 2;  // registers are short: see there
    using KC = Code<KB, F32>;
    using VC = Code<VB, F32>;
    const AttnArgs& a = x.a;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int l16 = lane & 15, g = lane >> 4;
    // Consecutive blocks run on different XCDs, in turn.  Chunks of one index
    // lie together, the first ones first, and each index starts one row further:
    // a long sequence's chunks, and the many short ones' lack of them, spread
    // over the XCDs (with the chunk index fastest, 64 ragged sequences kept one
    // XCD busy all the time and another a tenth of it: 115 against 85 us).  The
    // tiles of one chunk follow each other on one XCD, whose L2 they share.
    const uint32_t lin = blockIdx.y * gridDim.x + blockIdx.x, slot = lin >> 3;
    const int qt = (int)(slot % (uint32_t)x.tiles);
    const uint32_t item = slot / (uint32_t)x.tiles * 8 + (lin & 7);
    if (item >= x.items) return;
    const int split = (int)(item / x.rows);
    const uint32_t row = (item + (uint32_t)split) % x.rows;
    const int kvh = (int)(row % (uint32_t)a.c.heads), b = (int)(row / (uint32_t)a.c.heads);
    const int per = a.q_heads / a.c.heads;
    const int r0 = 16 * qt, nr = min(16, per - r0);  // query heads of this block
    const int64_t row0 = (int64_t)b * a.q_heads + (int64_t)kvh * per + r0;

    // positions lo .. n - 1, this block's from t_begin to t_end
    const int64_t reach = a.table_pages * a.c.page;
    const int n = (int)min<int64_t>(max(a.lens[b], 0), reach);
    const int lo = a.window > 0 && a.window < n ? (int)(n - a.window) : 0;
    const int64_t begin = (lo & ~(kAttnTile - 1)) + (int64_t)split * x.chunk;
    if (begin >= n && split > 0) return;  // the first chunk writes even nothing
    const int t_begin = (int)min<int64_t>(begin, n);
    const int t_end = (int)min<int64_t>(begin + x.chunk, n);

    // ---- the tiles' places and loads
    const int64_t prow = (int64_t)a.c.page * G;  // scales of a (page, head)
    const int32_t* table = a.table + (int64_t)b * a.table_pages;
    const int first = t_begin + wave * kAttnTile;  // this wave's tiles: first + i kHop
    // the places of all of them, tile i in lane i (vector loads once: a scalar
    // load a tile would make every LDS wait wait for it, too)
    int place_id[2], place_at[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t pos = min((uint32_t)(first + lane * kHop) + 16u * h, (uint32_t)reach - 16u);
        const uint32_t pi = x.page.div(pos);
        place_at[h] = (int)(pos - pi * (uint32_t)a.c.page);
        place_id[h] = table[pi];
    }
    auto find = [&](int i) __attribute__((always_inline)) {
        AttnPlace w;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int id = __builtin_amdgcn_readlane(place_id[h], i);
            w.at[h] = __builtin_amdgcn_readlane(place_at[h], i);
            w.ok[h] = id >= 0 && id < a.c.pages;
            w.ph[h] = (int64_t)(w.ok[h] ? id : 0) * a.c.heads + kvh;
        }
        return w;
    };
    // rows of the (page, head) from which token i of the tile is row i
    auto rows_of = [&](const AttnPlace& w, int h) __attribute__((always_inline)) {
        return w.ph[h] * prow + (int64_t)(w.at[h] - 16 * h) * G;
    };
    // Wide heads leave no registers for the lane's part of every address: it is
    // worked out anew for a tile (a value that did not fit would be reloaded
    // in the loop, behind all loads in flight).  Some forms of four groups of 8-bit keys
    // spill all the same at two blocks a CU: up to 12 registers, 40 in bf16 calls
    // of more than eight queries.
    auto here = [&]() __attribute__((always_inline)) {
        int v = lane;
        if constexpr (kWide) asm volatile("" : "+v"(v));
        return v;
    };
    auto load_k = [&](const AttnPlace& w, KeyTile<KB, G>& t) __attribute__((always_inline)) {
        const int at = here(), l16 = at & 15, g = at >> 4;
        const int64_t bk = l16 < 8 ? rows_of(w, 0) : rows_of(w, 1);
        const uint8_t* kp = a.c.kc + bk * (8 * KB) + 2 * l16 * KROW + (KB == 8 ? 16 : 8) * g;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                const uint8_t* p = kp + h * KROW + 8 * KB * gr;
                if constexpr (KB == 8) {
                    t.k[h][gr] = *reinterpret_cast<const u32x4_t*>(p);
                } else {
                    const u32x2_t z = *reinterpret_cast<const u32x2_t*>(p);
                    t.k[h][gr >> 1][2 * (gr & 1)] = z.x;
                    t.k[h][gr >> 1][2 * (gr & 1) + 1] = z.y;
                }
            }
        }
        load_floats(a.c.ks + bk + 2 * l16 * G, t.sk);
        load_floats(a.c.vs + bk + 2 * l16 * G, t.sv);
    };
    auto load_v = [&](const AttnPlace& w, ValueTile<VB, G>& t) __attribute__((always_inline)) {
        const int at = here(), l16 = at & 15, g = at >> 4;
        // blocks of eight tokens; a block's 64 G values are its columns' 16 G words
        const uint8_t* vp = a.c.vc + (g < 2 ? rows_of(w, 0) : rows_of(w, 1)) * (8 * VB) +
                            (g * G * 16 + l16) * (4 * VB);
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

    // the first tile's loads go out before the queries' (a chunk without
    // positions reads a place that is there and counts nothing)
    const int last = max(0, t_end - 1 - first) / kHop;
    KeyTile<KB, G> tk;
    ValueTile<VB, G> tv0, tv1;
    AttnPlace w0 = find(0), w1 = find(min(1, last));
    load_k(w0, tk);
    load_v(w0, tv0);

    // ---- queries as operands: row l16 = 4 i + r is head 4 r + i, values 16 g ..
    // of each group in the order that the codes come in.  All waves' are the same:
    // those of wide heads lie in LDS, a group made by a wave each, so that the
    // registers leave room for two blocks a CU.
    static_assert(!kWide || G <= WAVES, "a wave a group");
    __shared__ u32x4_t ql[kWide ? NP : 1][kWide ? G : 1][2][64];
    __shared__ __attribute__((aligned(16))) float qsum[G][16];
    u32x4_t q[NP][kWide ? 1 : G][2];
    // -8 times the group's sum of head 4 r + g, where the codes are offset
    float qoff[NR][kWide ? 1 : G];
    auto query = [&](int gr, u32x4_t (&to)[NP][2]) __attribute__((always_inline)) {
        const int64_t head = (int64_t)kvh * per + r0 + min(4 * (l16 & 3) + (l16 >> 2), nr - 1);
        const int64_t at = (int64_t)b * a.ldq + head * a.c.dim;
        float sum = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int d0 = 64 * gr + 16 * g + 8 * h;
            uint32_t v[8];  // the eight values' bits, in order
            if (x.q_vec) {  // eight values lie wholly inside or outside the head
                const bool in = d0 < a.c.dim;
                const int64_t i = at + (in ? d0 : 0);
                if constexpr (F32) {
                    const u32x4_t* z =
                        reinterpret_cast<const u32x4_t*>(static_cast<const float*>(a.Q) + i);
                    const u32x4_t z0 = z[0], z1 = z[1];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = in ? (j < 4 ? z0[j & 3] : z1[j & 3]) : 0u;
                } else {
                    const u32x4_t z = *reinterpret_cast<const u32x4_t*>(
                        static_cast<const uint16_t*>(a.Q) + i);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[j] = in ? (j & 1 ? z[j >> 1] >> 16 : z[j >> 1] & 0xFFFFu) : 0u;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int64_t i = at + min(d0 + j, a.c.dim - 1);
                    const uint32_t z = F32 ? static_cast<const uint32_t*>(a.Q)[i]
                                           : (uint32_t)static_cast<const uint16_t*>(a.Q)[i];
                    v[j] = d0 + j < a.c.dim ? z : 0u;
                }
            }
            uint32_t p[NP][8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t z = v[key_order<KB, F32>(j)];
                if constexpr (F32) {
                    split3(__uint_as_float(z), p[0][j], p[NP > 1 ? 1 : 0][j], p[NP > 1 ? 2 : 0][j]);
                } else {
                    p[0][j] = z;
                    sum += __uint_as_float(z << 16);
                }
            }
#pragma unroll
            for (int k = 0; k < NP; ++k)
                to[k][h] = u32x4_t{p[k][0] | p[k][1] << 16, p[k][2] | p[k][3] << 16,
                                   p[k][4] | p[k][5] << 16, p[k][6] | p[k][7] << 16};
        }
        return quad_sum(sum);  // of row l16, in every lane of the column
    };
    if constexpr (kWide) {
        if (wave < G) {
            u32x4_t to[NP][2];
            const float sum = query(wave, to);
#pragma unroll
            for (int k = 0; k < NP; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) ql[k][wave][h][lane] = to[k][h];
            if (g == 0) qsum[wave][l16] = -8.0f * sum;
        }
        __syncthreads();
    } else {
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
            u32x4_t to[NP][2];
            const float sum = query(gr, to);
#pragma unroll
            for (int k = 0; k < NP; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h) q[k][gr][h] = to[k][h];
#pragma unroll
            for (int r = 0; r < NR; ++r)
                qoff[r][gr] = KC::kOffset ? -8.0f * __shfl(sum, 4 * g + r) : 0.0f;
        }
    }

    const float sc = a.scale * 1.4426950408889634f;  // powers of two from here on
    constexpr float kRoom = 8.0f;  // of a new base above the largest score
    float m[NR], l[NR];            // head 4 r + g: bases, sums of this lane's tokens
    float voff[NR][G];              // this lane's sum of p sV, where the codes are offset
    f32x4_t o[G][4];                // heads 4 g .. 4 g + 3, values 64 gr + 4 l16 + i
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.0f;
#pragma unroll
        for (int gr = 0; gr < G; ++gr) voff[r][gr] = 0.0f;
    }
#pragma unroll
    for (int gr = 0; gr < G; ++gr)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[gr][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    __shared__ __attribute__((aligned(16))) AttnWaveLds<G, NR> lds[WAVES];
    // scores of the tile in tk: token 2 l16 + h, head 4 r + g
    auto scores = [&](float (&s)[2][NR]) __attribute__((always_inline)) {
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
            u32x4_t qa[NP][2];
#pragma unroll
            for (int p = 0; p < NP; ++p)
#pragma unroll
                for (int i = 0; i < 2; ++i) qa[p][i] = kWide ? ql[p][gr][i][lane] : q[p][gr][i];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x4_t d = {0.f, 0.f, 0.f, 0.f};
                if constexpr (KC::kOffset) {
                    if constexpr (kWide)
                        d = *reinterpret_cast<const f32x4_t*>(&qsum[gr][4 * g]);
                    else
#pragma unroll
                        for (int r = 0; r < NR; ++r) d[r] = qoff[r][gr];
                }
                u32x4_t k0, k1;
                if constexpr (KB == 8) {
                    k0 = key_operand8(tk.k[h][gr][0], tk.k[h][gr][1]);
                    k1 = key_operand8(tk.k[h][gr][2], tk.k[h][gr][3]);
                } else {
                    k0 = key_operand4<F32>(tk.k[h][gr >> 1][2 * (gr & 1)]);
                    k1 = key_operand4<F32>(tk.k[h][gr >> 1][2 * (gr & 1) + 1]);
                }
#pragma unroll
                for (int p = 0; p < NP; ++p) {
                    d = mma(qa[p][0], k0, d);
                    d = mma(qa[p][1], k1, d);
                }
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float f = tk.sk[h * G + gr] * sc;
                    s[h][r] = gr == 0 ? f * d[r] : __builtin_fmaf(f, d[r], s[h][r]);
                }
            }
            if constexpr (kWide) __builtin_amdgcn_sched_barrier(0);
        }
    };
    // the tile's probabilities, times the values' scales, to LDS
    auto weigh = [&](int t0, const AttnPlace& w, float (&s)[2][NR], float (&sv)[2 * G]) __attribute__((always_inline)) {
        if (t0 < lo || t0 + kAttnTile > n || !w.ok[0] || !w.ok[1]) {
            // what is not there counts as nothing, whatever the memory holds
            const bool ok = l16 < 8 ? w.ok[0] : w.ok[1];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int pos = t0 + 2 * l16 + h;
                const bool in = ok && pos >= lo && pos < n;
#pragma unroll
                for (int r = 0; r < NR; ++r) s[h][r] = in ? s[h][r] : -INFINITY;
#pragma unroll
                for (int gr = 0; gr < G; ++gr) sv[h * G + gr] = in ? sv[h * G + gr] : 0.0f;
            }
        }
        bool past = false;
#pragma unroll
        for (int r = 0; r < NR; ++r) past |= fmaxf(s[0][r], s[1][r]) > m[r];
        if (__any(past)) {
            float al[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float top = row_max(fmaxf(s[0][r], s[1][r]));
                const float mt = top > m[r] ? top + kRoom : m[r];
                al[r] = mt == m[r] ? 1.0f : __builtin_amdgcn_exp2f(m[r] - mt);
                m[r] = mt;
                l[r] *= al[r];
#pragma unroll
                for (int gr = 0; gr < G; ++gr) voff[r][gr] *= al[r];
            }
            // head 4 g + j: register g of lane row j
            float ao[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ao[j] = __shfl(al[0], 16 * j);
#pragma unroll
                for (int r = 1; r < NR; ++r) {
                    const float v = __shfl(al[r], 16 * j);
                    ao[j] = g == r ? v : ao[j];
                }
            }
#pragma unroll
            for (int gr = 0; gr < G; ++gr)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[gr][i][j] *= ao[j];
        }
        lds_wave_sync();  // the last tile's probabilities are read
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const float base = m[r] == -INFINITY ? 0.0f : m[r];
            const float p0 = __builtin_amdgcn_exp2f(s[0][r] - base);
            const float p1 = __builtin_amdgcn_exp2f(s[1][r] - base);
            l[r] += p0 + p1;
#pragma unroll
            for (int gr = 0; gr < G; ++gr) {
                float y0 = p0 * sv[gr], y1 = p1 * sv[G + gr];
                if constexpr (VC::kOffset) voff[r][gr] += y0 + y1;
#pragma unroll
                for (int k = 0; k < PP; ++k) {
                    uint32_t pair;
                    if (k + 1 < PP) {
                        pair = high_pair(y0, y1);
                        y0 -= __uint_as_float(__float_as_uint(y0) & 0xFFFF0000u);
                        y1 -= __uint_as_float(__float_as_uint(y1) & 0xFFFF0000u);
                    } else {
                        pair = bf16_pair(y0, y1);
                    }
                    *reinterpret_cast<uint32_t*>(&lds[wave].probs[gr][k][4 * r + g][4 * l16]) = pair;
                }
            }
        }
        lds_wave_sync();
    };
    // the second product of the tile in tv
    auto values = [&](const ValueTile<VB, G>& tv) __attribute__((always_inline)) {
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
            u32x4_t ap[PP];
#pragma unroll
            for (int k = 0; k < PP; ++k)  // rows past the heads repeat one that is there
                ap[k] = *reinterpret_cast<const u32x4_t*>(
                    &lds[wave].probs[gr][k][l16 % (4 * NR)][16 * g]);
            u32x4_t bv[4];
            if constexpr (VB == 8)
                value_operands8(tv.v[2 * gr], tv.v[2 * gr + 1], bv);
            else
                value_operands4<F32>(tv.v[gr], bv);
#pragma unroll
            for (int k = 0; k < PP; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[gr][i] = mma(ap[k], bv[i], o[gr][i]);
        }
    };

    if (first < t_end) {
        // Tile i's second product runs next to tile i + 1's first one, which
        // does not depend on it; loads are a whole tile ahead (past the last
        // one they repeat: no branches around them).
        float s[2][NR], sv[2 * G];
        auto take = [&](const AttnPlace& next) __attribute__((always_inline)) {  // the tile in tk; then the next one's loads
            scores(s);
#pragma unroll
            for (int i = 0; i < 2 * G; ++i) sv[i] = tk.sv[i];
            load_k(next, tk);
            if constexpr (kWide) __builtin_amdgcn_sched_barrier(0);
        };
        take(w1);
        weigh(first, w0, s, sv);
        // wa: the place of tile i + 1
        auto turn = [&](int i, AttnPlace& wa, const ValueTile<VB, G>& now, ValueTile<VB, G>& next) __attribute__((always_inline)) {
            if constexpr (!kWide) load_v(wa, next);
            const AttnPlace wb = find(min(i + 2, last));
            take(wb);
            values(now);
            if constexpr (kWide) {  // now and next are one: not before its last use
                __builtin_amdgcn_sched_barrier(0);
                load_v(wa, next);
            }
            weigh(first + (i + 1) * kHop, wa, s, sv);
            wa = wb;
        };
        if constexpr (kWide) {
            for (int i = 0; i < last; ++i) turn(i, w1, tv0, tv0);
            values(tv0);
        } else {
            int i = 0;
            for (; i + 1 < last; i += 2) {
                turn(i, w1, tv0, tv1);
                turn(i + 1, w1, tv1, tv0);
            }
            if (i < last) {
                turn(i, w1, tv0, tv1);
                values(tv1);
            } else {
                values(tv0);
            }
        }
    }

    // ---- the waves' parts: a common base, then sums in wave order
    __shared__ float ml[WAVES][2][16];
    __shared__ float vo[WAVES][G][16];  // what the values' codes are offset by
    __syncthreads();  // every wave is done with its probabilities
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        l[r] = row_sum(l[r]);
        if (l16 == 0) {
            ml[wave][0][4 * r + g] = m[r];
            ml[wave][1][4 * r + g] = l[r];
        }
#pragma unroll
        for (int gr = 0; gr < G; ++gr)
            if constexpr (VC::kOffset) {
                const float v = row_sum(voff[r][gr]);
                if (l16 == 0) vo[wave][gr][4 * r + g] = -8.0f * v;
            } else {
                if (l16 == 0) vo[wave][gr][4 * r + g] = 0.0f;
            }
    }
    if (g < NR) {  // heads 4 g + j that there may be
#pragma unroll
        for (int gr = 0; gr < G; ++gr)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<f32x4_t*>(&lds[wave].red[4 * g + j][64 * gr + 4 * l16]) =
                    f32x4_t{o[gr][0][j], o[gr][1][j], o[gr][2][j], o[gr][3][j]};
    }
    __syncthreads();
    for (int i = tid; i < nr * (W / 4); i += 64 * WAVES) {
        const int r = i / (W / 4), d = i % (W / 4) * 4;
        float mx = ml[0][0][r];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) mx = fmaxf(mx, ml[w][0][r]);
        const float base = mx == -INFINITY ? 0.0f : mx;
        float sum = 0.0f;
        f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float e = __builtin_amdgcn_exp2f(ml[w][0][r] - base);
            sum += e * ml[w][1][r];
            const f32x4_t z = *reinterpret_cast<const f32x4_t*>(&lds[w].red[r][d]);
            const float c = vo[w][d >> 6][r];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = __builtin_fmaf(e, z[k] + c, v[k]);
        }
        if (x.splits > 1) {
            float* out = x.part + ((row0 + r) * x.splits + split) * (W + 4);
            *reinterpret_cast<f32x4_t*>(out + d) = v;
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

template <int WAVES, int KB, int VB, int G, bool F32>
void attn_heads(const AttnKernelArgs& k, dim3 grid, hipStream_t s) {
    const int per = k.a.q_heads / k.a.c.heads;
    if (per <= 4)
        attn_decode_kernel<WAVES, KB, VB, G, 1, F32><<<grid, 64 * WAVES, 0, s>>>(k);
    else if (per <= 8)
        attn_decode_kernel<WAVES, KB, VB, G, 2, F32><<<grid, 64 * WAVES, 0, s>>>(k);
    else
        attn_decode_kernel<WAVES, KB, VB, G, 4, F32><<<grid, 64 * WAVES, 0, s>>>(k);
}

template <int WAVES, int KB, int VB, bool F32>
hipError_t attn_width(const AttnKernelArgs& k, dim3 grid, hipStream_t s) {
    if (k.a.c.groups == 1) {
        attn_heads<WAVES, KB, VB, 1, F32>(k, grid, s);
    } else if (k.a.c.groups == 2) {
        attn_heads<WAVES, KB, VB, 2, F32>(k, grid, s);
    } else if constexpr (WAVES == kAttnWaves) {
        if (k.a.c.groups == 3)
            attn_heads<WAVES, KB, VB, 3, F32>(k, grid, s);
        else
            attn_heads<WAVES, KB, VB, 4, F32>(k, grid, s);
    } else {
        return hipErrorInvalidValue;  // the plan takes four waves here
    }
    return hipGetLastError();
}

template <int WAVES, bool F32>
hipError_t attn_bits(const AttnKernelArgs& k, hipStream_t s) {
    const uint32_t blocks = (k.items + 7) / 8 * 8 * (uint32_t)k.tiles;  // below 2^31
    const uint32_t gx = std::min<uint32_t>(blocks, 1u << 20);
    const dim3 grid(gx, (blocks + gx - 1) / gx);
    if (k.a.c.kbits == 4)
        return k.a.c.vbits == 4 ? attn_width<WAVES, 4, 4, F32>(k, grid, s)
                                : attn_width<WAVES, 4, 8, F32>(k, grid, s);
    return k.a.c.vbits == 4 ? attn_width<WAVES, 8, 4, F32>(k, grid, s)
                            : attn_width<WAVES, 8, 8, F32>(k, grid, s);
}

}  // namespace
}  // namespace qt
