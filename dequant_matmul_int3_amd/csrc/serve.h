// Internal interface between the C-ABI layer of the serving calls
// (api_serve.cpp) and their kernels, and the host rules that choose forms and
// size workspaces.  Arguments here are already validated.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "qt_internal.h"

namespace qt {

constexpr int64_t kServeMaxTokens = int64_t(1) << 22;
// pages * page: positions and a block's tiles past them in 31 bits
constexpr int64_t kKvMaxSlots = (int64_t(1) << 31) - (1 << 16);
constexpr int64_t kKvMaxPage = 65536;
constexpr int64_t kKvMaxHeads = 1024;
constexpr int64_t kKvMaxDim = 256;
constexpr int64_t kAttnMaxBatch = 65535;
constexpr int64_t kAttnMaxGroupHeads = 256;  // query heads per key-value head
constexpr int64_t kAttnMaxChunk = 2048;
constexpr int kAttnWaves = 4, kAttnMaxWaves = 8;  // of a block

// x / d for x < 2^31 as a product: mul = ceil(2^(32 + sh) / d) with
// 2^sh < d <= 2^(sh + 1), so that mul < 2^32 and the excess x / 2^(32 + sh) is
// below 1 / d.
struct FastDiv {
    uint32_t d, mul, sh;
    __host__ __device__ static FastDiv of(uint32_t d) {
        FastDiv f{d, 0, 0};
        while ((uint64_t(2) << f.sh) < d) ++f.sh;
        if (d > 1) f.mul = (uint32_t)(((uint64_t(1) << (32 + f.sh)) + d - 1) / d);
        return f;
    }
    __host__ __device__ uint32_t div(uint32_t x) const {
        return d > 1 ? (uint32_t)(((uint64_t)x * mul) >> 32) >> sh : x;
    }
};

// A paged cache: codes [pages][heads][page][groups * 8 bits] and scales
// [pages][heads][page][groups] of the keys and of the values.
struct KvCache {
    uint8_t* kc;
    float* ks;
    int kbits;
    uint8_t* vc;
    float* vs;
    int vbits;
    int64_t pages;
    int page, heads, dim, groups;
};

struct KvRows {  // of one call: [T x heads x dim], rows ld elements apart
    const void* K;
    int64_t ldk;
    const void* V;
    int64_t ldv;
    bool bf16;
};
hipError_t launch_kv_write(const KvCache& c, const KvRows& r, const int32_t* slots, int64_t T,
                           hipStream_t s);
hipError_t launch_kv_read(const KvCache& c, const int32_t* slots, int64_t R, void* K, void* V,
                          bool bf16, hipStream_t s);

struct AttnArgs {
    KvCache c;
    const void* Q;  // [B x q_heads x dim], rows ldq elements apart
    int64_t ldq;
    bool bf16;
    int B, q_heads;
    const int32_t* table;  // [B x table_pages]
    int64_t table_pages;
    const int32_t* lens;   // [B]
    int64_t window;        // 0: everything
    float scale;
    void* out;             // [B x q_heads x dim]
    float* lse;            // [B x q_heads] or null
};

// How the positions are cut: chunks of `chunk` positions, `splits` of them at
// most; more than one leaves partial results in the workspace, which a second
// launch joins.  A short context that would be cut into a few chunks goes to one
// block of eight waves instead (700 positions, 8 heads: 10.6 us where chunks of
// 256 took 6.7 and their join 3.8 and a launch more; of 1530 positions 19.5 us
// against 12.1 and 3.6).  Wide heads need more registers than eight waves have.
struct AttnPlan {
    int waves, chunk, splits;
    int64_t bytes;
};
inline AttnPlan attn_plan(int64_t B, int64_t heads, int64_t q_heads, int64_t dim,
                          int64_t table_pages, int64_t page, int64_t window) {
    constexpr int64_t kStep = 128;      // four waves of 32 positions
    // Two blocks for every CU, which are in flight together; shorter chunks pay
    // where wide heads make them slow and lengths differ (24 sequences of up to
    // 12000 positions, 256 values: 44.8 against 52.5 us, of equal lengths 67.9
    // against 68.3; of 128 values 8 sequences take 31.5 us against 30.2).
    const int64_t G = (dim + kGroup - 1) / kGroup;
    const int64_t blocks = G > 2 ? 768 : 512;
    constexpr int64_t kOne = 1024;      // up to here eight waves take all of it
    int64_t span = table_pages * page;
    // a window may start inside a tile of 32
    if (window) span = std::min(span, std::min(window, span) + 31);
    const int64_t tiles = (q_heads / heads + 15) / 16;
    const int64_t rows = B * heads * tiles;
    const int64_t want = std::max<int64_t>(1, (blocks + rows - 1) / rows);
    int64_t chunk = (span + want - 1) / want;
    chunk = (chunk + kStep - 1) / kStep * kStep;
    chunk = std::min<int64_t>(std::max<int64_t>(chunk, 2 * kStep), kAttnMaxChunk);
    AttnPlan p;
    p.waves = kAttnWaves;
    if (chunk < span && span <= kOne && G <= 2) {
        p.waves = kAttnMaxWaves;
        chunk = (span + kStep - 1) / kStep * kStep;
    }
    p.chunk = (int)chunk;
    p.splits = (int)std::max<int64_t>(1, (span + chunk - 1) / chunk);
    p.bytes = p.splits == 1 ? 0 : B * q_heads * p.splits * (G * kGroup + 4) * 4;
    return p;
}
// Blocks of the first launch, which are numbered in 31 bits.
inline bool attn_fits(const AttnPlan& p, int64_t B, int64_t heads, int64_t q_heads) {
    return (B * heads * p.splits + 7) / 8 * 8 * ((q_heads / heads + 15) / 16) < (int64_t(1) << 31) &&
           B * q_heads < (int64_t(1) << 24);  // blocks of 256 threads of the second
}
hipError_t launch_attn_decode(const AttnArgs& a, void* workspace, hipStream_t s);

// ------------------------------------------- expert layer for a few tokens
constexpr int kFewMaxTokens = 16;
constexpr int kFewMaxTopK = 32;
constexpr int kFewMaxExperts = 512;
constexpr int64_t kFewMaxDim = int64_t(1) << 20;
constexpr int64_t kFewLong = 1000000000;  // see few_long

struct FewMat {
    const uint8_t* packed;  // [E][rows x groups] packed groups
    const float* scales;
    int bits;
};
struct FewArgs {
    const void* X;  // [T x D]
    bool bf16;
    int T, E, k, act;
    int64_t D, F;
    const float* logits;  // [T x E]
    FewMat gate, up, down;
    void* out;  // [T x D]
};

// Workspace: the routing of the call, then the activations of the pairs as three bf16
// pieces, all of their 24 bits: [pieces][pairs][groups of F x 64].
constexpr int kFewPieces = 3;
constexpr int64_t few_align(int64_t b) { return (b + 15) / 16 * 16; }
struct FewPlan {
    int64_t pairs, fp;        // pairs at most, F padded to whole groups
    int64_t pair, planes;     // offsets of the parts in bytes; the experts are first
    int64_t bytes;
};
inline FewPlan few_plan(int64_t T, int64_t k, int64_t F) {
    FewPlan p;
    p.pairs = T * k;
    p.fp = (F + kGroup - 1) / kGroup * kGroup;
    // the number of active experts (16 bytes) and each one's expert and first
    // pair; then the pairs' tokens and weights
    p.pair = 16 + few_align(p.pairs * 4);
    p.planes = p.pair + few_align(p.pairs * 8);
    p.bytes = p.planes + kFewPieces * p.pairs * p.fp * 2;
    return p;
}
// Long streams of weights, and many tokens, go through the launches of the full
// layer: its blocks read 3.6 TB/s and take five tokens an expert at once, where the
// two launches above reach 3.0 and slow down with an expert's tokens; but they
// are five (seven with a bf16 call's conversions) and cost 20 to 35 us more for few
// experts.  Measured by bytes times tokens (int3, us a call: bf16 through the two
// launches / the layer's with its conversions; f32 likewise, the two launches of large
// ones with rows off 16 bytes, which cost them up to a tenth):
//   10^9   experts, k             T   bf16         f32
//   0.07   128 of 2048 x 768, 8   2    27 /  47     27 /  42
//   0.26   the same               4    44 /  51     46 /  45
//   0.36   64 of 2048 x 1408, 6   4    47 /  52     48 /  47
//   0.62   128 of 7168 x 2048, 8  2    90 / 106     99 / 101
//   0.62   8 of 4096 x 14336, 2   2    80 / 116     84 / 112
//   1.06   128 of 2048 x 768, 8   8    72 /  63     88 /  58
//   1.23   16 of 8192 x 7168, 4   2   169 / 172    206 / 167
//   1.45   64 of 2048 x 1408, 6   8    80 /  65    101 /  62
//   2.47   128 of 7168 x 2048, 8  4   172 / 174    215 / 170
//   2.47   8 of 4096 x 14336, 2   4   159 / 159    174 / 154
//   2.77   16 of 8192 x 7168, 4   3   225 / 216    277 / 211
//   22.2   128 of 7168 x 2048, 8  12  419 / 343    698 / 346
// The layer takes SiLU, widths that are multiples of 128 and f32 rows aligned to 16
// bytes; other calls pay the difference above.
inline int64_t few_stream(int64_t T, int64_t k, int64_t E, int64_t D, int64_t F, int gate_bits,
                          int up_bits, int down_bits) {
    auto group = [](int bits) { return bits == 3 ? 28 : 36; };  // bytes, scale included
    return std::min(T * k, E) * (F * ((D + kGroup - 1) / kGroup) * (group(gate_bits) + group(up_bits)) +
                                 D * ((F + kGroup - 1) / kGroup) * group(down_bits));
}
inline bool few_long(int64_t T, int64_t k, int64_t E, int64_t D, int64_t F, int gate_bits,
                     int up_bits, int down_bits) {
    return D % 128 == 0 && F % 128 == 0 &&
           T * few_stream(T, k, E, D, F, gate_bits, up_bits, down_bits) >= kFewLong;
}
// The full layer's workspace, after it a bf16 call's tokens and outputs in f32.
inline int64_t few_long_bytes(int64_t T, int64_t k, int64_t E, int64_t D, int64_t F, bool bf16) {
    return few_align((int64_t)moe_layer_workspace(T, k, E, D, F)) + (bf16 ? 2 * few_align(T * D * 4) : 0);
}
inline int64_t few_workspace(int64_t T, int64_t k, int64_t E, int64_t D, int64_t F, bool bf16) {
    const int64_t n = few_plan(T, k, F).bytes;
    return few_long(T, k, E, D, F, 4, 4, 4) ? std::max(n, few_long_bytes(T, k, E, D, F, bf16)) : n;
}
hipError_t launch_moe_few(const FewArgs& a, void* workspace, hipStream_t s);

}  // namespace qt
