// The expert layer for a few tokens (up to 16), in two launches unless the weights'
// stream is long:
//   1. h = act(Wgate_e x_t) * (Wup_e x_t) for every pair of a token and one of
//      its k experts;
//   2. out_t = sum_e w_te Wdown_e h_te.
// The weights' stream is what both cannot do without.  Of 128 experts of 7168 x 2048,
// int3, k = 8, one token takes 36 + 24 us (2.9 and 2.1 TB/s).  In the first launch
// the stream (103 MB, 15 to 20 us) and its unpacking (2.7 vector instructions a code,
// 17 us) come one after the other more than at once: a block is one tile there, and
// its first weights are loaded after the routing.  The second waits for a
// wave's few chunks.  Twelve tokens (68 experts live) take 419 us a call through the two
// launches, 343 through the full layer's: such streams go there (few_long).  Codes enter the bf16 matrix cores exactly, each group's
// products are summed in f32 and scaled by the group's f32 scale.  (Codes as they
// lie, as FP4 operands next to inputs in FP8 pieces, save the unpacking; but the
// products are not summed exactly there, f32 outputs came out 1.7e-5 off, and the
// pieces of the inputs cost what the unpacking did.)
//
// Every block of the first launch routes all tokens by itself (a wave a token: k
// rounds of a maximum over the wave), which costs less than a launch of its
// own; block 0 leaves the routing for the second one.
#include "lds_barrier.h"
#include "serve.h"
#include "unpack.h"

namespace qt {
namespace {

constexpr int kUpWaves = 4, kDownWaves = 8;
// Groups of a chunk, a wave's unit of work.
constexpr int kUpCG = 4, kDownCG = 8;
constexpr int kRoundGroups = kUpWaves * kUpCG;
// Tokens of a pass at most, and the inputs staged at a time: their rows (an f32
// token has three) of at least 16 groups (a round of the waves' chunks), rows 16
// bytes apart in the banks.  With eight rows four blocks fit a CU, which pays more
// than the second pass (from the caches) of an expert with more tokens costs: twelve
// tokens' 68 experts of 7168 x 2048 took 310 us with twelve rows, 296 with eight.
template <bool BF16>
constexpr int kPassTokens = BF16 ? 8 : 4;
template <bool BF16>
constexpr int kPassRows = BF16 ? kPassTokens<true> : 3 * kPassTokens<false>;
template <bool BF16>
constexpr int kSlabBytes = kPassRows<BF16> * (kRoundGroups * 128 + 16);

// Weights of 16 rows come in 16-byte pieces, consecutive lanes on consecutive
// pieces of a row, and go through LDS of the wave's own: lane 16 h + r reads its
// 16 codes of a group of row r from there (a lane loading its row's groups
// itself touches a line of its own with every load, which the address path of
// the caches takes one after the other).  Rows are 16 bytes apart in the banks:
// conflict-free.
template <int BITS, int CG>
struct Tile {
    static constexpr int kGB = BITS == 3 ? kGroupBytes : kGroupBytesI4;
    static constexpr int kRow = CG * kGB;        // bytes of a row's chunk
    static constexpr int kPitch = kRow + 16;
    static constexpr int kParts = kRow / 16;     // pieces of a row
    static constexpr int kPieces = 16 * kParts;  // of the tile
    static_assert(kRow % 16 == 0, "whole pieces");
    // the 16 codes of lane (row, h4) of group j
    static __device__ __forceinline__ Quarter quarter(const uint8_t* tile, int j, int h4, int row) {
        const uint8_t* p = tile + row * kPitch + j * kGB;
        if constexpr (BITS == 3)
            return Quarter{*reinterpret_cast<const uint32_t*>(p + 4 * h4),
                           *reinterpret_cast<const uint32_t*>(p + 16 + 4 * (h4 >> 1))};
        const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p + 8 * h4);
        return Quarter{w.x, w.y};
    }
};
typedef u32x4_t u32x4_g __attribute__((aligned(8)));  // rows of an odd number of groups
// 16 bytes of which the last 8 or all may lie past the row (zeros then)
__device__ __forceinline__ u32x4_t piece(const uint8_t* p, int left) {
    if (left >= 16) return *reinterpret_cast<const u32x4_g*>(p);
    if (left < 8) return u32x4_t{0u, 0u, 0u, 0u};
    const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p);
    return u32x4_t{w.x, w.y, 0u, 0u};
}

struct FewKernelArgs {
    FewArgs a;
    int GD, GF;          // groups of D and of F
    int pairs;           // T k
    int32_t* count;      // active experts; from 4 on: expert | first pair << 16 of each
    int32_t* token;      // [pairs] token of a pair; pairs go by expert, then token
    float* weight;       // [pairs] weight of a pair
    uint16_t* planes;    // [pieces][pairs][64 GF]
    bool x_vec;          // eight inputs may be loaded at once
    int slab;            // bytes of the staged inputs
};

// A logit's bits made monotone as an unsigned number, above 0 (-0 as +0).
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return max((u & 0x80000000u) ? ~u : (u | 0x80000000u), 1u);
}
__device__ __forceinline__ float key_value(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
template <int N>
__device__ __forceinline__ uint32_t ror_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + N, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t wave_max_key(uint32_t v) {
    v = ror_max<8>(v);
    v = ror_max<4>(v);
    v = ror_max<2>(v);
    v = ror_max<1>(v);
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(a[0], a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max(b[0], b[1]);
}
// inclusive sum over the lanes up to this one
template <int CTRL, int ROWS>
__device__ __forceinline__ int add_dpp(int v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, true);
}
__device__ __forceinline__ int wave_scan(int v) {
    v = add_dpp<0x111, 0xF>(v);  // row_shr 1, 2, 4, 8
    v = add_dpp<0x112, 0xF>(v);
    v = add_dpp<0x114, 0xF>(v);
    v = add_dpp<0x118, 0xF>(v);
    v = add_dpp<0x142, 0xA>(v);  // a row's last lane to the next row
    return add_dpp<0x143, 0xC>(v);  // lane 31 to the upper half
}

// The routing of all tokens in LDS.
struct Route {
    uint32_t mask[kFewMaxExperts];   // tokens of an expert
    uint32_t act[kFewMaxTokens * kFewMaxTopK];  // active experts, ascending: expert, first pair << 16
    int32_t n;
};
// What only the routing itself needs, and block 0.
struct Picks {
    int32_t sel[kFewMaxTokens][kFewMaxTopK];
    float wgt[kFewMaxTokens][kFewMaxTopK];
};

// M: experts per lane (E <= 64 M)
template <int M>
__device__ __forceinline__ void route(const FewKernelArgs& x, Route& r, Picks& c) {
    const FewArgs& a = x.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int E = a.E, k = a.k;
    for (int e = tid; e < E; e += 64 * kUpWaves) r.mask[e] = 0;
    __syncthreads();
    for (int t = wave; t < a.T; t += kUpWaves) {
        uint32_t key[M];
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int e = lane + 64 * m;
            const float v = a.logits[(int64_t)t * E + min(e, E - 1)];
            key[m] = e < E ? key_of(v) : 0u;  // below every real key
        }
        float top = 0.0f, sum = 0.0f, mine = 0.0f;
        for (int j = 0; j < k; ++j) {
            uint32_t best = key[0];
#pragma unroll
            for (int m = 1; m < M; ++m) best = max(best, key[m]);
            best = wave_max_key(best);
            // the lowest expert that has it
            int id = -1;
#pragma unroll
            for (int m = M - 1; m >= 0; --m) {
                const uint64_t b = __ballot(key[m] == best);
                if (b) id = 64 * m + __ffsll((unsigned long long)b) - 1;
            }
#pragma unroll
            for (int m = 0; m < M; ++m)
                if (lane + 64 * m == id) key[m] = 0u;
            const float v = key_value(best);
            if (j == 0) top = v;
            const float e = expf(v - top);
            sum += e;
            if (lane == j) mine = e;
            if (lane == 0) {
                c.sel[t][j] = id;
                atomicOr(&r.mask[id], 1u << t);
            }
        }
        if (lane < k) c.wgt[t][lane] = mine / sum;
    }
    __syncthreads();
    if (wave == 0) {  // active experts and their first pairs
        int n = 0, p = 0;
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int e = 64 * m + lane;
            const uint32_t who = e < E ? r.mask[e] : 0u;
            const uint64_t b = __ballot(who != 0);
            const int inc = wave_scan(__popc(who));
            if (who)
                r.act[n + __popcll(b & ((1ull << lane) - 1))] =
                    (uint32_t)e | (uint32_t)(p + inc - __popc(who)) << 16;
            n += __popcll(b);
            p += __builtin_amdgcn_readlane(inc, 63);
        }
        if (lane == 0) r.n = n;
    }
    __syncthreads();
}

// Sixteen codes as two exact operands: v for int3 (the byte table and packed
// conversion of exact_quarter, without its reordering), 16 v for int4 (the
// nibbles of a word as the high halves of signed bytes).  Both come in the
// order 0 4 1 5 2 6 3 7 within each eight, which is the order that the inputs
// are staged in.
__device__ __forceinline__ constexpr int code_at(int place) { return (place & 1) * 4 + (place >> 1); }
__device__ __forceinline__ constexpr int place_of(int code) { return (code & 3) * 2 + (code >> 2); }
template <int BITS>
__device__ __forceinline__ void operands(const Quarter& q, int h4, u32x4_t& lo8, u32x4_t& hi8) {
    if constexpr (BITS == 3) {
        // byte b of f[i] is code 4 b + i
        const uint32_t b = __builtin_amdgcn_perm(0u, q.b, high_sel(h4));
        const uint32_t t = (b | (b << 4)) & 0x0F0F0F0Fu;
        uint32_t f[4];
        f[0] = (q.a & 0x03030303u) | ((t << 2) & 0x04040404u);
        f[1] = ((q.a >> 2) & 0x03030303u) | ((t << 1) & 0x04040404u);
        f[2] = ((q.a >> 4) & 0x03030303u) | (t & 0x04040404u);
        f[3] = ((q.a >> 6) & 0x03030303u) | ((t >> 1) & 0x04040404u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = __builtin_amdgcn_perm(0x06040200u, 0x82848688u, f[i]);
            lo8[i] = __builtin_bit_cast(
                uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[i], 256.0f, false));
            hi8[i] = __builtin_bit_cast(
                uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(f[i], 256.0f, true));
        }
    } else {
        auto word = [](uint32_t w) {
            // byte b of e is code 2 b, of o code 2 b + 1
            const uint32_t t = w ^ 0x88888888u, e = (t << 4) & 0xF0F0F0F0u, o = t & 0xF0F0F0F0u;
            auto at = [&](int c) {
                return __float_as_uint((float)(int8_t)((c & 1 ? o : e) >> (8 * (c >> 1))));
            };
            u32x4_t r;
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_perm(at(4 + i), at(i), 0x07060302u);
            return r;
        };
        lo8 = word(q.a);
        hi8 = word(q.b);
    }
}
// Blocks (of a wave a SIMD) on a CU: widths that differ take more registers.
constexpr int up_blocks(int gb, int ub) { return gb == ub ? 4 : 3; }
template <int BITS>
constexpr float kUnit = BITS == 3 ? 1.0f : 0.0625f;

__device__ __forceinline__ f32x4_t mma(const u32x4_t& a, const u32x4_t& b, const f32x4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

template <int GB, int UB, int M, bool BF16>
__global__ __launch_bounds__(64 * kUpWaves) __attribute__((amdgpu_waves_per_eu(up_blocks(GB, UB)))) void
moe_few_up_kernel(const FewKernelArgs x) {
    constexpr int W = kUpWaves;
    constexpr int RT = kPassTokens<BF16>;      // tokens a pass
    const FewArgs& a = x.a;
    using TG = Tile<GB, kUpCG>;
    using TU = Tile<UB, kUpCG>;
    __shared__ Route rt;
    // a wave's chunk; at a tile's end its sums
    struct Own {
        union {
            struct {
                uint8_t g[16 * TG::kPitch], u[16 * TU::kPitch];  // u right after g
            } w;
            f32x4_t red[2][64];
        };
        float s[2][kUpCG][16];
    };
    __shared__ __attribute__((aligned(16))) Own own[W];
    // the staged inputs; before them what only the routing needs
    extern __shared__ __attribute__((aligned(16))) uint8_t slab[];
    Picks& picks = *reinterpret_cast<Picks*>(slab);
    route<M>(x, rt, picks);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h4 = lane >> 4, l16 = lane & 15;
    const int G = x.GD, FT = x.GF * 4;
    const int rounds = (G + kRoundGroups - 1) / kRoundGroups;
    if (blockIdx.x == 0) {
        if (tid == 0) x.count[0] = rt.n;
        for (int i = tid; i < rt.n; i += 64 * W) x.count[4 + i] = (int)rt.act[i];
        for (int i = tid; i < rt.n * a.T; i += 64 * W) {
            const int n = i / a.T, t = i % a.T, e = (int)(rt.act[n] & 0xFFFFu);
            const uint32_t m = rt.mask[e];
            if (!(m >> t & 1)) continue;
            float w = 0.0f;
            for (int j = 0; j < a.k; ++j) w = picks.sel[t][j] == e ? picks.wgt[t][j] : w;
            const int p = (int)(rt.act[n] >> 16) + __popc(m & ((1u << t) - 1));
            x.token[p] = t;
            x.weight[p] = w;
        }
    }
    // this block's tiles, next to each other: mostly of one expert
    const int items = rt.n * FT;
    const int it0 = (int)((int64_t)items * blockIdx.x / gridDim.x);
    const int it1 = (int)((int64_t)items * (blockIdx.x + 1) / gridDim.x);
    if (it0 >= it1) return;

    constexpr int NL = (TG::kPieces + TU::kPieces + 63) / 64;
    struct Chunk {
        u32x4_t p[NL];
        float sg, su;
    };
    // A block's work as steps of one round each: tile after tile, its tokens in
    // passes of RT (a pass reads the weights again).  Tile f of active expert n is
    // counted on (dividing by FT at every step took as long as an eighth of it).
    struct Step {
        int it, n, f, p0, c;
        uint32_t act, who;  // of expert n
    };
    auto enter = [&](Step& t) __attribute__((always_inline)) {
        t.act = (uint32_t)__builtin_amdgcn_readfirstlane((int)rt.act[t.n]);
        t.who = (uint32_t)__builtin_amdgcn_readfirstlane((int)rt.mask[t.act & 0xFFFFu]);
    };
    auto advance = [&](Step& t) __attribute__((always_inline)) {
        if (t.it >= it1 || ++t.c < rounds) return;
        t.c = 0;
        t.p0 += RT;
        if (t.p0 < __popc(t.who)) return;
        t.p0 = 0;
        if (++t.it == it1) {  // past the last step its loads repeat
            t.c = rounds - 1;
        } else if (++t.f == FT) {
            t.f = 0;
            ++t.n;
            enter(t);
        }
    };
    // The chunk of this wave in round c of a tile (zeros past the row): the tile's
    // and chunk's place is the wave's, a lane's own place in it stays.
    int off[NL], own_at[NL];  // of a lane's pieces, in the weights and in LDS
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int id = lane + 64 * i;
        own_at[i] = id < TG::kPieces
                        ? id / TG::kParts * TG::kPitch + id % TG::kParts * 16
                        : 16 * TG::kPitch + (id - TG::kPieces) / TU::kParts * TU::kPitch +
                              (id - TG::kPieces) % TU::kParts * 16;
        off[i] = id < TG::kPieces
                     ? id / TG::kParts * G * TG::kGB + id % TG::kParts * 16
                     : min((id - TG::kPieces) / TU::kParts, 15) * G * TU::kGB +
                           (id - TG::kPieces) % TU::kParts * 16;
    }
    const int soff = (lane >> 2) * G + (lane & 3);  // row lane / 4, group lane % 4
    auto load = [&](const Step& t, Chunk& k) __attribute__((always_inline)) {
        const int e = (int)(t.act & 0xFFFFu);
        const int f0 = t.f * 16, q0 = kUpCG * (t.c * W + wave);
        if (q0 + kUpCG <= G && f0 + 16 <= a.F) {
            const int64_t at = ((int64_t)e * a.F + f0) * G + q0;
            const uint8_t *g = a.gate.packed + at * TG::kGB, *u = a.up.packed + at * TU::kGB;
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const uint8_t* p = 64 * i + 63 < TG::kPieces ? g
                                   : 64 * i >= TG::kPieces   ? u
                                   : lane + 64 * i < TG::kPieces ? g : u;
                k.p[i] = *reinterpret_cast<const u32x4_g*>(p + (uint32_t)off[i]);
            }
            k.sg = (a.gate.scales + at)[(uint32_t)soff];
            k.su = (a.up.scales + at)[(uint32_t)soff];
            return;
        }
        // at an edge: rows past F are the last one, groups past the row zeros (a
        // chunk past it loads its last group's scales)
        const int rowmax = max(min(15, (int)(a.F - 1 - f0)), 0);
        const int64_t base = (int64_t)e * a.F + (f0 < a.F ? f0 : 0);
        int here = lane;
        asm volatile("" : "+v"(here));  // this path's places are worked out in it, not kept
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const int id = here + 64 * i;
            const bool up = id >= TG::kPieces;
            const int r = up ? id - TG::kPieces : id;
            const int parts = up ? TU::kParts : TG::kParts, gb = up ? TU::kGB : TG::kGB;
            const int row = min(r / parts, rowmax), part = r % parts;
            const uint8_t* m = up ? a.up.packed : a.gate.packed;
            k.p[i] = piece(m + ((base + row) * G + q0) * gb + 16 * part, (G - q0) * gb - 16 * part);
        }
        const int64_t at = (base + min(here >> 2, rowmax)) * G + min(q0 + (here & 3), G - 1);
        const bool in = q0 + (here & 3) < G;
        k.sg = a.gate.scales[at];
        k.su = a.up.scales[at];
        if (!in) k.sg = k.su = 0.0f;
    };
    f32x4_t acc[2];
    const uint8_t* arow = slab;
    int regs = 1;  // registers of the results that hold rows
    auto mul = [&](int c, int s0, const Chunk& k) __attribute__((always_inline)) {
        const int q0 = kUpCG * (c * W + wave);
        Own& o = own[wave];
        lds_wave_sync();  // the chunk before is read
#pragma unroll
        for (int i = 0; i < NL; ++i)
            if (64 * i + 63 < TG::kPieces + TU::kPieces || lane + 64 * i < TG::kPieces + TU::kPieces)
                *reinterpret_cast<u32x4_t*>(reinterpret_cast<uint8_t*>(&o.w) + own_at[i]) = k.p[i];
        o.s[0][lane & 3][lane >> 2] = k.sg * kUnit<GB>;
        o.s[1][lane & 3][lane >> 2] = k.su * kUnit<UB>;
        lds_wave_sync();
#pragma unroll
        for (int j = 0; j < kUpCG; ++j) {
            const u32x4_t* xp = reinterpret_cast<const u32x4_t*>(arow + (q0 + j - s0) * 128);
            const u32x4_t x0 = xp[0], x1 = xp[1];
            u32x4_t wl[2], wh[2];
            operands<GB>(TG::quarter(o.w.g, j, h4, l16), h4, wl[0], wh[0]);
            operands<UB>(TU::quarter(o.w.u, j, h4, l16), h4, wl[1], wh[1]);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const f32x4_t p = mma(x1, wh[z], mma(x0, wl[z], f32x4_t{0.f, 0.f, 0.f, 0.f}));
                const float s = o.s[z][j][l16];
                acc[z][0] = __builtin_fmaf(s, p[0], acc[z][0]);
                if (regs > 1) {  // uniform
#pragma unroll
                    for (int r = 1; r < (BF16 ? RT / 4 : 3); ++r)
                        acc[z][r] = __builtin_fmaf(s, p[r], acc[z][r]);
                }
            }
        }
    };
    Step now{it0, it0 / FT, it0 % FT, 0, 0, 0, 0};
    enter(now);
    Step ahead = now;
    auto load_ahead = [&](Chunk& k) __attribute__((always_inline)) {
        load(ahead, k);
        advance(ahead);
    };
    int have_e = -1, have_p = 0, have_c = 0;  // what the stage holds: rounds have_c ..
    int S = 1;                                // .. have_c + S - 1
    // the rows of the pass's tokens for rounds c .. c + S - 1, zero past D
    auto stage = [&](int e, int who, int nt) __attribute__((always_inline)) {
        const int rows = BF16 ? nt : 3 * nt;
        S = min((x.slab / rows - 16) / (kRoundGroups * 128), rounds);
        const int pitch = S * (kRoundGroups * 128) + 16;
        // bf16: token m is row 4 (m % 4) + m / 4, so that up to four tokens take one
        // register of the results; f32: row 4 m + piece
        const int lrow = BF16 ? min(4 * (l16 & 3) + (l16 >> 2), nt - 1)
                              : min(l16 >> 2, nt - 1) * 3 + min(l16 & 3, 2);
        regs = BF16 ? (nt + 3) / 4 : 3;
        arow = slab + lrow * pitch + 32 * h4;
        have_e = e;
        have_p = now.p0;
        have_c = now.c;
        lds_barrier();  // the stage is read
        const int vals = min(S, rounds - now.c) * (32 * W);  // of eight
        uint32_t left = (uint32_t)who;
        for (int z = 0; z < now.p0; ++z) left &= left - 1;
        for (int m = 0; m < nt; ++m, left &= left - 1) {
            const int64_t t = __ffs(left) - 1;
            for (int v = tid; v < vals; v += 64 * W) {
                const int64_t d = (int64_t)now.c * (256 * W) + 8 * v;
                uint32_t q[8], b[3][8];
                if (x.x_vec) {
                    const int64_t at = t * a.D + (d < a.D ? d : 0);
                    if constexpr (BF16) {
                        const u32x4_t z = *reinterpret_cast<const u32x4_t*>(
                            static_cast<const uint16_t*>(a.X) + at);
#pragma unroll
                        for (int y = 0; y < 8; ++y) q[y] = y & 1 ? z[y >> 1] >> 16 : z[y >> 1] & 0xFFFFu;
                    } else {
                        const u32x4_t* z =
                            reinterpret_cast<const u32x4_t*>(static_cast<const float*>(a.X) + at);
                        const u32x4_t z0 = z[0], z1 = z[1];
#pragma unroll
                        for (int y = 0; y < 8; ++y) q[y] = y < 4 ? z0[y & 3] : z1[y & 3];
                    }
                } else {
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        const int64_t at = t * a.D + (d + y < a.D ? d + y : 0);
                        q[y] = BF16 ? (uint32_t)static_cast<const uint16_t*>(a.X)[at]
                                    : static_cast<const uint32_t*>(a.X)[at];
                    }
                }
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                    const uint32_t z = d + code_at(y) < a.D ? q[code_at(y)] : 0u;
                    if constexpr (BF16)
                        b[0][y] = z;
                    else
                        split3(__uint_as_float(z), b[0][y], b[1][y], b[2][y]);
                }
#pragma unroll
                for (int pc = 0; pc < (BF16 ? 1 : 3); ++pc)
                    *reinterpret_cast<u32x4_t*>(slab + (BF16 ? m : 3 * m + pc) * pitch +
                                                16 * v) =
                        u32x4_t{b[pc][0] | b[pc][1] << 16, b[pc][2] | b[pc][3] << 16,
                                b[pc][4] | b[pc][5] << 16, b[pc][6] | b[pc][7] << 16};
            }
        }
        lds_barrier();
    };
    // the pass's sums of all waves, and its activations
    auto finish = [&](int first, int nt, int f0) __attribute__((always_inline)) {
        lds_wave_sync();  // the chunk is read
        own[wave].red[0][lane] = acc[0];
        own[wave].red[1][lane] = acc[1];
        lds_barrier();
        for (int z = tid; z < nt * 16; z += 64 * W) {
            const int m = z >> 4, c = z & 15;
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    if constexpr (BF16) {
                        s[y] += own[w].red[y][16 * (m & 3) + c][m >> 2];
                    } else {
                        const f32x4_t v = own[w].red[y][16 * m + c];
                        s[y] += (v[0] + v[1]) + v[2];
                    }
                }
            const bool in = f0 + c < a.F;
            const float h = in ? act_value(s[0], a.act) * s[1] : 0.0f;
            const int64_t at =
                (int64_t)(first + m) * (x.GF * 64) + f0 + (c & 8) + place_of(c & 7);
            const int64_t plane = (int64_t)x.pairs * x.GF * 64;
            uint32_t b0, b1, b2;
            split3(h, b0, b1, b2);
            x.planes[at] = (uint16_t)b0;
            x.planes[plane + at] = (uint16_t)b1;
            x.planes[2 * plane + at] = (uint16_t)b2;
        }
        lds_barrier();  // the sums are read
    };
    // one step from the chunk in k; false after the last one
    auto turn = [&](const Chunk& k) __attribute__((always_inline)) {
        const int e = (int)(now.act & 0xFFFFu), who = (int)now.who;
        const int nt = min(RT, __popc(who) - now.p0);
        if (have_e != e || have_p != now.p0 || now.c < have_c || now.c >= have_c + S)
            stage(e, who, nt);
        if (now.c == 0) acc[0] = acc[1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        mul(now.c, have_c * (4 * W), k);
        if (now.c + 1 == rounds) finish((int)(now.act >> 16) + now.p0, nt, now.f * 16);
        advance(now);
        return now.it < it1;
    };
    // the weights two steps ahead
    Chunk k0, k1, k2;
    load_ahead(k0);
    load_ahead(k1);
    for (;;) {
        load_ahead(k2);
        if (!turn(k0)) break;
        load_ahead(k0);
        if (!turn(k1)) break;
        load_ahead(k1);
        if (!turn(k2)) break;
    }
}

// Second launch: a block of 8 waves owns 16 outputs of every token and walks
// all active experts; its waves take chunks of eight groups in turn and add each
// chunk's products, times the pairs' weights, to sums of their own in LDS, which
// are added at the end in wave order.  Rows of the matrix operand are the
// pieces of an expert's tokens.
//
// Weights are loaded two chunks ahead and activations one; a chunk's expert and
// pairs, the addresses of both, come from LDS.
//
// An expert's rows are staged in LDS where it has one token (as many as leave two
// blocks a CU); one with more tokens reads them from the caches.  At the 128
// registers of two blocks a CU 19 to 26 go to scratch memory (36 to 64 bytes a lane).
template <int DB, bool BF16>
__global__ __launch_bounds__(64 * kDownWaves) __attribute__((amdgpu_waves_per_eu(4))) void
moe_few_down_kernel(const FewKernelArgs x) {
    constexpr int W = kDownWaves, CG = kDownCG;
    constexpr int NP = kFewPieces;  // of an activation
    constexpr int PT = 4;           // rows of a token: its pieces and one unused
    constexpr int RT = 16 / PT;     // tokens of a row tile: a lane's result rows are one's
    constexpr int kRowPitch = CG * 128 + 16;
    using TD = Tile<DB, CG>;
    constexpr int NL = TD::kPieces / 64;
    static_assert(TD::kPieces % 64 == 0, "whole loads");
    const FewArgs& a = x.a;
    constexpr int kPairs = kFewMaxTokens * kFewMaxTopK;
    struct Own {
        uint8_t w[16 * TD::kPitch];
        uint8_t h[NP * kRowPitch];
        float s[CG][16];
    };
    __shared__ __attribute__((aligned(16))) Own own[W];
    __shared__ uint32_t act[kPairs + 1];
    __shared__ uint8_t token[kPairs];
    __shared__ float weight[kPairs];
    __shared__ float sums[W][kFewMaxTokens][16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h4 = lane >> 4, l16 = lane & 15;
    const int G = x.GF, nchunk = (G + CG - 1) / CG;
    const int64_t o0 = (int64_t)blockIdx.x * 16;
    const int n = x.count[0], units = n * nchunk;
    for (int i = tid; i < x.pairs; i += 64 * W) {
        act[i] = (uint32_t)x.count[4 + i];
        token[i] = (uint8_t)x.token[i];
        weight[i] = x.weight[i];
    }
    for (int i = lane; i < a.T * 16; i += 64) sums[wave][i >> 4][i & 15] = 0.0f;
    __syncthreads();
    if (tid == 0) act[n] = (uint32_t)x.pairs << 16;
    __syncthreads();
    const int rowmax = (int)min<int64_t>(15, a.D - 1 - o0);
    const int64_t plane = (int64_t)x.pairs * G * 64;
    Own& o = own[wave];

    // a wave's units in turn: expert i and chunk c, kept as it goes
    struct At {
        int i, c;
    };
    auto advance = [&](At t) __attribute__((always_inline)) {
        t.c += W;
        while (t.c >= nchunk) {
            t.c -= nchunk;
            ++t.i;
        }
        if (t.i >= n) t = At{n - 1, nchunk - 1};  // past the last unit: it repeats
        return t;
    };
    struct Weights {
        u32x4_t p[NL];
        float s[2];
    };
    // a lane's place in a chunk stays, the chunk's is the wave's
    int off[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int id = lane + 64 * i;
        off[i] = min(id / TD::kParts, rowmax) * G * TD::kGB + id % TD::kParts * 16;
    }
    // scales: row lane / 4, groups lane % 4 and lane % 4 + 4
    const int soff = min(lane >> 2, rowmax) * G;
    auto load = [&](const At& t, Weights& w) __attribute__((always_inline)) {
        const int q0 = t.c * CG, left = G - q0;
        const int e = __builtin_amdgcn_readfirstlane((int)(act[t.i] & 0xFFFFu));
        const int64_t at = ((int64_t)e * a.D + o0) * G + q0;
        const uint8_t* p = a.down.packed + at * TD::kGB;
        const float* sc = a.down.scales + at;
        if (left >= CG) {
#pragma unroll
            for (int i = 0; i < NL; ++i)
                w.p[i] = *reinterpret_cast<const u32x4_g*>(p + (uint32_t)off[i]);
#pragma unroll
            for (int z = 0; z < 2; ++z) w.s[z] = (sc + 4 * z)[(uint32_t)(soff + (lane & 3))];
            return;
        }
        int here = lane;
        asm volatile("" : "+v"(here));  // this path's places are worked out in it, not kept
#pragma unroll
        for (int i = 0; i < NL; ++i)
            w.p[i] = piece(p + (uint32_t)off[i],
                           left * TD::kGB - 16 * ((here + 64 * i) % TD::kParts));
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const int q = (here & 3) + 4 * z;
            const float s = sc[(uint32_t)(soff + min(q, left - 1))];
            w.s[z] = q < left ? s : 0.0f;
        }
    };
    // operand row r of tokens from p0 on: pieces of token after token
    auto row_of = [&](const At& t, int p0, int r) __attribute__((always_inline)) {
        const int first = (int)(act[t.i] >> 16), end = (int)(act[t.i + 1] >> 16);
        return x.planes + r % NP * plane +
               ((int64_t)min(first + p0 + r / NP, end - 1) * G + t.c * CG) * 64;
    };
    auto load_h = [&](const At& t, u32x4_t (&h)[NP]) __attribute__((always_inline)) {
        // a lane's 16 bytes of each row (past the row its last group's)
        const int at = min(lane, 8 * (G - t.c * CG) - 1) * 8;
#pragma unroll
        for (int r = 0; r < NP; ++r)
            h[r] = *reinterpret_cast<const u32x4_t*>(row_of(t, 0, r) + at);
    };
    if (wave < units) {
        Weights w[3];
        u32x4_t h[NP];
        At now{0, wave};
        while (now.c >= nchunk) {
            now.c -= nchunk;
            ++now.i;
        }
        At next = advance(now), then;
        load(now, w[0]);
        load(next, w[1]);
        load_h(now, h);
        auto turn = [&](int u, const Weights& w0, Weights& w2) __attribute__((always_inline)) {
            then = advance(next);
            load(then, w2);
            const int first = (int)(act[now.i] >> 16), end = (int)(act[now.i + 1] >> 16);
            lds_wave_sync();  // the chunk before is read
#pragma unroll
            for (int i = 0; i < NL; ++i) {
                const int id = lane + 64 * i;
                *reinterpret_cast<u32x4_t*>(o.w + id / TD::kParts * TD::kPitch +
                                            id % TD::kParts * 16) = w0.p[i];
            }
            o.s[lane & 3][lane >> 2] = w0.s[0] * kUnit<DB>;
            o.s[(lane & 3) + 4][lane >> 2] = w0.s[1] * kUnit<DB>;
#pragma unroll
            for (int r = 0; r < NP; ++r)
                *reinterpret_cast<u32x4_t*>(o.h + r * kRowPitch + 16 * lane) = h[r];
            load_h(next, h);
            lds_wave_sync();
            // this lane's operand row: piece of a token, a valid one past them
            const int tok = l16 / PT, pc = min(l16 % PT, NP - 1);
            auto product = [&](const uint8_t* hp) __attribute__((always_inline)) {
                f32x4_t part = {0.f, 0.f, 0.f, 0.f};
                const int live = min(CG, G - now.c * CG);
#pragma unroll
                for (int j = 0; j < CG; ++j) {
                    // (past the row the scale is 0 and any group will do)
                    const u32x4_t* p =
                        reinterpret_cast<const u32x4_t*>(hp + min(j, live - 1) * 128 + 32 * h4);
                    u32x4_t wl, wh;
                    operands<DB>(TD::quarter(o.w, j, h4, l16), h4, wl, wh);
                    const float s = o.s[j][l16];
                    const f32x4_t y = mma(p[1], wh, mma(p[0], wl, f32x4_t{0.f, 0.f, 0.f, 0.f}));
#pragma unroll
                    for (int r = 0; r < NP; ++r)
                        part[r] = __builtin_fmaf(s, y[r], part[r]);
                }
                return part;
            };
            // the products of the tokens from p0 on, to this wave's sums
            auto add = [&](int p0, const f32x4_t& part) __attribute__((always_inline)) {
                lds_wave_sync();  // another lane may have added to this token before
                const int p = first + p0 + h4;
                if (p < end) {
                    float& sum = sums[wave][token[p]][l16];
                    sum = __builtin_fmaf(weight[p], (part[0] + part[1]) + part[2], sum);
                }
            };
            if (end - first == 1) {
                add(0, product(o.h + pc * kRowPitch));
            } else {
                for (int p0 = 0; p0 < end - first; p0 += RT)
                    add(p0, product(reinterpret_cast<const uint8_t*>(
                                        row_of(now, p0, min(tok, end - first - 1 - p0) * NP + pc))));
            }
            now = next;
            next = then;
            return u + W < units;
        };
        for (int u = wave;; u += 3 * W) {
            if (!turn(u, w[0], w[2])) break;
            if (!turn(u + W, w[1], w[0])) break;
            if (!turn(u + 2 * W, w[2], w[1])) break;
        }
    }
    __syncthreads();
    for (int z = tid; z < a.T * 16; z += 64 * W) {
        const int t = z >> 4, c = z & 15;
        if (o0 + c >= a.D) continue;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) s += sums[w][t][c];
        if constexpr (BF16)
            static_cast<__bf16*>(a.out)[t * a.D + o0 + c] = (__bf16)s;
        else
            static_cast<float*>(a.out)[t * a.D + o0 + c] = s;
    }
}

template <int GB, int UB, int M, bool BF16>
hipError_t start_up(const FewKernelArgs& x, int64_t items, hipStream_t s) {
    // all blocks resident: as many as the LDS of a CU takes, four at most (their
    // registers)
    const int64_t fixed = sizeof(Route) + kUpWaves * (16 * (Tile<GB, kUpCG>::kPitch +
                                                            Tile<UB, kUpCG>::kPitch) +
                                                      2 * kUpCG * 16 * 4);
    const int64_t per_cu = std::min<int64_t>(up_blocks(GB, UB), 160 * 1024 / (fixed + x.slab + 512));
    const unsigned grid = (unsigned)std::min<int64_t>(items, 256 * per_cu);
    moe_few_up_kernel<GB, UB, M, BF16><<<grid, 64 * kUpWaves, x.slab, s>>>(x);
    return hipGetLastError();
}
template <int GB, int UB, bool BF16>
hipError_t run_up(const FewKernelArgs& x, hipStream_t s) {
    const int64_t items = std::min<int64_t>(x.pairs, x.a.E) * x.GF * 4;
    return x.a.E <= 128 ? start_up<GB, UB, 2, BF16>(x, items, s)
                        : start_up<GB, UB, 8, BF16>(x, items, s);
}
template <bool BF16>
hipError_t up_bits(const FewKernelArgs& x, hipStream_t s) {
    if (x.a.gate.bits == 3)
        return x.a.up.bits == 3 ? run_up<3, 3, BF16>(x, s) : run_up<3, 4, BF16>(x, s);
    return x.a.up.bits == 3 ? run_up<4, 3, BF16>(x, s) : run_up<4, 4, BF16>(x, s);
}

template <int DB, bool BF16>
hipError_t run_down(const FewKernelArgs& x, hipStream_t s) {
    const unsigned grid = (unsigned)((x.a.D + 15) / 16);
    moe_few_down_kernel<DB, BF16><<<grid, 64 * kDownWaves, 0, s>>>(x);
    return hipGetLastError();
}

// bf16 tokens to f32 and back (one rounding), around the full layer's launches.
__global__ __launch_bounds__(256) void widen_kernel(const uint16_t* x, float* y, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        y[i] = __uint_as_float((uint32_t)x[i] << 16);
}
__global__ __launch_bounds__(256) void narrow_kernel(const float* x, __bf16* y, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        y[i] = (__bf16)x[i];
}

hipError_t run_long(const FewArgs& a, void* workspace, hipStream_t s) {
    const int64_t n = (int64_t)a.T * a.D;
    const unsigned grid = (unsigned)std::min<int64_t>((n + 255) / 256, 2048);
    const float* in = static_cast<const float*>(a.X);
    float* out = static_cast<float*>(a.out);
    if (a.bf16) {
        float* x = reinterpret_cast<float*>(
            static_cast<uint8_t*>(workspace) +
            few_align((int64_t)moe_layer_workspace(a.T, a.k, a.E, a.D, a.F)));
        out = x + few_align(n * 4) / 4;
        widen_kernel<<<grid, 256, 0, s>>>(static_cast<const uint16_t*>(a.X), x, n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
        in = x;
    }
    const hipError_t e = launch_moe_layer(
        in, a.T, a.D, a.F, a.logits, a.E, a.k, a.gate.packed, a.gate.scales, a.gate.bits,
        a.up.packed, a.up.scales, a.up.bits, a.down.packed, a.down.scales, a.down.bits, out,
        workspace, s);
    if (e != hipSuccess || !a.bf16) return e;
    narrow_kernel<<<grid, 256, 0, s>>>(out, static_cast<__bf16*>(a.out), n);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_few(const FewArgs& a, void* workspace, hipStream_t s) {
    // the full layer takes SiLU, and f32 rows aligned to 16 bytes
    const bool wide_rows = a.bf16 || ((reinterpret_cast<uintptr_t>(a.X) | reinterpret_cast<uintptr_t>(a.out)) & 15) == 0;
    if (wide_rows && a.act == 0 &&
        few_long(a.T, a.k, a.E, a.D, a.F, a.gate.bits, a.up.bits, a.down.bits))
        return run_long(a, workspace, s);
    const FewPlan p = few_plan(a.T, a.k, a.F);
    uint8_t* w = static_cast<uint8_t*>(workspace);
    FewKernelArgs x;
    x.a = a;
    x.GD = (int)((a.D + kGroup - 1) / kGroup);
    x.GF = (int)(p.fp / kGroup);
    x.pairs = (int)p.pairs;
    x.count = reinterpret_cast<int32_t*>(w);
    x.token = reinterpret_cast<int32_t*>(w + p.pair);
    x.weight = reinterpret_cast<float*>(x.token + p.pairs);
    x.planes = reinterpret_cast<uint16_t*>(w + p.planes);
    x.x_vec = a.D % 8 == 0 && (reinterpret_cast<uintptr_t>(a.X) & 15) == 0;
    // the tokens' rows whole, where they fit; the routing's picks lie there first
    const int64_t rounds = (x.GD + kRoundGroups - 1) / kRoundGroups;
    const int64_t rows = a.bf16 ? std::min(a.T, kPassTokens<true>) : 3 * std::min(a.T, kPassTokens<false>);
    x.slab = (int)std::max<int64_t>(
        sizeof(Picks), std::min<int64_t>(a.bf16 ? kSlabBytes<true> : kSlabBytes<false>,
                                         rows * (rounds * kRoundGroups * 128 + 16)));
    const hipError_t e = a.bf16 ? up_bits<true>(x, s) : up_bits<false>(x, s);
    if (e != hipSuccess) return e;
    if (a.down.bits == 3) return a.bf16 ? run_down<3, true>(x, s) : run_down<3, false>(x, s);
    return a.bf16 ? run_down<4, true>(x, s) : run_down<4, false>(x, s);
}

}  // namespace qt
