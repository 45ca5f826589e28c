// The expert layer for a few tokens (up to 16) in two launches:
//   1. h = act(Wgate_e x_t) * (Wup_e x_t) for every pair of a token and one of
//      its k experts;
//   2. out_t = sum_e w_te Wdown_e h_te.
// The weights' stream bounds both.  Every block of the first launch routes all
// tokens by itself (a wave a token: k rounds of a maximum over the wave), which
// costs less than a launch of its own; block 0 leaves the routing for the
// second one.  Codes enter the matrix cores exactly, each group's products are
// summed in f32 and scaled by the group's f32 scale.
#include "lds_barrier.h"
#include "serve.h"
#include "unpack.h"

namespace qt {
namespace {

constexpr int kUpWaves = 4, kDownWaves = 8;
// The first launch keeps its blocks for all tiles; four of them fit a CU.
constexpr int kUpBlocks = 4 * 256;
// Tokens of a pass at most, and the inputs staged at a time: 12 rows of at least 16 groups (a round of the
// waves' chunks), rows 16 bytes apart in the banks.
constexpr int kPassRows = 12;
constexpr int kSlabBytes = kPassRows * (4 * kUpWaves * 128 + 16);

struct FewKernelArgs {
    FewArgs a;
    int GD, GF;          // groups of D and of F
    int pairs;           // T k
    int32_t* count;      // active experts; from 4 on: expert | first pair << 16 of each
    int32_t* token;      // [pairs] token of a pair; pairs go by expert, then token
    float* weight;       // [pairs] weight of a pair
    uint16_t* planes;    // [pieces][pairs][64 GF]
    bool x_vec;          // eight inputs may be loaded at once
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
template <int BITS>
constexpr float kUnit = BITS == 3 ? 1.0f : 0.0625f;

__device__ __forceinline__ f32x4_t mma(const u32x4_t& a, const u32x4_t& b, const f32x4_t& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

template <int GB, int UB, int M, bool BF16>
__global__ __launch_bounds__(64 * kUpWaves) void moe_few_up_kernel(const FewKernelArgs x) {
    constexpr int W = kUpWaves;
    constexpr int RT = BF16 ? kPassRows : 4;   // tokens a pass
    constexpr int GBY = GB == 3 ? kGroupBytes : kGroupBytesI4;
    constexpr int UBY = UB == 3 ? kGroupBytes : kGroupBytesI4;
    const FewArgs& a = x.a;
    __shared__ Route rt;
    __shared__ __attribute__((aligned(16))) union {
        Picks picks;
        uint8_t stage[kSlabBytes];
    } lds;
    __shared__ __attribute__((aligned(16))) f32x4_t red[W][2][64];
    route<M>(x, rt, lds.picks);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h4 = lane >> 4, l16 = lane & 15;
    const int G = x.GD, FT = x.GF * 4;
    const int rounds = ((G + 3) / 4 + W - 1) / W;  // of the waves' chunks
    if (blockIdx.x == 0) {
        if (tid == 0) x.count[0] = rt.n;
        for (int i = tid; i < rt.n; i += 64 * W) x.count[4 + i] = (int)rt.act[i];
        for (int i = tid; i < rt.n * a.T; i += 64 * W) {
            const int n = i / a.T, t = i % a.T, e = (int)(rt.act[n] & 0xFFFFu);
            const uint32_t m = rt.mask[e];
            if (!(m >> t & 1)) continue;
            float w = 0.0f;
            for (int j = 0; j < a.k; ++j) w = lds.picks.sel[t][j] == e ? lds.picks.wgt[t][j] : w;
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

    struct Chunk {
        RowGroup<GB> g;
        RowGroup<UB> u;
        float sg, su;
    };
    // the chunk of this wave in round c of a tile (past the row a valid group,
    // whose scale is 0)
    auto load = [&](int it, int c, Chunk& k) __attribute__((always_inline)) {
        const int e = (int)(rt.act[it / FT] & 0xFFFFu), f0 = it % FT * 16;
        const int64_t row = (int64_t)e * a.F + min<int64_t>(f0 + l16, a.F - 1);
        const int q = 4 * (c * W + wave) + h4;
        const int64_t at = row * G + min(q, G - 1);
        k.g.load(a.gate.packed + at * GBY);
        k.u.load(a.up.packed + at * UBY);
        k.sg = a.gate.scales[at];
        k.su = a.up.scales[at];
    };
    f32x4_t acc[2];
    const uint8_t* arow = lds.stage;
    int regs = 1;  // registers of the results that hold rows
    auto mul = [&](int c, int s0, const Chunk& k) __attribute__((always_inline)) {
        const int q0 = 4 * (c * W + wave);
        Quarter qg[4], qu[4];
        k.g.quarters(qg);
        k.u.quarters(qu);
        uint32_t sg[4], su[4];
        const bool in = q0 + h4 < G;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sg[j] = in ? __float_as_uint(k.sg * kUnit<GB>) : 0u;
            su[j] = in ? __float_as_uint(k.su * kUnit<UB>) : 0u;
        }
        transpose_rows(sg);
        transpose_rows(su);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const u32x4_t* xp = reinterpret_cast<const u32x4_t*>(arow + (q0 + j - s0) * 128);
            const u32x4_t x0 = xp[0], x1 = xp[1];
            u32x4_t wl[2], wh[2];
            operands<GB>(qg[j], h4, wl[0], wh[0]);
            operands<UB>(qu[j], h4, wl[1], wh[1]);
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const f32x4_t p = mma(x1, wh[z], mma(x0, wl[z], f32x4_t{0.f, 0.f, 0.f, 0.f}));
                const float s = __uint_as_float(z == 0 ? sg[j] : su[j]);
                acc[z][0] = __builtin_fmaf(s, p[0], acc[z][0]);
                if (regs > 1) {  // uniform
                    acc[z][1] = __builtin_fmaf(s, p[1], acc[z][1]);
                    acc[z][2] = __builtin_fmaf(s, p[2], acc[z][2]);
                }
            }
        }
    };
    // A block's work as steps of one round each: tile after tile, its tokens in
    // passes of RT (a pass reads the weights again).
    struct Step {
        int it, p0, c;
    };
    auto tokens_of = [&](int it) __attribute__((always_inline)) {
        return __builtin_amdgcn_readfirstlane((int)rt.mask[rt.act[it / FT] & 0xFFFFu]);
    };
    auto advance = [&](Step& t) __attribute__((always_inline)) {
        if (t.it >= it1 || ++t.c < rounds) return;
        t.c = 0;
        t.p0 += RT;
        if (a.T <= RT || t.p0 >= __popc(tokens_of(t.it))) {
            t.p0 = 0;
            ++t.it;
        }
    };
    Step now{it0, 0, 0}, ahead = now;
    auto load_ahead = [&](Chunk& k) __attribute__((always_inline)) {
        // past the last step its loads repeat
        load(min(ahead.it, it1 - 1), ahead.it < it1 ? ahead.c : rounds - 1, k);
        advance(ahead);
    };
    int have_e = -1, have_p = 0, have_c = 0;  // what the stage holds: rounds have_c ..
    int S = 1;                                // .. have_c + S - 1
    // the rows of the pass's tokens for rounds c .. c + S - 1, zero past D
    auto stage = [&](int e, int who, int nt) __attribute__((always_inline)) {
        const int rows = BF16 ? nt : 3 * nt;
        S = min((kSlabBytes / rows - 16) / (512 * W), rounds);
        const int pitch = S * (512 * W) + 16;
        // bf16: token m is row 4 (m % 4) + m / 4, so that up to four tokens take one
        // register of the results; f32: row 4 m + piece
        const int lrow = BF16 ? min(4 * (l16 & 3) + (l16 >> 2), nt - 1)
                              : min(l16 >> 2, nt - 1) * 3 + min(l16 & 3, 2);
        regs = BF16 ? (nt + 3) / 4 : 3;
        arow = lds.stage + lrow * pitch + 32 * h4;
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
                    *reinterpret_cast<u32x4_t*>(lds.stage + (BF16 ? m : 3 * m + pc) * pitch +
                                                16 * v) =
                        u32x4_t{b[pc][0] | b[pc][1] << 16, b[pc][2] | b[pc][3] << 16,
                                b[pc][4] | b[pc][5] << 16, b[pc][6] | b[pc][7] << 16};
            }
        }
        lds_barrier();
    };
    // the pass's sums of all waves, and its activations
    auto finish = [&](int first, int nt, int f0) __attribute__((always_inline)) {
        lds_barrier();  // the sums of the pass before are read
        red[wave][0][lane] = acc[0];
        red[wave][1][lane] = acc[1];
        lds_barrier();
        for (int z = tid; z < nt * 16; z += 64 * W) {
            const int m = z >> 4, c = z & 15;
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    if constexpr (BF16) {
                        s[y] += red[w][y][16 * (m & 3) + c][m >> 2];
                    } else {
                        const f32x4_t v = red[w][y][16 * m + c];
                        s[y] += (v[0] + v[1]) + v[2];
                    }
                }
            const bool in = f0 + c < a.F;
            const float h = in ? act_value(s[0], a.act) * s[1] : 0.0f;
            const int64_t at =
                (int64_t)(first + m) * (x.GF * 64) + f0 + (c & 8) + place_of(c & 7);
            const int64_t plane = (int64_t)x.pairs * x.GF * 64;
            if constexpr (BF16) {
                const float hi = __uint_as_float(__float_as_uint(h) & 0xFFFF0000u);
                x.planes[at] = (uint16_t)(__float_as_uint(hi) >> 16);
                x.planes[plane + at] = __builtin_bit_cast(uint16_t, (__bf16)(h - hi));
            } else {
                uint32_t b0, b1, b2;
                split3(h, b0, b1, b2);
                x.planes[at] = (uint16_t)b0;
                x.planes[plane + at] = (uint16_t)b1;
                x.planes[2 * plane + at] = (uint16_t)b2;
            }
        }
    };
    // one step from the chunk in k; false after the last one
    auto turn = [&](const Chunk& k) __attribute__((always_inline)) {
        const uint32_t act = __builtin_amdgcn_readfirstlane((int)rt.act[now.it / FT]);
        const int e = (int)(act & 0xFFFFu), who = tokens_of(now.it);
        const int nt = min(RT, __popc(who) - now.p0);
        if (have_e != e || have_p != now.p0 || now.c < have_c || now.c >= have_c + S)
            stage(e, who, nt);
        if (now.c == 0) acc[0] = acc[1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        mul(now.c, have_c * (4 * W), k);
        if (now.c + 1 == rounds) finish((int)(act >> 16) + now.p0, nt, now.it % FT * 16);
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
// all active experts; its waves take chunks of four groups in turn and add each
// chunk's products, times the pairs' weights, to sums of their own in LDS, which
// are added at the end in wave order.  Rows of the matrix operand are the
// pieces of an expert's tokens.
//
// Weights are loaded three chunks ahead and activations one; a chunk's expert
// and pairs, the addresses of both, come from LDS.
template <int DB, bool BF16>
__global__ __launch_bounds__(64 * kDownWaves) __attribute__((amdgpu_waves_per_eu(4))) void
moe_few_down_kernel(const FewKernelArgs x) {
    constexpr int W = kDownWaves;
    constexpr int PT = BF16 ? 2 : 4;   // rows of a token: its pieces (and one unused)
    constexpr int RT = 16 / PT;        // tokens of a row tile
    constexpr int NW = 4 / PT;         // tokens of a lane's four result rows
    constexpr int BY = DB == 3 ? kGroupBytes : kGroupBytesI4;
    const FewArgs& a = x.a;
    constexpr int kPairs = kFewMaxTokens * kFewMaxTopK;
    __shared__ uint32_t act[kPairs + 1];
    __shared__ int32_t token[kPairs];
    __shared__ float weight[kPairs];
    __shared__ float sums[W][kFewMaxTokens][16];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h4 = lane >> 4, l16 = lane & 15;
    const int G = x.GF, nchunk = (G + 3) / 4;
    const int64_t o0 = (int64_t)blockIdx.x * 16;
    const int n = x.count[0], units = n * nchunk;
    for (int i = tid; i < x.pairs; i += 64 * W) {
        act[i] = (uint32_t)x.count[4 + i];
        token[i] = x.token[i];
        weight[i] = x.weight[i];
    }
    for (int i = lane; i < a.T * 16; i += 64) sums[wave][i >> 4][i & 15] = 0.0f;
    __syncthreads();
    if (tid == 0) act[n] = (uint32_t)x.pairs << 16;
    __syncthreads();
    const int64_t orow = min<int64_t>(o0 + l16, a.D - 1);
    const int piece = BF16 ? l16 & 1 : min(l16 & 3, 2);
    const uint16_t* plane = x.planes + piece * ((int64_t)x.pairs * G * 64) + 16 * h4;

    struct Weights {
        RowGroup<DB> w;
        float s;
    };
    auto expert_of = [&](int u) __attribute__((always_inline)) { return min(u, units - 1) / nchunk; };
    auto load = [&](int u, Weights& w) __attribute__((always_inline)) {
        const int i = expert_of(u);
        const int q = min(4 * (min(u, units - 1) - i * nchunk) + h4, G - 1);
        const int64_t r = ((int64_t)(act[i] & 0xFFFFu) * a.D + orow) * G + q;
        w.w.load(a.down.packed + r * BY);
        w.s = a.down.scales[r];
    };
    // this lane's operand row of unit u's first group, tokens from p0 on
    auto row_of = [&](int u, int p0) __attribute__((always_inline)) {
        const int i = expert_of(u), first = (int)(act[i] >> 16), end = (int)(act[i + 1] >> 16);
        const int p = min(first + p0 + l16 / PT, end - 1);
        return plane + ((int64_t)p * G + 4 * (min(u, units - 1) - i * nchunk)) * 64;
    };
    // group j of it (past the row the last one, scale 0)
    auto operand = [&](const uint16_t* row, int left, int j, u32x4_t (&v)[2])
                       __attribute__((always_inline)) {
        const u32x4_t* p = reinterpret_cast<const u32x4_t*>(row + min(j, left) * 64);
        v[0] = p[0];
        v[1] = p[1];
    };
    auto left_of = [&](int u) __attribute__((always_inline)) {
        return G - 1 - 4 * (min(u, units - 1) - expert_of(u) * nchunk);
    };
    if (wave < units) {
        Weights w[4];
        u32x4_t v[4][2];
#pragma unroll
        for (int i = 0; i < 3; ++i) load(wave + i * W, w[i]);
        {
            const uint16_t* row = row_of(wave, 0);
#pragma unroll
            for (int j = 0; j < 4; ++j) operand(row, left_of(wave), j, v[j]);
        }
        auto turn = [&](int u, const Weights& w0, Weights& w3) __attribute__((always_inline)) {
            load(u + 3 * W, w3);
            const int i = u / nchunk, first = (int)(act[i] >> 16), end = (int)(act[i + 1] >> 16);
            const uint16_t* ahead = row_of(u + W, 0);
            const int left = left_of(u + W);
            Quarter qd[4];
            w0.w.quarters(qd);
            uint32_t sd[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sd[j] = 4 * (u - i * nchunk) + h4 < G ? __float_as_uint(w0.s * kUnit<DB>) : 0u;
            transpose_rows(sd);
            auto product = [&](bool last) __attribute__((always_inline)) {
                f32x4_t part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    u32x4_t wl, wh;
                    operands<DB>(qd[j], h4, wl, wh);
                    const float s = __uint_as_float(sd[j]);
                    const f32x4_t p =
                        mma(v[j][1], wh, mma(v[j][0], wl, f32x4_t{0.f, 0.f, 0.f, 0.f}));
#pragma unroll
                    for (int r = 0; r < 4; ++r) part[r] = __builtin_fmaf(s, p[r], part[r]);
                    if (last) operand(ahead, left, j, v[j]);
                }
                return part;
            };
            // the products of the tokens from p0 on, to this wave's sums
            auto add = [&](int p0, const f32x4_t& part) __attribute__((always_inline)) {
                lds_wave_sync();  // another lane may have added to this token before
#pragma unroll
                for (int z = 0; z < NW; ++z) {
                    const int p = first + p0 + NW * h4 + z;
                    if (p < end) {
                        const float y = BF16 ? part[2 * z] + part[2 * z + 1]
                                             : (part[0] + part[1]) + part[2];
                        float& sum = sums[wave][token[p]][l16];
                        sum = __builtin_fmaf(weight[p], y, sum);
                    }
                }
            };
            // more tokens than a row tile: their rows are loaded as they come
            for (int p0 = 0; p0 + RT < end - first; p0 += RT) {
                add(p0, product(false));
                const uint16_t* row = row_of(u, p0 + RT);
#pragma unroll
                for (int j = 0; j < 4; ++j) operand(row, left_of(u), j, v[j]);
            }
            add((end - first - 1) / RT * RT, product(true));
            return u + W < units;
        };
        for (int u = wave;; u += 4 * W) {
            if (!turn(u, w[0], w[3])) break;
            if (!turn(u + W, w[1], w[0])) break;
            if (!turn(u + 2 * W, w[2], w[1])) break;
            if (!turn(u + 3 * W, w[3], w[2])) break;
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

template <int GB, int UB, bool BF16>
hipError_t run_up(const FewKernelArgs& x, hipStream_t s) {
    const int64_t items = std::min<int64_t>(x.pairs, x.a.E) * x.GF * 4;
    const unsigned grid = (unsigned)std::min<int64_t>(items, kUpBlocks);
    if (x.a.E <= 128)
        moe_few_up_kernel<GB, UB, 2, BF16><<<grid, 64 * kUpWaves, 0, s>>>(x);
    else
        moe_few_up_kernel<GB, UB, 8, BF16><<<grid, 64 * kUpWaves, 0, s>>>(x);
    return hipGetLastError();
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

}  // namespace

hipError_t launch_moe_few(const FewArgs& a, void* workspace, hipStream_t s) {
    const FewPlan p = few_plan(a.T, a.k, a.F, a.bf16);
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
    const hipError_t e = a.bf16 ? up_bits<true>(x, s) : up_bits<false>(x, s);
    if (e != hipSuccess) return e;
    if (a.down.bits == 3) return a.bf16 ? run_down<3, true>(x, s) : run_down<3, false>(x, s);
    return a.bf16 ? run_down<4, true>(x, s) : run_down<4, false>(x, s);
}

}  // namespace qt
