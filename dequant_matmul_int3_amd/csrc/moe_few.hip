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
// Inputs staged at a time: 12 rows of at least 16 groups (a round of the
// waves' chunks), rows 16 bytes apart in the banks.
constexpr int kPassRows = 12;
constexpr int kSlabBytes = kPassRows * (4 * kUpWaves * 128 + 16);

struct FewKernelArgs {
    FewArgs a;
    int GD, GF;          // groups of D and of F
    int pairs;           // T k
    int32_t* count;      // active experts; from 4 on: [pairs] expert, [pairs] first pair
    float* weight;       // [pairs][T] weight of (active expert, token), 0: not its token
    int32_t* prow;       // [pairs][T] pair of (active expert, token)
    uint16_t* planes;    // [pieces][pairs][64 GF]
    bool x_vec;          // four inputs may be loaded at once
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

// Sixteen codes as two exact operands: v for int3, 16 v for int4 (the nibbles
// of a word as the high halves of signed bytes).
template <int BITS>
__device__ __forceinline__ void operands(const Quarter& q, int h4, u32x4_t& lo8, u32x4_t& hi8) {
    if constexpr (BITS == 3) {
        exact_quarter(q, h4, 3, lo8, hi8);
    } else {
        auto word = [](uint32_t w) {
            const uint32_t t = w ^ 0x88888888u, e = (t << 4) & 0xF0F0F0F0u, o = t & 0xF0F0F0F0u;
            auto at = [](uint32_t v, int b) { return __float_as_uint((float)(int8_t)(v >> (8 * b))); };
            u32x4_t r;
#pragma unroll
            for (int b = 0; b < 4; ++b) r[b] = __builtin_amdgcn_perm(at(o, b), at(e, b), 0x07060302u);
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
        for (int i = tid; i < rt.n; i += 64 * W) {
            x.count[4 + i] = (int)(rt.act[i] & 0xFFFFu);
            x.count[4 + x.pairs + i] = (int)(rt.act[i] >> 16);
        }
        for (int i = tid; i < rt.n * a.T; i += 64 * W) {
            const int n = i / a.T, t = i % a.T, e = (int)(rt.act[n] & 0xFFFFu);
            float w = 0.0f;
            for (int j = 0; j < a.k; ++j) w = lds.picks.sel[t][j] == e ? lds.picks.wgt[t][j] : w;
            const uint32_t m = rt.mask[e];
            x.weight[i] = w;
            x.prow[i] = (int)(rt.act[n] >> 16) + (m >> t & 1 ? __popc(m & ((1u << t) - 1)) : 0);
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
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[z][r] = __builtin_fmaf(s, p[r], acc[z][r]);
            }
        }
    };
    int have_e = -1, have_p = -1, have_s = -1;  // what the stage holds
    Chunk k0, k1;
    load(it0, 0, k0);
    for (int it = it0; it < it1; ++it) {
        const uint32_t act = rt.act[it / FT];
        const int e = (int)(act & 0xFFFFu), f0 = it % FT * 16;
        const uint32_t who = rt.mask[e];
        const int n = __popc(who);
        // tokens in passes of RT; a pass reads the weights (again)
        for (int p0 = 0; p0 < n; p0 += RT) {
            const int nt = min(RT, n - p0);
            const int rows = BF16 ? nt : 3 * nt;
            // rounds staged at a time
            const int S = min((kSlabBytes / rows - 16) / (512 * W), rounds);
            const int pitch = S * (512 * W) + 16;
            const int lrow = BF16 ? min(l16, nt - 1) : min(l16 >> 2, nt - 1) * 3 + min(l16 & 3, 2);
            arow = lds.stage + lrow * pitch + 32 * h4;
            acc[0] = acc[1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            const bool tail = p0 + RT >= n;  // the tile's last pass
            for (int c0 = 0; c0 < rounds; c0 += S) {
                if (have_e != e || have_p != p0 || have_s != c0) {
                    have_e = e;
                    have_p = p0;
                    have_s = c0;
                    lds_barrier();  // the stage is read
                    // token rows of the rounds, zero past D
                    const int vals = min(S, rounds - c0) * (64 * W);  // of four
                    uint32_t left = who;
                    for (int z = 0; z < p0; ++z) left &= left - 1;
                    for (int m = 0; m < nt; ++m, left &= left - 1) {
                        const int64_t t = __ffs(left) - 1;
                        for (int v = tid; v < vals; v += 64 * W) {
                            const int64_t d = (int64_t)c0 * (256 * W) + 4 * v;
                            uint32_t q[4], b[3][4];
                            if (x.x_vec) {
                                const int64_t at = t * a.D + (d < a.D ? d : 0);
                                if constexpr (BF16) {
                                    const u32x2_t z = *reinterpret_cast<const u32x2_t*>(
                                        static_cast<const uint16_t*>(a.X) + at);
                                    q[0] = z.x & 0xFFFFu;
                                    q[1] = z.x >> 16;
                                    q[2] = z.y & 0xFFFFu;
                                    q[3] = z.y >> 16;
                                } else {
                                    const u32x4_t z = *reinterpret_cast<const u32x4_t*>(
                                        static_cast<const float*>(a.X) + at);
#pragma unroll
                                    for (int y = 0; y < 4; ++y) q[y] = z[y];
                                }
                            } else {
#pragma unroll
                                for (int y = 0; y < 4; ++y) {
                                    const int64_t at = t * a.D + (d + y < a.D ? d + y : 0);
                                    q[y] = BF16 ? (uint32_t)static_cast<const uint16_t*>(a.X)[at]
                                                : static_cast<const uint32_t*>(a.X)[at];
                                }
                            }
#pragma unroll
                            for (int y = 0; y < 4; ++y) {
                                if (d + y >= a.D) q[y] = 0u;
                                if constexpr (BF16)
                                    b[0][y] = q[y];
                                else
                                    split3(__uint_as_float(q[y]), b[0][y], b[1][y], b[2][y]);
                            }
#pragma unroll
                            for (int pc = 0; pc < (BF16 ? 1 : 3); ++pc)
                                *reinterpret_cast<u32x2_t*>(
                                    lds.stage + (BF16 ? m : 3 * m + pc) * pitch + 8 * v) =
                                    u32x2_t{b[pc][0] | b[pc][1] << 16, b[pc][2] | b[pc][3] << 16};
                        }
                    }
                    lds_barrier();
                }
                const int c1 = min(rounds, c0 + S);
                for (int c = c0; c < c1; ++c) {
                    // the next chunk: of this pass, of the next pass or of the next tile
                    const bool on = c + 1 < rounds;
                    load(on || !tail ? it : min(it + 1, it1 - 1), on ? c + 1 : 0, k1);
                    mul(c, c0 * (4 * W), k0);
                    k0 = k1;
                }
            }
            lds_barrier();  // the sums of the pass before are read
            red[wave][0][lane] = acc[0];
            red[wave][1][lane] = acc[1];
            lds_barrier();
            // element (row m, column c): lane 16 (m / 4) + c, register m % 4
            for (int z = tid; z < nt * 16; z += 64 * W) {
                const int m = z >> 4, c = z & 15;
                float s[2] = {0.0f, 0.0f};
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        if constexpr (BF16) {
                            s[y] += red[w][y][16 * (m >> 2) + c][m & 3];
                        } else {
                            const f32x4_t v = red[w][y][16 * m + c];
                            s[y] += (v[0] + v[1]) + v[2];
                        }
                    }
                const bool in = f0 + c < a.F;
                const float h = in ? act_value(s[0], a.act) * s[1] : 0.0f;
                const int64_t at = (int64_t)((int)(act >> 16) + p0 + m) * (x.GF * 64) + f0 + c;
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
        }
    }
}

// Second launch: a block of 8 waves owns 16 outputs of every token and walks
// all active experts; its waves take chunks of four groups in turn.  A row of
// the matrix operand is a token's piece, so that the sums over the experts
// stay in place; rows of tokens that an expert does not have get the weight 0.
// MT: row tiles of 8 (two pieces) or 4 (three) tokens.
//
// A chunk's weights and activations are loaded a chunk ahead, its expert and
// its tokens' pairs another one: each is an address for the next.
template <int DB, int MT, bool BF16>
__global__ __launch_bounds__(64 * kDownWaves) void moe_few_down_kernel(const FewKernelArgs x) {
    constexpr int W = kDownWaves;
    constexpr int TPT = BF16 ? 8 : 4;  // tokens of a row tile
    constexpr int BY = DB == 3 ? kGroupBytes : kGroupBytesI4;
    constexpr int NW = BF16 ? 2 : 1;   // tokens of a lane's four result rows
    const FewArgs& a = x.a;
    __shared__ __attribute__((aligned(16))) f32x4_t red[W][MT][64];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h4 = lane >> 4, l16 = lane & 15;
    const int G = x.GF, nchunk = (G + 3) / 4;
    const int64_t o0 = (int64_t)blockIdx.x * 16;
    const int n = x.count[0], units = n * nchunk;
    const int64_t orow = min<int64_t>(o0 + l16, a.D - 1);
    const int piece = BF16 ? l16 & 1 : min(l16 & 3, 2);
    const uint16_t* plane = x.planes + piece * ((int64_t)x.pairs * G * 64) + 16 * h4;
    f32x4_t acc[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    struct Who {  // of a unit: its expert, this lane's operand row and result rows
        int e, row[MT];
        float wt[MT][NW];
    };
    struct Weights {
        RowGroup<DB> w;
        float s;
    };
    auto look = [&](int u, Who& k) __attribute__((always_inline)) {
        const int i = min(u, units - 1) / nchunk;
        k.e = x.count[4 + i];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            k.row[mt] = x.prow[i * a.T + min(mt * TPT + (BF16 ? l16 >> 1 : l16 >> 2), a.T - 1)];
#pragma unroll
            for (int z = 0; z < NW; ++z) {
                const int t = mt * TPT + (BF16 ? 2 * h4 + z : h4);
                const float v = x.weight[i * a.T + min(t, a.T - 1)];
                k.wt[mt][z] = t < a.T ? v : 0.0f;
            }
        }
    };
    auto load = [&](int u, const Who& k, Weights& w) __attribute__((always_inline)) {
        const int q = min(4 * (min(u, units - 1) % nchunk) + h4, G - 1);
        const int64_t r = ((int64_t)k.e * a.D + orow) * G + q;
        w.w.load(a.down.packed + r * BY);
        w.s = a.down.scales[r];
    };
    // group j of the unit's operand rows (past the row a valid group, scale 0)
    auto operand = [&](int u, const Who& k, int j, u32x4_t (&v)[MT][2])
                       __attribute__((always_inline)) {
        const int q = min(4 * (min(u, units - 1) % nchunk) + j, G - 1);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const u32x4_t* p =
                reinterpret_cast<const u32x4_t*>(plane + ((int64_t)k.row[mt] * G + q) * 64);
            v[mt][0] = p[0];
            v[mt][1] = p[1];
        }
    };
    if (wave < units) {
        Who cur, next, then;
        Weights w0, w1;
        u32x4_t v[4][MT][2];
        look(wave, cur);
        look(wave + W, next);
        load(wave, cur, w0);
#pragma unroll
        for (int j = 0; j < 4; ++j) operand(wave, cur, j, v[j]);
        for (int u = wave; u < units; u += W) {
            look(u + 2 * W, then);
            load(u + W, next, w1);
            Quarter qd[4];
            w0.w.quarters(qd);
            uint32_t sd[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                sd[j] = 4 * (u % nchunk) + h4 < G ? __float_as_uint(w0.s * kUnit<DB>) : 0u;
            transpose_rows(sd);
            f32x4_t part[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) part[mt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                u32x4_t wl, wh;
                operands<DB>(qd[j], h4, wl, wh);
                const float s = __uint_as_float(sd[j]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const f32x4_t p =
                        mma(v[j][mt][1], wh, mma(v[j][mt][0], wl, f32x4_t{0.f, 0.f, 0.f, 0.f}));
#pragma unroll
                    for (int r = 0; r < 4; ++r) part[mt][r] = __builtin_fmaf(s, p[r], part[mt][r]);
                }
                operand(u + W, next, j, v[j]);
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // another token's products, whatever they are, do not count
                    const float w = cur.wt[mt][BF16 ? r >> 1 : 0];
                    acc[mt][r] = __builtin_fmaf(w, w != 0.0f ? part[mt][r] : 0.0f, acc[mt][r]);
                }
            cur = next;
            next = then;
            w0 = w1;
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) red[wave][mt][lane] = acc[mt];
    __syncthreads();
    for (int z = tid; z < a.T * 16; z += 64 * W) {
        const int t = z >> 4, c = z & 15, mt = t / TPT, m = t % TPT;
        if (o0 + c >= a.D) continue;
        float s = 0.0f;
        for (int w = 0; w < W; ++w) {
            if constexpr (BF16) {
                const f32x4_t v = red[w][mt][16 * (m >> 1) + c];
                s += m & 1 ? v[2] + v[3] : v[0] + v[1];
            } else {
                const f32x4_t v = red[w][mt][16 * m + c];
                s += (v[0] + v[1]) + v[2];
            }
        }
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
    const int mt = (x.a.T + (BF16 ? 7 : 3)) / (BF16 ? 8 : 4);
    if (mt == 1)
        moe_few_down_kernel<DB, 1, BF16><<<grid, 64 * kDownWaves, 0, s>>>(x);
    else if (mt == 2)
        moe_few_down_kernel<DB, 2, BF16><<<grid, 64 * kDownWaves, 0, s>>>(x);
    else if constexpr (!BF16)
        moe_few_down_kernel<DB, 4, BF16><<<grid, 64 * kDownWaves, 0, s>>>(x);
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
    x.weight = reinterpret_cast<float*>(w + p.weight);
    x.prow = reinterpret_cast<int32_t*>(x.weight + p.pairs * a.T);
    x.planes = reinterpret_cast<uint16_t*>(w + p.planes);
    x.x_vec = a.D % 4 == 0 && (reinterpret_cast<uintptr_t>(a.X) & (a.bf16 ? 7 : 15)) == 0;
    const hipError_t e = a.bf16 ? up_bits<true>(x, s) : up_bits<false>(x, s);
    if (e != hipSuccess) return e;
    if (a.down.bits == 3) return a.bf16 ? run_down<3, true>(x, s) : run_down<3, false>(x, s);
    return a.bf16 ? run_down<4, true>(x, s) : run_down<4, false>(x, s);
}

}  // namespace qt
