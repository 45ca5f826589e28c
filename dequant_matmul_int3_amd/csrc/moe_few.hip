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
// Inputs staged at a time: 16 rows of at least 16 groups, 16 bytes apart in the banks.
constexpr int kSlabBytes = 16 * (16 * 128 + 16);
static_assert((kSlabBytes / 16 - 16) / 128 >= 4 * kUpWaves, "a round of chunks for 16 rows");

struct FewKernelArgs {
    FewArgs a;
    int GD, GF;          // groups of D and of F
    int pairs;           // T k
    int32_t* count;      // active experts; from 4 on: [pairs] expert, [pairs] first pair
    float* weight;       // [pairs][T] weight of (active expert, token), 0: not its token
    int32_t* prow;       // [pairs][T] pair of (active expert, token)
    uint16_t* planes;    // [pieces][pairs][64 GF]
};

__device__ __forceinline__ uint64_t key_of(float v, int e) {
    const uint32_t u = __float_as_uint(v + 0.0f);  // -0 as +0
    const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((uint64_t)o << 32) | (uint32_t)(0xFFFF - e);
}
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
template <int N>
__device__ __forceinline__ uint64_t ror_max(uint64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)v, 0x120 + N, 0xF, 0xF, false);
    const uint32_t hi =
        (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(v >> 32), 0x120 + N, 0xF, 0xF, false);
    const uint64_t w = ((uint64_t)hi << 32) | lo;
    return w > v ? w : v;
}
__device__ __forceinline__ uint64_t wave_max_key(uint64_t v) {
    v = ror_max<8>(v);
    v = ror_max<4>(v);
    v = ror_max<2>(v);
    v = ror_max<1>(v);
    {
        const auto l = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
        const auto h = __builtin_amdgcn_permlane16_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32),
                                                        false, false);
        const uint64_t x = ((uint64_t)h[0] << 32) | l[0], y = ((uint64_t)h[1] << 32) | l[1];
        v = x > y ? x : y;
    }
    const auto l = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
    const auto h = __builtin_amdgcn_permlane32_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false,
                                                    false);
    const uint64_t x = ((uint64_t)h[0] << 32) | l[0], y = ((uint64_t)h[1] << 32) | l[1];
    return x > y ? x : y;
}

// The routing of all tokens in LDS.
struct Route {
    uint32_t mask[kFewMaxExperts];   // tokens of an expert
    int32_t act[kFewMaxTokens * kFewMaxTopK];   // active experts, ascending
    int32_t first[kFewMaxTokens * kFewMaxTopK]; // an active expert's first pair
    int32_t sel[kFewMaxTokens][kFewMaxTopK];
    float wgt[kFewMaxTokens][kFewMaxTopK];
    int32_t n;
};

// M: experts per lane (E <= 64 M)
template <int M>
__device__ void route(const FewKernelArgs& x, Route& r) {
    const FewArgs& a = x.a;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int E = a.E, k = a.k;
    for (int e = tid; e < E; e += 64 * kUpWaves) r.mask[e] = 0;
    __syncthreads();
    for (int t = wave; t < a.T; t += kUpWaves) {
        uint64_t key[M];
#pragma unroll
        for (int m = 0; m < M; ++m) {
            const int e = lane + 64 * m;
            const float v = a.logits[(int64_t)t * E + min(e, E - 1)];
            key[m] = e < E ? key_of(v, e) : 0ull;  // below every real key
        }
        uint64_t prev = ~0ull;
        float top = 0.0f, sum = 0.0f, mine = 0.0f;
        for (int j = 0; j < k; ++j) {
            uint64_t best = 0;
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const uint64_t c = key[m] < prev ? key[m] : 0ull;
                best = c > best ? c : best;
            }
            prev = wave_max_key(best);
            const float v = key_value(prev);
            if (j == 0) top = v;
            const float e = expf(v - top);
            sum += e;
            if (lane == j) mine = e;
            if (lane == 0) {
                const int id = 0xFFFF - (int)(prev & 0xFFFFu);
                r.sel[t][j] = id;
                atomicOr(&r.mask[id], 1u << t);
            }
        }
        if (lane < k) r.wgt[t][lane] = mine / sum;
    }
    __syncthreads();
    if (wave == 0) {  // active experts and their first pairs
        int n = 0, p = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + lane;
            const uint32_t m = e < E ? r.mask[e] : 0u;
            const uint64_t b = __ballot(m != 0);
            int inc = __popc(m);
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int y = __shfl_up(inc, d);
                if (lane >= d) inc += y;
            }
            if (m) {
                const int i = n + __popcll(b & ((1ull << lane) - 1));
                r.act[i] = e;
                r.first[i] = p + inc - __popc(m);
            }
            n += __popcll(b);
            p += __shfl(inc, 63);
        }
        if (lane == 0) r.n = n;
    }
    __syncthreads();
}

// One lane's whole groups of a row, four groups a chunk (one per lane row).
template <int BITS>
struct Piece {
    RowGroup<BITS> w;
    float s;
};

template <int GB, int UB, int M, bool BF16>
__global__ __launch_bounds__(64 * kUpWaves) void moe_few_up_kernel(const FewKernelArgs x) {
    constexpr int W = kUpWaves;
    constexpr int RT = BF16 ? 16 : 4;   // tokens a pass
    constexpr int GBY = GB == 3 ? kGroupBytes : kGroupBytesI4;
    constexpr int UBY = UB == 3 ? kGroupBytes : kGroupBytesI4;
    const FewArgs& a = x.a;
    __shared__ Route rt;
    __shared__ __attribute__((aligned(16))) uint8_t stage[kSlabBytes];
    __shared__ __attribute__((aligned(16))) f32x4_t red[W][2][64];
    route<M>(x, rt);
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int h4 = lane >> 4, l16 = lane & 15;
    const int G = x.GD, nchunk = (G + 3) / 4, FT = x.GF * 4;
    if (blockIdx.x == 0) {
        if (tid == 0) x.count[0] = rt.n;
        for (int i = tid; i < rt.n; i += 64 * W) {
            x.count[4 + i] = rt.act[i];
            x.count[4 + x.pairs + i] = rt.first[i];
        }
        for (int i = tid; i < rt.n * a.T; i += 64 * W) {
            const int n = i / a.T, t = i % a.T, e = rt.act[n];
            float w = 0.0f;
            for (int j = 0; j < a.k; ++j) w = rt.sel[t][j] == e ? rt.wgt[t][j] : w;
            const uint32_t m = rt.mask[e];
            x.weight[i] = w;
            x.prow[i] = rt.first[n] + (m >> t & 1 ? __popc(m & ((1u << t) - 1)) : 0);
        }
    }
    const int items = rt.n * FT;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        const int i = it / FT, f0 = (it % FT) * 16, e = rt.act[i];
        const uint32_t who = rt.mask[e];
        const int n = __popc(who);
        const int64_t row = (int64_t)e * a.F + min<int64_t>(f0 + l16, a.F - 1);
        const uint8_t* gp = a.gate.packed + row * G * GBY;
        const uint8_t* up = a.up.packed + row * G * UBY;
        const float* gs = a.gate.scales + row * G;
        const float* us = a.up.scales + row * G;
        // tokens in passes of RT; a pass reads the weights (again)
        for (int p0 = 0; p0 < n; p0 += RT) {
            const int nt = min(RT, n - p0);
            const int rows = BF16 ? nt : 3 * nt;
            // groups staged at a time: whole rounds of the waves' chunks
            int S = (kSlabBytes / rows - 16) / 128 / (4 * W) * (4 * W);
            S = max(4 * W, min(S, (G + 4 * W - 1) / (4 * W) * (4 * W)));
            const int pitch = S * 128 + 16;
            const int lrow = BF16 ? min(l16, nt - 1) : min(l16 >> 2, nt - 1) * 3 + min(l16 & 3, 2);
            const uint8_t* arow = stage + lrow * pitch + 32 * h4;
            f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
            Piece<GB> g0, g1;
            Piece<UB> u0, u1;
            auto load = [&](int c, Piece<GB>& g, Piece<UB>& u) {
                const int q = min(4 * c + h4, G - 1);
                g.w.load(gp + (int64_t)q * GBY);
                u.w.load(up + (int64_t)q * UBY);
                g.s = gs[q];
                u.s = us[q];
            };
            auto mul = [&](int c, int s0, const Piece<GB>& g, const Piece<UB>& u) {
                Quarter qg[4], qu[4];
                g.w.quarters(qg);
                u.w.quarters(qu);
                uint32_t sg[4], su[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = 4 * c + h4 < G;
                    sg[j] = in ? __float_as_uint(g.s * code_unit(GB)) : 0u;
                    su[j] = in ? __float_as_uint(u.s * code_unit(UB)) : 0u;
                }
                transpose_rows(sg);
                transpose_rows(su);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const u32x4_t* xp =
                        reinterpret_cast<const u32x4_t*>(arow + (4 * c + j - s0) * 128);
                    const u32x4_t x0 = xp[0], x1 = xp[1];
                    u32x4_t wl[2], wh[2];
                    exact_quarter(qg[j], h4, GB, wl[0], wh[0]);
                    exact_quarter(qu[j], h4, UB, wl[1], wh[1]);
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        f32x4_t p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8_t, x0), __builtin_bit_cast(bf16x8_t, wl[z]),
                            f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
                        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8_t, x1), __builtin_bit_cast(bf16x8_t, wh[z]),
                            p, 0, 0, 0);
                        const float s = __uint_as_float(z == 0 ? sg[j] : su[j]);
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[z][r] = __builtin_fmaf(s, p[r], acc[z][r]);
                    }
                }
            };
            if (f0 < a.F) {  // else a tile of the last group's padding
                load(min(wave, nchunk - 1), g0, u0);
                for (int s0 = 0; s0 < G; s0 += S) {
                    lds_barrier();  // the stage is read
                    // token rows of the slab, zero past D
                    const int vals = S * 64 / 4;
                    for (int v = tid; v < nt * vals; v += 64 * W) {
                        const int m = v / vals, d4 = v % vals * 4;
                        uint32_t left = who;
                        for (int z = 0; z < p0 + m; ++z) left &= left - 1;
                        const int t = __ffs(left) - 1;
                        const int64_t d = (int64_t)s0 * 64 + d4;
                        uint32_t b[3][4];
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const bool in = d + z < a.D;
                            const int64_t at = (int64_t)t * a.D + (in ? d + z : 0);
                            if constexpr (BF16) {
                                const uint32_t q = static_cast<const uint16_t*>(a.X)[at];
                                b[0][z] = in ? q : 0u;
                            } else {
                                const float q = static_cast<const float*>(a.X)[at];
                                split3(in ? q : 0.0f, b[0][z], b[1][z], b[2][z]);
                            }
                        }
#pragma unroll
                        for (int pc = 0; pc < (BF16 ? 1 : 3); ++pc)
                            *reinterpret_cast<u32x2_t*>(stage + ((BF16 ? m : 3 * m + pc) * pitch) +
                                                        2 * d4) =
                                u32x2_t{b[pc][0] | b[pc][1] << 16, b[pc][2] | b[pc][3] << 16};
                    }
                    lds_barrier();
                    const int cend = min(nchunk, (s0 + S) / 4);
                    for (int c = s0 / 4 + wave; c < cend; c += W) {
                        load(min(c + W, nchunk - 1), g1, u1);
                        mul(c, s0, g0, u0);
                        g0 = g1;
                        u0 = u1;
                    }
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
                const int64_t at =
                    (int64_t)(rt.first[i] + p0 + m) * (x.GF * 64) + f0 + c;
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
template <int DB, int MT, bool BF16>
__global__ __launch_bounds__(64 * kDownWaves) void moe_few_down_kernel(const FewKernelArgs x) {
    constexpr int W = kDownWaves;
    constexpr int TPT = BF16 ? 8 : 4;  // tokens of a row tile
    constexpr int BY = DB == 3 ? kGroupBytes : kGroupBytesI4;
    const FewArgs& a = x.a;
    __shared__ __attribute__((aligned(16))) f32x4_t red[W][MT][64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int h4 = lane >> 4, l16 = lane & 15;
    const int G = x.GF, nchunk = (G + 3) / 4;
    const int64_t o0 = (int64_t)blockIdx.x * 16;
    const int n = x.count[0], units = n * nchunk;
    const int64_t orow = min<int64_t>(o0 + l16, a.D - 1);
    const int64_t plane = (int64_t)x.pairs * G * 64;
    const int piece = BF16 ? l16 & 1 : min(l16 & 3, 2);
    f32x4_t acc[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    struct Unit {
        Piece<DB> w;
        const uint16_t* row[MT];  // this lane's operand row at the chunk's first group
        float wt[MT][BF16 ? 2 : 1];
        bool live[MT];
    };
    auto load = [&](int u, Unit& k) {
        const int i = u / nchunk, c = u % nchunk;
        const int q = min(4 * c + h4, G - 1);
        const int64_t r = ((int64_t)x.count[4 + i] * a.D + orow) * G + q;
        k.w.w.load(a.down.packed + r * BY);
        k.w.s = a.down.scales[r];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int t = min(mt * TPT + (BF16 ? l16 >> 1 : l16 >> 2), a.T - 1);
            k.row[mt] = x.planes + piece * plane + (int64_t)x.prow[i * a.T + t] * (G * 64) +
                        c * 256 + 16 * h4;
            float any = 0.0f;
#pragma unroll
            for (int z = 0; z < (BF16 ? 2 : 1); ++z) {
                const int tt = mt * TPT + (BF16 ? 2 * h4 + z : h4);
                k.wt[mt][z] = tt < a.T ? x.weight[i * a.T + tt] : 0.0f;
                any += k.wt[mt][z];
            }
            k.live[mt] = __any(any != 0.0f);
        }
    };
    auto mul = [&](int u, const Unit& k) {
        const int c = u % nchunk;
        Quarter qd[4];
        k.w.w.quarters(qd);
        uint32_t sd[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sd[j] = 4 * c + h4 < G ? __float_as_uint(k.w.s * code_unit(DB)) : 0u;
        transpose_rows(sd);
        f32x4_t part[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) part[mt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = min(j, G - 1 - 4 * c) * 64;  // past the row: a valid group, scale 0
            u32x4_t wl, wh;
            exact_quarter(qd[j], h4, DB, wl, wh);
            const float s = __uint_as_float(sd[j]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if (MT > 1 && !k.live[mt]) continue;
                const u32x4_t* xp = reinterpret_cast<const u32x4_t*>(k.row[mt] + at);
                f32x4_t p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8_t, xp[0]), __builtin_bit_cast(bf16x8_t, wl),
                    f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0);
                p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, xp[1]),
                                                            __builtin_bit_cast(bf16x8_t, wh), p, 0,
                                                            0, 0);
#pragma unroll
                for (int r = 0; r < 4; ++r) part[mt][r] = __builtin_fmaf(s, p[r], part[mt][r]);
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if (MT > 1 && !k.live[mt]) continue;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                // another token's products, whatever they are, do not count
                const float w = k.wt[mt][BF16 ? r >> 1 : 0];
                acc[mt][r] = __builtin_fmaf(w, w != 0.0f ? part[mt][r] : 0.0f, acc[mt][r]);
            }
        }
    };
    if (wave < units) {
        Unit k0, k1;
        load(wave, k0);
        for (int u = wave;; u += 2 * W) {
            load(min(u + W, units - 1), k1);
            mul(u, k0);
            if (u + W >= units) break;
            load(min(u + 2 * W, units - 1), k0);
            mul(u + W, k1);
            if (u + 2 * W >= units) break;
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
    const unsigned grid = (unsigned)std::min<int64_t>(items, 1024);
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
    const hipError_t e = a.bf16 ? up_bits<true>(x, s) : up_bits<false>(x, s);
    if (e != hipSuccess) return e;
    if (a.down.bits == 3) return a.bf16 ? run_down<3, true>(x, s) : run_down<3, false>(x, s);
    return a.bf16 ? run_down<4, true>(x, s) : run_down<4, false>(x, s);
}

}  // namespace qt
