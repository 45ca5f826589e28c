// The gated feed-forward block's first half on packed weights:
//   H[t,f] = act(sum_i Wg[f,i] X[t,i]) * (sum_i Wu[f,i] X[t,i])
// with both projections, the activation and the product in one kernel; on
// request the pre-activations are kept in f32 for the backward pass.
//
// f32 inputs are split exactly into three bf16 pieces (a small launch writes
// them as planes), so that both types run on the bf16 matrix cores; bf16
// inputs whose rows are not whole groups are copied into padded planes, or a few
// rows into LDS by every block.
//
// Small form (up to 64 rows of bf16 or pieces): the weights' stream bounds
// it.  A block of W waves owns 16 features; a lane loads whole 24- or 32-byte
// groups of one row of each projection (four groups of a row lie next to each
// other), the waves take different groups, and the codes enter the matrix
// cores exactly: each group's products are summed in f32 and scaled by the
// group's f32 scale, as the vector forms of the library do.
//
// One token of 18432 x 7168 (115 MB): 34 us, 3.4 TB/s; it issues 2.8 vector
// instructions per code, about 20 us of the vector ALUs' time.
//
// Tile form: a block of 8 waves owns 128 MT tokens x 8 NT features of both
// projections and walks the inner axis one group at a time.  The inputs are
// laid out as matrix operands by a small launch first and go straight from
// global memory into registers; the weights are unpacked once per block into
// LDS in operand order.  Codes and inputs are exact, each group's products are
// scaled by the f32 scale (two FMAs per matrix instruction): weights rounded to
// bf16(s v) would save them (1.08 against 1.35 ms at 4096 x 5120 x 2 17408) but
// leave the pre-activations 4e-3 off, and with them the f32 gradients of the
// scales.  That shape takes 1.41 ms (1030 TFLOP/s), 1.49 with pre written, the
// matrix cores busy 43 % of the cycles; the FMAs and the unpacking bound it.
#include <algorithm>

#include "lds_barrier.h"
#include "tune.h"
#include "unpack.h"

namespace qt {
namespace {

typedef f32x4_t f32x4_u __attribute__((aligned(4)));
typedef u32x2_t u32x2_u __attribute__((aligned(2)));
typedef u32x4_t u32x4_u __attribute__((aligned(2)));

// ------------------------------------------------------------ input planes
// X [T x D] -> bf16 planes: the value itself (bf16) or its three pieces (f32),
// zero past D.  BLOCKED false: [NP][T][Dp] rows.  BLOCKED true: matrix-operand
// order, [NP][ceil(T/16)][Dp/32] blocks of 64 lanes x 16 bytes (lane l holds
// values 8 (l / 16) .. + 7 of token l % 16), zero past T: every operand load of
// the tiles is then one contiguous kilobyte (rows read in place touch 16 half lines per
// load, at strides that share memory channels).
template <bool BF16, bool BLOCKED>
__global__ __launch_bounds__(256) void planes_kernel(const void* __restrict__ X, int64_t T,
                                                     int64_t D, int64_t Dp,
                                                     uint16_t* __restrict__ P) {
    const int64_t i =
        ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    const int64_t Tp = BLOCKED ? (T + 15) / 16 * 16 : T;
    if (i >= Tp * (Dp / 8)) return;
    int64_t t, d0;
    if constexpr (BLOCKED) {
        const int64_t blk = i >> 6, kb = Dp / 32;
        t = blk / kb * 16 + (i & 15);
        d0 = blk % kb * 32 + ((i & 63) >> 4) * 8;
    } else {
        t = i / (Dp / 8);
        d0 = i % (Dp / 8) * 8;
    }
    uint32_t h[8], m[8], l[8];
    if (BF16 && t < T && d0 + 8 <= D) {
        const uint16_t* x = reinterpret_cast<const uint16_t*>(X) + t * D + d0;
        reinterpret_cast<u32x4_t*>(P)[i] = *reinterpret_cast<const u32x4_u*>(x);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const bool in = t < T && d0 + e < D;
        const int64_t at = in ? t * D + d0 + e : 0;
        if constexpr (BF16) {
            const uint32_t b = reinterpret_cast<const uint16_t*>(X)[at];
            h[e] = in ? b : 0u;
        } else {
            const float f = reinterpret_cast<const float*>(X)[at];
            split3(in ? f : 0.0f, h[e], m[e], l[e]);
        }
    }
    auto put = [&](int64_t plane, const uint32_t (&v)[8]) {
        reinterpret_cast<u32x4_t*>(P)[plane * (Tp * Dp / 8) + i] =
            u32x4_t{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
    };
    put(0, h);
    if constexpr (!BF16) {
        put(1, m);
        put(2, l);
    }
}

// --------------------------------------------------------------- small form
struct SmallArgs {
    const uint8_t *gp, *up;
    const float *gs, *us;
    int64_t F, G, D;
    const void* X;        // rows: bf16 rows of whole groups, 16-byte aligned; else [T x D]
    int32_t R, T, act;    // R: rows of A, the pieces of the T tokens
    void* H;
    float* pre;
    int64_t pre_stride;   // T * F
};

// Where the rows of A come from: bf16 rows in global memory, or LDS, where
// every block copies the (few) tokens' values or pieces first.
enum Rows { kGlobalRows, kStagedBf16, kStagedF32 };
// LDS row of a staged row, in bf16 elements (16 bytes apart in the banks)
__host__ __device__ inline int64_t staged_row(int64_t G) { return G * kGroup + 8; }

template <int GB, int UB, int MT, Rows ROWS, bool BF16OUT>
__global__ __launch_bounds__(1024) void ffn_small_kernel(const SmallArgs a) {
    // the staged rows, then [W][2][MT][64] f32x4 sums
    extern __shared__ __attribute__((aligned(16))) float red[];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, W = blockDim.x >> 6;
    const int h4 = lane >> 4, l16 = lane & 15;
    const int64_t f0 = (int64_t)blockIdx.x * 16;
    const int64_t row = std::min<int64_t>(f0 + l16, a.F - 1);
    constexpr int GBY = GB == 3 ? kGroupBytes : kGroupBytesI4;
    constexpr int UBY = UB == 3 ? kGroupBytes : kGroupBytesI4;
    const uint8_t* gp = a.gp + row * a.G * GBY;
    const uint8_t* up = a.up + row * a.G * UBY;
    const float* gs = a.gs + row * a.G;
    const float* us = a.us + row * a.G;
    const uint16_t* arow[MT];
    uint16_t* stage = reinterpret_cast<uint16_t*>(red);
    const int srow = (int)staged_row(a.G);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int64_t r = std::min(16 * mt + l16, a.R - 1);
        if constexpr (ROWS == kGlobalRows)
            arow[mt] = static_cast<const uint16_t*>(a.X) + r * a.G * kGroup + 16 * h4;
        else
            arow[mt] = stage + r * srow + 16 * h4;
    }

    const int G = (int)a.G;
    const int nchunk = (G + 3) / 4;

    f32x4_t acc[2][MT];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) acc[x][mt] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    struct Chunk {
        RowGroup<GB> g;
        RowGroup<UB> u;
        float sg, su;
    };
    // four groups of the lane's row, one per lane row; past the row a valid
    // group is read and not used
    auto load = [&](int c, Chunk& k) {
        const int g = std::min(4 * c + h4, G - 1);
        k.g.load(gp + (int64_t)g * GBY);
        k.u.load(up + (int64_t)g * UBY);
        k.sg = gs[g];
        k.su = us[g];
    };
    auto mul = [&](int c, const Chunk& k) {
        Quarter qg[4], qu[4];
        k.g.quarters(qg);
        k.u.quarters(qu);
        uint32_t sg[4], su[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            sg[j] = 4 * c + h4 < G ? __float_as_uint(k.sg * code_unit(GB)) : 0u;
            su[j] = 4 * c + h4 < G ? __float_as_uint(k.su * code_unit(UB)) : 0u;
        }
        transpose_rows(sg);
        transpose_rows(su);
        // the rows of group j + 1 are read while group j is multiplied; groups
        // past the row read a valid one and have the scale 0
        u32x4_t x[2][MT][2];
        auto read_x = [&](int j) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const u32x4_t* p = reinterpret_cast<const u32x4_t*>(
                    arow[mt] + std::min(4 * c + j, G - 1) * kGroup);
                x[j & 1][mt][0] = p[0];
                x[j & 1][mt][1] = p[1];
            }
        };
        read_x(0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j < 3) read_x(j + 1);
            {
                u32x4_t wl[2], wh[2];
                exact_quarter(qg[j], h4, GB, wl[0], wh[0]);
                exact_quarter(qu[j], h4, UB, wl[1], wh[1]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const bf16x8_t alo = __builtin_bit_cast(bf16x8_t, x[j & 1][mt][0]);
                    const bf16x8_t ahi = __builtin_bit_cast(bf16x8_t, x[j & 1][mt][1]);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        f32x4_t p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            alo, __builtin_bit_cast(bf16x8_t, wl[i]), f32x4_t{0.f, 0.f, 0.f, 0.f},
                            0, 0, 0);
                        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            ahi, __builtin_bit_cast(bf16x8_t, wh[i]), p, 0, 0, 0);
                        const float s = __uint_as_float(i == 0 ? sg[j] : su[j]);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[i][mt][r] = __builtin_fmaf(s, p[r], acc[i][mt][r]);
                    }
                }
            }
        }
    };
    Chunk k0, k1;
    load(std::min(wave, nchunk - 1), k0);
    if constexpr (ROWS != kGlobalRows) {
        // the first chunk's weights are in flight meanwhile
        const int nv = G * kGroup / 8;  // eight values at a time
        constexpr int ESZ = ROWS == kStagedBf16 ? 2 : 4, N4 = ESZ / 2;
        const bool vec = a.D % 8 == 0 && (reinterpret_cast<uintptr_t>(a.X) & 15) == 0;
        for (int t = 0; t < a.T; ++t) {
            const char* x = static_cast<const char*>(a.X) + (int64_t)t * a.D * ESZ;
            auto put = [&](int v, const u32x4_t* w) {
                if constexpr (ROWS == kStagedBf16) {
                    *reinterpret_cast<u32x4_t*>(stage + t * srow + 8 * v) = w[0];
                } else {
                    u32x4_t o[3];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t h[2], m[2], l[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            split3(__uint_as_float(w[e >> 1][2 * (e & 1) + i]), h[i], m[i], l[i]);
                        o[0][e] = h[0] | h[1] << 16;
                        o[1][e] = m[0] | m[1] << 16;
                        o[2][e] = l[0] | l[1] << 16;
                    }
#pragma unroll
                    for (int pc = 0; pc < 3; ++pc)
                        *reinterpret_cast<u32x4_t*>(stage + (pc * a.T + t) * srow + 8 * v) = o[pc];
                }
            };
            if (vec) {
                // four pieces in flight; those past D read the row's first and
                // become zero
                for (int v0 = tid; v0 < nv; v0 += 4 * blockDim.x) {
                    u32x4_t w[4][N4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int v = v0 + k * blockDim.x;
                        const bool in = 8 * (int64_t)v < a.D;
#pragma unroll
                        for (int i = 0; i < N4; ++i)
                            w[k][i] = *reinterpret_cast<const u32x4_t*>(
                                x + (in ? (int64_t)v * 8 * ESZ : 0) + 16 * i);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int v = v0 + k * blockDim.x;
                        if (8 * (int64_t)v >= a.D)
#pragma unroll
                            for (int i = 0; i < N4; ++i) w[k][i] = u32x4_t{0u, 0u, 0u, 0u};
                        if (v < nv) put(v, w[k]);
                    }
                }
            } else {
                for (int v = tid; v < nv; v += blockDim.x) {
                    uint32_t e[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t d = std::min<int64_t>(8 * (int64_t)v + i, a.D - 1);
                        if constexpr (ROWS == kStagedBf16)
                            e[i] = reinterpret_cast<const uint16_t*>(x)[d];
                        else
                            e[i] = reinterpret_cast<const uint32_t*>(x)[d];
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (8 * (int64_t)v + i >= a.D) e[i] = 0u;
                    u32x4_t w[N4];
                    if constexpr (ROWS == kStagedBf16) {
                        w[0] = u32x4_t{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16,
                                       e[6] | e[7] << 16};
                    } else {
                        w[0] = u32x4_t{e[0], e[1], e[2], e[3]};
                        w[N4 - 1] = u32x4_t{e[4], e[5], e[6], e[7]};
                    }
                    put(v, w);
                }
            }
        }
        __syncthreads();
    }
    // The waves take the chunks in turn, so that a block reads a row's bytes in
    // order: a chunk of 96 bytes ends inside a line, and waves that each took a
    // range of their own fetched most lines twice (for 12 tokens of
    // 18432 x 7168 85 us against 56).
    for (int c = wave; c < nchunk; c += 2 * W) {
        load(std::min(c + W, nchunk - 1), k1);
        mul(c, k0);
        if (c + W >= nchunk) break;
        load(std::min(c + 2 * W, nchunk - 1), k0);
        mul(c + W, k1);
    }
    if constexpr (ROWS != kGlobalRows) __syncthreads();  // the sums take the rows' place
    // the waves' sums in wave order, then rows [m][16] of both projections
    f32x4_t* r4 = reinterpret_cast<f32x4_t*>(red);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) r4[(wave * 2 * MT + x * MT + mt) * 64 + lane] = acc[x][mt];
    __syncthreads();
    constexpr int N4 = 2 * MT * 64;
    for (int i = tid; i < N4; i += blockDim.x) {
        f32x4_t s = r4[i];
        for (int w = 1; w < W; ++w) s += r4[w * N4 + i];
        r4[i] = s;  // only this thread reads or writes slot i of any wave
    }
    __syncthreads();
    // element (x, m, c): lane 16 (m % 16 / 4) + c of tile m / 16, register m % 4
    auto at = [&](int x, int m, int c) {
        return red[((x * MT + (m >> 4)) * 64 + 16 * ((m & 15) >> 2) + c) * 4 + (m & 3)];
    };
    const int np = a.R / a.T;
    for (int i = tid; i < a.T * 16; i += blockDim.x) {
        const int t = i >> 4, c = i & 15;
        if (f0 + c >= a.F) continue;
        float g = at(0, t, c), u = at(1, t, c);
        for (int p = 1; p < np; ++p) {
            g += at(0, p * a.T + t, c);
            u += at(1, p * a.T + t, c);
        }
        const int64_t o = (int64_t)t * a.F + f0 + c;
        if (a.pre) {
            a.pre[o] = g;
            a.pre[a.pre_stride + o] = u;
        }
        const float h = act_value(g, a.act) * u;
        if constexpr (BF16OUT)
            static_cast<__bf16*>(a.H)[o] = (__bf16)h;
        else
            static_cast<float*>(a.H)[o] = h;
    }
}

template <int GB, int UB, int MT, Rows ROWS, bool BF16OUT>
hipError_t run_small(const SmallArgs& a, hipStream_t s) {
    const int64_t blocks = cdiv(a.F, 16);
    // waves per block: enough that a CU holds about 16 of them, no more than
    // there are chunks of four groups, and what the sums' LDS allows
    const int most = std::min<int64_t>(MT == 1 ? 16 : 8, std::max<int64_t>(1, cdiv(a.G, 4)));
    int W = 4;
    while (W < 16 && blocks * W < 16 * kCUs) W *= 2;
    W = std::min(W, most);
    size_t lds = (size_t)W * 2 * MT * 64 * 16;
    if (ROWS != kGlobalRows) lds = std::max(lds, (size_t)(a.R * staged_row(a.G) * 2));
    hipLaunchKernelGGL((ffn_small_kernel<GB, UB, MT, ROWS, BF16OUT>), dim3((unsigned)blocks),
                       dim3(64 * W), lds, s, a);
    return hipGetLastError();
}

template <int GB, int UB>
hipError_t small_bits(const SmallArgs& a, bool bf16, bool staged, hipStream_t s) {
    if (staged)
        return bf16 ? run_small<GB, UB, 1, kStagedBf16, true>(a, s)
                    : run_small<GB, UB, 1, kStagedF32, false>(a, s);
    const int mt = (a.R + 15) / 16;
#define QT_SMALL(M)                                                   \
    return bf16 ? run_small<GB, UB, M, kGlobalRows, true>(a, s)       \
                : run_small<GB, UB, M, kGlobalRows, false>(a, s)
    if (mt == 1) QT_SMALL(1);
    if (mt == 2) QT_SMALL(2);
    if (mt == 3) QT_SMALL(3);
    QT_SMALL(4);
#undef QT_SMALL
}

// ---------------------------------------------------------------- tile form
constexpr int kThreads = kTileThreads;

struct TileArgs {
    QMat gate, up;
    int64_t F, G;
    const uint16_t* A;   // blocked planes [NP][T16][2 G] of 1 KB
    int64_t T;
    int act, splits;
    int64_t mblk, nblk;  // token and feature blocks
    void* H;
    float* pre;          // [2][T][F] or null
    float* part;         // [splits][2][T][F], splits > 1
};

// four consecutive values of a row, those before `left` only
__device__ __forceinline__ void store4(float* p, const f32x4_t& v, int64_t left) {
    if (left >= 4) {
        *reinterpret_cast<f32x4_u*>(p) = v;
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (r < left) p[r] = v[r];
    }
}
__device__ __forceinline__ void store4(__bf16* p, const f32x4_t& v, int64_t left) {
    if (left >= 4) {
        *reinterpret_cast<u32x2_u*>(p) = u32x2_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (r < left) p[r] = (__bf16)v[r];
    }
}

// NP pieces per input, MT 16-token tiles per wave, NT weight tiles (an
// even number) per block; a weight tile is 8 gate rows and 8 up rows of the same features.
template <int GB, int UB, int NP, int MT, int NT>
__global__ __launch_bounds__(kThreads) void ffn_tile_kernel(const TileArgs a) {
    // eight weight tiles, one per wave, of which NT are used: every wave runs
    // the same straight code
    __shared__ __attribute__((aligned(16))) u32x4_t ws[2][8 * 2 * 64];
    __shared__ __attribute__((aligned(16))) float ss[2][8 * 16];
    __shared__ __attribute__((aligned(16))) float turn[8 * 16 * (NT * 16 + 4)];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h4 = lane >> 4, l16 = lane & 15;
    const int64_t tile = xcd_range(blockIdx.x, gridDim.x);
    const int64_t n = tile % a.nblk, mm = tile / a.nblk;
    const int64_t m0 = (mm % a.mblk) * (128 * MT);
    const int sp = (int)(mm / a.mblk);
    const int G = (int)a.G;
    const int g0 = split_begin(G, sp, a.splits), g1 = split_begin(G, sp + 1, a.splits);

    // ---- weights: wave w unpacks weight tile w (four groups' words at a
    // time); rows past F read a valid row and are not stored
    RowFeed<GB, UB> feed;
    feed.init(a.gate, a.up, l16 >= 8,
              std::min<int64_t>(n * (NT * 8) + wave * 8 + (l16 & 7), a.F - 1), G, h4);
    feed.load(g0);
    // word j of the feed, group g, into LDS buffer buf; groups past the block's
    // range get the scale 0 and add nothing
    auto unpack = [&](int buf, int j, int g) {
        u32x4_t lo8, hi8;
        feed.exact(j, h4, lo8, hi8);
        u32x4_t* d = &ws[buf][(2 * wave + (h4 >> 1)) * 64 + 32 * (h4 & 1) + l16];
        d[0] = lo8;
        d[16] = hi8;
        ss[buf][wave * 16 + l16] = g < g1 ? feed.scale(j) : 0.0f;  // four lanes, one value
    };

    // ---- inputs: one kilobyte per 16 tokens and 32 inner elements; token
    // tiles past T read a valid one
    const int64_t t16 = (a.T + 15) / 16, plane = t16 * 2 * G * 512;
    const uint16_t* ap[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        ap[mt] = a.A + std::min<int64_t>(m0 / 16 + wave * MT + mt, t16 - 1) * (2 * G * 512) + 8 * lane;
    struct In {
        u32x4_t v[NP][MT][2];
    };
    auto load_a = [&](int g, In& x) {
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
                    x.v[p][mt][ks] = *reinterpret_cast<const u32x4_t*>(
                        ap[mt] + p * plane + (int64_t)(2 * g + ks) * 512);
    };

    f32x4_t acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // One group: products of the inputs x and LDS buffer buf, and the unpacking
    // of word j of the feed into the other buffer.  Register r of lane l of a
    // product is token 4 (l / 16) + r and weight row l % 16, so a lane needs one
    // scale per weight tile (the other way round it needs four, and their LDS
    // reads took half as long as the operands').  A weight tile's operands are
    // read one tile ahead, a product's scale FMAs follow two products later,
    // and the scheduling groups ask for vector instructions after every matrix
    // instruction: they fill the matrix core's shadow.
    auto step = [&](int buf, const In& x, int j, int gnext) {
        bf16x8_t b[2][2];
        float sc[NT];
        f32x4_t part[3];
        auto read_b = [&](int nt) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
                b[nt & 1][ks] = __builtin_bit_cast(bf16x8_t, ws[buf][(2 * nt + ks) * 64 + lane]);
        };
        read_b(0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sc[nt] = ss[buf][nt * 16 + l16];
#pragma unroll
        for (int q = 0; q < NT * MT + 2; ++q) {
            const int nt = q / MT, mt = q % MT, pn = (q - 2) / MT, pm = (q - 2) % MT;
            if (mt == 0 && nt + 1 < NT) read_b(nt + 1);
            if (q < NT * MT) {
                f32x4_t p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int pc = 0; pc < NP; ++pc)
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks)
                        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8_t, x.v[pc][mt][ks]), b[nt & 1][ks], p, 0, 0,
                            0);
                part[q % 3] = p;
            }
            if (q >= 2) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[pm][pn][r] = __builtin_fmaf(sc[pn], part[(q - 2) % 3][r], acc[pm][pn][r]);
            }
            if (q == NT * MT / 2) unpack(1 - buf, j, gnext);
        }
        // 0x8: matrix instruction, 0x2: other vector instruction
#pragma unroll
        for (int i = 0; i < 2 * NP * NT * MT; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x2, 2, 0);
        }
    };

    // group g: inputs in registers, weights in LDS buffer (g - g0) & 1; the
    // loads of the next group's inputs are in flight meanwhile (past the last
    // group of the row they repeat it).  The feed's words of four groups are exchanged in
    // every fourth step, when the words of the four before are used up, and
    // the loads of the next four are issued.
    In x0, x1;
    load_a(g0, x0);
    feed.take();
    feed.load(g0 + 4);
    unpack(0, 0, g0);
    lds_barrier();
    auto group = [&](int g, int j, const In& xc, In& xn) {
        load_a(std::min(g + 1, G - 1), xn);
        if (j == 3) {
            feed.take();
            feed.load(g + 5);
        }
        step(j & 1, xc, (j + 1) & 3, g + 1);
        lds_barrier();
    };
    // four groups per turn with one exit (several exits with the accumulators
    // live made the compiler spill them)
    for (int g = g0; g < g1; g += 4) {
        group(g, 0, x0, x1);
        group(g + 1, 1, x1, x0);
        group(g + 2, 2, x0, x1);
        group(g + 3, 3, x1, x0);
    }

    // Each wave turns 16 tokens at a time through LDS, so that a lane ends with
    // four consecutive features of a token, gate and up.
    constexpr int kRow = NT * 16 + 4;
    float* tl = turn + wave * 16 * kRow;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                tl[(4 * h4 + r) * kRow + nt * 16 + l16] = acc[mt][nt][r];
        lds_wave_sync();
#pragma unroll
        for (int i = 0; i < NT / 2; ++i) {
            const int k = i * 64 + lane, tt = k / (2 * NT), qd = k % (2 * NT);
            const f32x4_t* at =
                reinterpret_cast<const f32x4_t*>(&tl[tt * kRow + (qd >> 1) * 16 + (qd & 1) * 4]);
            const f32x4_t g = at[0], u = at[2];
            const int64_t t = m0 + wave * (16 * MT) + mt * 16 + tt;
            const int64_t f = n * (NT * 8) + 4 * qd;
            const int64_t left = a.F - f, o = t * a.F + f;
            if (t >= a.T || left <= 0) continue;
            if (a.splits > 1) {
                float* p = a.part + (int64_t)sp * 2 * a.T * a.F + o;
                store4(p, g, left);
                store4(p + a.T * a.F, u, left);
            } else {
                if (a.pre) {
                    store4(a.pre + o, g, left);
                    store4(a.pre + a.T * a.F + o, u, left);
                }
                f32x4_t h;
#pragma unroll
                for (int r = 0; r < 4; ++r) h[r] = act_value(g[r], a.act) * u[r];
                if constexpr (NP == 1) store4(static_cast<__bf16*>(a.H) + o, h, left);
                else store4(static_cast<float*>(a.H) + o, h, left);
            }
        }
        lds_wave_sync();  // the next 16 tokens take their place
    }
}

// Joins the splits' sums in split order, then the activation and product.
template <bool BF16>
__global__ __launch_bounds__(256) void ffn_join_kernel(const float* __restrict__ part, int splits,
                                                       int64_t n, int act, void* H, float* pre) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    const int64_t left = n - i;
    f32x4_t g = {0.f, 0.f, 0.f, 0.f}, u = g;
    for (int s = 0; s < splits; ++s) {
        const float* p = part + (int64_t)s * 2 * n + i;
        if (left >= 4) {
            g += *reinterpret_cast<const f32x4_u*>(p);
            u += *reinterpret_cast<const f32x4_u*>(p + n);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (r < left) {
                    g[r] += p[r];
                    u[r] += p[n + r];
                }
        }
    }
    if (pre) {
        store4(pre + i, g, left);
        store4(pre + n + i, u, left);
    }
    f32x4_t h;
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = act_value(g[r], act) * u[r];
    if constexpr (BF16) store4(static_cast<__bf16*>(H) + i, h, left);
    else store4(static_cast<float*>(H) + i, h, left);
}

template <int GB, int UB, int NP, int MT, int NT>
hipError_t run_tile(const TileArgs& a, hipStream_t s) {
    const int64_t nb = a.mblk * a.nblk * a.splits;
    hipLaunchKernelGGL((ffn_tile_kernel<GB, UB, NP, MT, NT>), dim3((unsigned)nb),
                       dim3(kThreads), 0, s, a);
    return hipGetLastError();
}
template <int NP, int MT, int NT>
hipError_t tile_bits(const TileArgs& a, hipStream_t s) {
    if (a.gate.bits == 3)
        return a.up.bits == 3 ? run_tile<3, 3, NP, MT, NT>(a, s) : run_tile<3, 4, NP, MT, NT>(a, s);
    return a.up.bits == 3 ? run_tile<4, 3, NP, MT, NT>(a, s) : run_tile<4, 4, NP, MT, NT>(a, s);
}

}  // namespace

hipError_t launch_x_planes(const void* X, bool bf16, bool blocked, int64_t T, int64_t D,
                           uint16_t* planes, hipStream_t s) {
    const int64_t Dp = pad_to(D, kGroup);
    const GridRows g = grid_rows(x_planes_blocks(T, D, blocked), 256);
    const dim3 grid(g.x, g.y), block(256);
#define QT_PLANES(B, K) \
    hipLaunchKernelGGL((planes_kernel<B, K>), grid, block, 0, s, X, T, D, Dp, planes)
    if (bf16) {
        if (blocked) QT_PLANES(true, true);
        else QT_PLANES(true, false);
    } else {
        if (blocked) QT_PLANES(false, true);
        else QT_PLANES(false, false);
    }
#undef QT_PLANES
    return hipGetLastError();
}

hipError_t launch_ffn_gated(const FfnArgs& a, void* workspace, hipStream_t s) {
    const FfnPlan p = ffn_plan(a.T, a.D, a.F, a.bf16);
    if (!ffn_fits(p, a.T, a.F)) return hipErrorInvalidValue;
    const int64_t G = cdiv(a.D, kGroup);
    const int np = ffn_pieces(a.bf16);
    const uint16_t* A = static_cast<const uint16_t*>(a.X);
    char* w = static_cast<char*>(workspace);
    if (p.planes) {
        uint16_t* planes = reinterpret_cast<uint16_t*>(w + p.planes_off);
        const hipError_t e = launch_x_planes(a.X, a.bf16, !p.small, a.T, a.D, planes, s);
        if (e != hipSuccess) return e;
        A = planes;
    }
    if (p.small) {
        const SmallArgs sa{a.gate.packed, a.up.packed, a.gate.scales, a.up.scales, a.F, G, a.D, A,
                           (int32_t)(np * a.T), (int32_t)a.T, a.act, a.H, a.pre, a.T * a.F};
        if (a.gate.bits == 3)
            return a.up.bits == 3 ? small_bits<3, 3>(sa, a.bf16, p.staged, s)
                                  : small_bits<3, 4>(sa, a.bf16, p.staged, s);
        return a.up.bits == 3 ? small_bits<4, 3>(sa, a.bf16, p.staged, s)
                              : small_bits<4, 4>(sa, a.bf16, p.staged, s);
    }
    TileArgs ta{a.gate, a.up, a.F, G, A, a.T, a.act, p.splits, cdiv(a.T, 128 * p.mt),
                cdiv(a.F, 8 * p.nt), a.H, a.pre,
                p.splits > 1 ? reinterpret_cast<float*>(w + p.part_off) : nullptr};
    hipError_t e;
    if (a.bf16)
        e = p.mt == 1   ? tile_bits<1, 1, 8>(ta, s)
            : p.mt == 2 ? tile_bits<1, 2, 8>(ta, s)
                        : tile_bits<1, 4, 6>(ta, s);
    else
        e = p.mt == 1 ? tile_bits<3, 1, 8>(ta, s) : tile_bits<3, 2, 8>(ta, s);
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t n = a.T * a.F, nb = cdiv(n, 1024);
    if (a.bf16)
        hipLaunchKernelGGL((ffn_join_kernel<true>), dim3((unsigned)nb), dim3(256), 0, s, ta.part,
                           p.splits, n, a.act, a.H, a.pre);
    else
        hipLaunchKernelGGL((ffn_join_kernel<false>), dim3((unsigned)nb), dim3(256), 0, s, ta.part,
                           p.splits, n, a.act, a.H, a.pre);
    return hipGetLastError();
}

}  // namespace qt
