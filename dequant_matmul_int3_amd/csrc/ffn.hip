// The gated feed-forward block's first half on packed weights:
//   H[t,f] = act(sum_i Wg[f,i] X[t,i]) * (sum_i Wu[f,i] X[t,i])
// with both projections, the activation and the product in one kernel; on
// request the pre-activations are kept in f32 for the backward pass.
//
// f32 inputs are split exactly into three bf16 pieces (a small launch writes
// them as planes), so that both types run on the bf16 matrix cores; bf16
// inputs whose rows are not whole groups are copied into padded planes.
//
// Small form (up to 64 rows of bf16 or pieces): the weights' stream bounds
// it.  A block of W waves owns 16 features; a lane loads whole 24- or 32-byte
// groups of one row of each projection (four groups of a row lie next to each
// other), the waves take different groups, and the codes enter the matrix
// cores exactly: each group's products are summed in f32 and scaled by the
// group's f32 scale, as the vector forms of the library do.
//
// Tile form: a block of 8 waves owns 128 MT tokens x 64 features of both
// projections and walks the inner axis one group at a time; the weights are
// unpacked once per block into LDS in matrix-operand order, the inputs go
// straight from global memory into registers.  bf16 inputs take the weights
// as bf16(s v), one rounding of each weight to the inputs' type: it saves two
// f32 FMAs per matrix instruction, which do not hide behind the matrix cores
// on this chip.  f32 inputs keep the exact codes and the f32 scale per group.
#include <algorithm>

#include "lds_barrier.h"
#include "tune.h"
#include "unpack.h"

namespace qt {
namespace {

// ------------------------------------------------------------ input planes
// X [T x D] -> planes [NP][T][Dp] bf16: the value itself (bf16) or its three
// pieces (f32), zero past D.
template <bool BF16>
__global__ __launch_bounds__(256) void planes_kernel(const void* __restrict__ X, int64_t T,
                                                     int64_t D, int64_t Dp,
                                                     uint16_t* __restrict__ P) {
    const int64_t per = Dp / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= T * per) return;
    const int64_t t = i / per, d0 = (i - t * per) * 8;
    uint32_t h[8], m[8], l[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const bool in = d0 + e < D;
        const int64_t at = t * D + (in ? d0 + e : 0);
        if constexpr (BF16) {
            const uint32_t b = reinterpret_cast<const uint16_t*>(X)[at];
            h[e] = in ? b : 0u;
        } else {
            const float f = reinterpret_cast<const float*>(X)[at];
            split3(in ? f : 0.0f, h[e], m[e], l[e]);
        }
    }
    auto put = [&](int64_t plane, const uint32_t (&v)[8]) {
        *reinterpret_cast<u32x4_t*>(P + (plane * T + t) * Dp + d0) =
            u32x4_t{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16};
    };
    put(0, h);
    if constexpr (!BF16) {
        put(1, m);
        put(2, l);
    }
}

// --------------------------------------------------------------- small form
template <int BITS>
struct RowGroup;  // one lane's group
template <>
struct RowGroup<3> {
    u32x2_t w[3];
    __device__ __forceinline__ void load(const uint8_t* __restrict__ p) {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(p) + i);
    }
    // lane row h gets quarter h of the four lane rows' groups
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
            w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p) + i);
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

struct SmallArgs {
    const uint8_t *gp, *up;
    const float *gs, *us;
    int64_t F, G, ld;     // ld: row stride of A in elements
    const uint16_t* A;    // [R] rows
    int32_t R, T, act;
    void* H;
    float* pre;
    int64_t pre_stride;   // T * F
};

template <int GB, int UB, int MT, bool BF16OUT>
__global__ __launch_bounds__(1024) void ffn_small_kernel(const SmallArgs a) {
    extern __shared__ __attribute__((aligned(16))) float red[];  // [W][2][MT][64] f32x4
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
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        arow[mt] = a.A + (int64_t)std::min(16 * mt + l16, a.R - 1) * a.ld + 16 * h4;

    const int G = (int)a.G;
    const int nchunk = (G + 3) / 4;
    const int c0 = (int)((int64_t)wave * nchunk / W), c1 = (int)((int64_t)(wave + 1) * nchunk / W);

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
            sg[j] = __float_as_uint(k.sg * code_unit(GB));
            su[j] = __float_as_uint(k.su * code_unit(UB));
        }
        transpose_rows(sg);
        transpose_rows(su);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (4 * c + j < G) {  // uniform
                u32x4_t wl[2], wh[2];
                exact_quarter(qg[j], h4, GB, wl[0], wh[0]);
                exact_quarter(qu[j], h4, UB, wl[1], wh[1]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const u32x4_t* ap =
                        reinterpret_cast<const u32x4_t*>(arow[mt] + (int64_t)(4 * c + j) * kGroup);
                    const bf16x8_t alo = __builtin_bit_cast(bf16x8_t, ap[0]);
                    const bf16x8_t ahi = __builtin_bit_cast(bf16x8_t, ap[1]);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        f32x4_t p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            alo, __builtin_bit_cast(bf16x8_t, wl[x]), f32x4_t{0.f, 0.f, 0.f, 0.f},
                            0, 0, 0);
                        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            ahi, __builtin_bit_cast(bf16x8_t, wh[x]), p, 0, 0, 0);
                        const float s = __uint_as_float(x == 0 ? sg[j] : su[j]);
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[x][mt][r] = __builtin_fmaf(s, p[r], acc[x][mt][r]);
                    }
                }
            }
        }
    };
    if (c0 < c1) {
        Chunk k0, k1;
        load(c0, k0);
        for (int c = c0; c < c1; c += 2) {
            load(std::min(c + 1, c1 - 1), k1);
            mul(c, k0);
            if (c + 1 >= c1) break;
            load(std::min(c + 2, c1 - 1), k0);
            mul(c + 1, k1);
        }
    }
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

template <int GB, int UB, int MT>
hipError_t run_small(const SmallArgs& a, bool bf16, hipStream_t s) {
    const int64_t blocks = cdiv(a.F, 16);
    // waves per block: enough that a CU holds about 16 of them, no more than
    // there are chunks of four groups, and what the sums' LDS allows
    const int most = std::min<int64_t>(MT == 1 ? 16 : 8, std::max<int64_t>(1, cdiv(a.G, 4)));
    int W = 4;
    while (W < 16 && blocks * W < 16 * kCUs) W *= 2;
    W = std::min(W, most);
    const size_t lds = (size_t)W * 2 * MT * 64 * 16;
    if (bf16)
        hipLaunchKernelGGL((ffn_small_kernel<GB, UB, MT, true>), dim3((unsigned)blocks),
                           dim3(64 * W), lds, s, a);
    else
        hipLaunchKernelGGL((ffn_small_kernel<GB, UB, MT, false>), dim3((unsigned)blocks),
                           dim3(64 * W), lds, s, a);
    return hipGetLastError();
}

template <int GB, int UB>
hipError_t small_mt(const SmallArgs& a, bool bf16, hipStream_t s) {
    const int mt = (a.R + 15) / 16;
    if (mt == 1) return run_small<GB, UB, 1>(a, bf16, s);
    if (mt == 2) return run_small<GB, UB, 2>(a, bf16, s);
    if (mt == 3) return run_small<GB, UB, 3>(a, bf16, s);
    return run_small<GB, UB, 4>(a, bf16, s);
}

// ---------------------------------------------------------------- tile form
constexpr int kThreads = 512;
constexpr int kNT = kTileN / 16;  // B tiles of a block: even ones gate, odd ones up

struct TileArgs {
    QMat gate, up;
    int64_t F, G;
    const uint16_t* A;   // planes [NP][T][ld]
    int64_t ld, T;
    int act, splits;
    int64_t mblk, nblk;  // token and feature blocks
    void* H;
    float* pre;          // [2][T][F] or null
    float* part;         // [splits][2][T][F], splits > 1
};

// Consecutive block ids run on different XCDs (8 of them, each with its own
// L2): the ids are remapped so that every XCD takes a contiguous range.
__device__ __forceinline__ int64_t xcd_range(int64_t lin, int64_t n) {
    const int64_t x = lin & 7, q = n >> 3, r = n & 7;
    return x * q + std::min(x, r) + (lin >> 3);
}

typedef f32x4_t f32x4_u __attribute__((aligned(4)));
typedef u32x2_t u32x2_u __attribute__((aligned(2)));

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

template <int NP, int MT>
__global__ __launch_bounds__(kThreads) void ffn_tile_kernel(const TileArgs a) {
    constexpr bool EXACT = NP == 3;
    __shared__ __attribute__((aligned(16))) u32x4_t ws[2][kNT * 2 * 64];
    __shared__ __attribute__((aligned(16))) float ss[2][kTileN];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h4 = lane >> 4, l16 = lane & 15;
    const int64_t tile = xcd_range(blockIdx.x, gridDim.x);
    const int64_t n = tile % a.nblk, mm = tile / a.nblk;
    const int64_t m0 = (mm % a.mblk) * (128 * MT);
    const int sp = (int)(mm / a.mblk);
    const int g0 = (int)(a.G * sp / a.splits), g1 = (int)(a.G * (sp + 1) / a.splits);

    // ---- weights: wave w unpacks B tile w, lane = (quarter, row); rows past
    // F read a valid row and are not stored
    const bool is_up = wave & 1;
    const QMat mat = is_up ? a.up : a.gate;
    const int q = h4;
    const int64_t frow = std::min<int64_t>(n * 64 + (wave >> 1) * 16 + l16, a.F - 1);
    const int gby = mat.bits == 3 ? kGroupBytes : kGroupBytesI4;
    const uint8_t* wp = mat.packed + frow * a.G * gby;
    const float* sp_ = mat.scales + frow * a.G;
    struct Raw {
        Quarter w;
        float s;
    };
    auto load_raw = [&](int g, Raw& r) {
        r.w = load_quarter(wp + (int64_t)g * gby, q, mat.bits);
        r.s = sp_[g];
    };
    auto unpack = [&](int buf, const Raw& r) {
        u32x4_t lo8, hi8;
        if constexpr (EXACT) {
            exact_quarter(r.w, q, mat.bits, lo8, hi8);
            if (q == 0) ss[buf][wave * 16 + l16] = r.s * code_unit(mat.bits);
        } else {
            scaled_quarter(r.w, q, mat.bits, r.s, lo8, hi8);
        }
        u32x4_t* d = &ws[buf][(2 * wave + (q >> 1)) * 64 + 32 * (q & 1) + l16];
        d[0] = lo8;
        d[16] = hi8;
    };

    // ---- inputs: lane's 8 consecutive values of its tokens, both 32-deep
    // steps of a group; tokens past T read a valid row
    const uint16_t* ap[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        ap[mt] = a.A +
                 std::min<int64_t>(m0 + wave * (16 * MT) + mt * 16 + l16, a.T - 1) * a.ld + 8 * h4;
    const int64_t plane = a.T * a.ld;
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
                        ap[mt] + p * plane + (int64_t)g * kGroup + 32 * ks);
    };

    f32x4_t acc[MT][kNT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) acc[mt][nt] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // The weights are the first operand: register r of lane l of a product
    // is feature 4 (l / 16) + r and token l % 16.
    auto step = [&](int buf, const In& x) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            bf16x8_t b[2];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
                b[ks] = __builtin_bit_cast(bf16x8_t, ws[buf][(2 * nt + ks) * 64 + lane]);
            f32x4_t sc;
            if constexpr (EXACT) sc = *reinterpret_cast<const f32x4_t*>(&ss[buf][nt * 16 + 4 * h4]);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                f32x4_t part;
                if constexpr (EXACT) part = f32x4_t{0.f, 0.f, 0.f, 0.f};
                else part = acc[mt][nt];
#pragma unroll
                for (int p = 0; p < NP; ++p)
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks)
                        part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            b[ks], __builtin_bit_cast(bf16x8_t, x.v[p][mt][ks]), part, 0, 0, 0);
                if constexpr (EXACT) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[mt][nt][r] = __builtin_fmaf(sc[r], part[r], acc[mt][nt][r]);
                } else {
                    acc[mt][nt] = part;
                }
            }
        }
    };

    // group g: inputs in registers, weights in LDS buffer (g - g0) & 1; the
    // loads of the next group's inputs and of the weights two groups ahead
    // are in flight meanwhile (past the last group they repeat it)
    In x0, x1;
    Raw r0, r1;
    const int last = g1 - 1;
    load_raw(g0, r0);
    load_a(g0, x0);
    load_raw(std::min(g0 + 1, last), r1);
    unpack(0, r0);
    lds_barrier();
    auto group = [&](int g, int buf, const In& xc, In& xn, Raw& rl, const Raw& ru) {
        load_a(std::min(g + 1, last), xn);
        load_raw(std::min(g + 2, last), rl);
        step(buf, xc);
        unpack(1 - buf, ru);
        lds_barrier();
        return g + 1 >= g1;
    };
    for (int g = g0;; g += 2) {
        if (group(g, 0, x0, x1, r0, r1)) break;
        if (group(g + 1, 1, x1, x0, r1, r0)) break;
    }

#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int64_t t = m0 + wave * (16 * MT) + mt * 16 + l16;
        if (t >= a.T) continue;
#pragma unroll
        for (int j = 0; j < kNT / 2; ++j) {
            const int64_t f = n * 64 + j * 16 + 4 * h4;
            const int64_t left = a.F - f, o = t * a.F + f;
            if (left <= 0) continue;
            const f32x4_t g = acc[mt][2 * j], u = acc[mt][2 * j + 1];
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

template <int NP, int MT>
hipError_t run_tile(const TileArgs& a, hipStream_t s) {
    const int64_t nb = a.mblk * a.nblk * a.splits;
    if (nb > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL((ffn_tile_kernel<NP, MT>), dim3((unsigned)nb), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_x_planes(const void* X, bool bf16, int64_t T, int64_t D, uint16_t* planes,
                           hipStream_t s) {
    const int64_t Dp = pad_to(D, kGroup);
    const int64_t nb = cdiv(T * (Dp / 8), 256);
    if (nb > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (bf16)
        hipLaunchKernelGGL((planes_kernel<true>), dim3((unsigned)nb), dim3(256), 0, s, X, T, D, Dp,
                           planes);
    else
        hipLaunchKernelGGL((planes_kernel<false>), dim3((unsigned)nb), dim3(256), 0, s, X, T, D, Dp,
                           planes);
    return hipGetLastError();
}

hipError_t launch_ffn_gated(const FfnArgs& a, void* workspace, hipStream_t s) {
    const FfnPlan p = ffn_plan(a.T, a.D, a.F, a.bf16);
    const int64_t G = cdiv(a.D, kGroup), Dp = G * kGroup;
    const int np = ffn_pieces(a.bf16);
    const uint16_t* A = static_cast<const uint16_t*>(a.X);
    char* w = static_cast<char*>(workspace);
    if (p.planes) {
        uint16_t* planes = reinterpret_cast<uint16_t*>(w + p.planes_off);
        const hipError_t e = launch_x_planes(a.X, a.bf16, a.T, a.D, planes, s);
        if (e != hipSuccess) return e;
        A = planes;
    }
    if (p.small) {
        const SmallArgs sa{a.gate.packed, a.up.packed, a.gate.scales, a.up.scales, a.F, G, Dp, A,
                           (int32_t)(np * a.T), (int32_t)a.T, a.act, a.H, a.pre, a.T * a.F};
        if (a.gate.bits == 3)
            return a.up.bits == 3 ? small_mt<3, 3>(sa, a.bf16, s) : small_mt<3, 4>(sa, a.bf16, s);
        return a.up.bits == 3 ? small_mt<4, 3>(sa, a.bf16, s) : small_mt<4, 4>(sa, a.bf16, s);
    }
    TileArgs ta{a.gate, a.up, a.F, G, A, Dp, a.T, a.act, p.splits, cdiv(a.T, 128 * p.mt),
                cdiv(a.F, kTileN / 2), a.H, a.pre,
                p.splits > 1 ? reinterpret_cast<float*>(w + p.part_off) : nullptr};
    hipError_t e;
    if (a.bf16)
        e = p.mt == 1 ? run_tile<1, 1>(ta, s) : p.mt == 2 ? run_tile<1, 2>(ta, s)
                                                          : run_tile<1, 4>(ta, s);
    else
        e = p.mt == 1 ? run_tile<3, 1>(ta, s) : run_tile<3, 2>(ta, s);
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t n = a.T * a.F, nb = cdiv(n, 1024);
    if (nb > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (a.bf16)
        hipLaunchKernelGGL((ffn_join_kernel<true>), dim3((unsigned)nb), dim3(256), 0, s, ta.part,
                           p.splits, n, a.act, a.H, a.pre);
    else
        hipLaunchKernelGGL((ffn_join_kernel<false>), dim3((unsigned)nb), dim3(256), 0, s, ta.part,
                           p.splits, n, a.act, a.H, a.pre);
    return hipGetLastError();
}

}  // namespace qt
