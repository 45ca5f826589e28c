// Backward passes through packed weights: the gradient of the input and of
// the group scales, of a linear layer (one matrix) or of the gated
// feed-forward block (two).
//   dX[t,i]  = sum_m sum_o dY_m[t,o] s_m[o,g(i)] v_m[o,i]
//   ds_m[o,g] = sum_t dY_m[t,o] sum_{j<64} v_m[o,64g+j] X[t,64g+j]
// For the block dY_0 = dH u act'(g) and dY_1 = dH act(g), from the
// pre-activations g, u that the forward pass kept in f32.
//
// Input gradient.  A matrix product with the weights' rows as its inner axis:
// a block of 8 waves owns 128 MT tokens x 128 inputs and walks the rows of
// both matrices 64 at a time.  dY is first written as one padded plane per
// matrix; the weights are unpacked once per block into LDS row by row and read
// back as matrix operands.
//   bf16: dY and the products s v are rounded once to bf16 (their sums are
//   f32), and the operands come out of LDS through the transposing reads of
//   gfx950, four rows of 16 columns at a time.  A lane's eight inner elements
//   are then rows 4h .. 4h+3 and 16+4h .. 16+4h+3 of a 32-row step, and the
//   dY plane is written in that order.
//   f32: both stay f32, on the f32 matrix instructions.
//
// Scale gradient.  The forward product once more, group by group: the exact
// codes times the inputs (three exact bf16 pieces of an f32 input) give each
// token's sum over the group in f32, which is multiplied by dY[t,o] in f32 and
// summed over the tokens.  dY is held in registers for the whole walk over the
// groups.  Nothing is rounded below f32, and the weights' gradient never
// exists.  Token blocks leave partial sums that a last launch adds in order.
#include <algorithm>

#include "lds_barrier.h"
#include "tune.h"
#include "unpack.h"

namespace qt {
namespace {

constexpr int kThreads = 512;
constexpr int kNT = kTileN / 16;

typedef f32x4_t f32x4_u __attribute__((aligned(4)));
typedef u32x2_t u32x2_u __attribute__((aligned(2)));

__device__ __forceinline__ int64_t xcd_range(int64_t lin, int64_t n) {
    const int64_t x = lin & 7, q = n >> 3, r = n & 7;
    return x * q + std::min(x, r) + (lin >> 3);
}

// Where the gradients dY come from.
struct GradSrc {
    int nmat, act;
    bool dy_bf16;
    const void* dY;    // dH (nmat 2) or dY (nmat 1)
    const float* pre;  // nmat 2: [2][T][O]
    int64_t T, O;
};
__device__ __forceinline__ float load_dy(const GradSrc& s, int64_t at) {
    if (s.dy_bf16)
        return __uint_as_float((uint32_t) static_cast<const uint16_t*>(s.dY)[at] << 16);
    return static_cast<const float*>(s.dY)[at];
}
// dY_m[t, o]
__device__ __forceinline__ float grad_at(const GradSrc& s, int m, int64_t t, int64_t o) {
    const int64_t at = t * s.O + o;
    const float d = load_dy(s, at);
    if (s.nmat == 1) return d;
    float dg, du;
    act_grads(s.pre[at], s.pre[s.T * s.O + at], d, s.act, dg, du);
    return m == 0 ? dg : du;
}

// ----------------------------------------------------------- gradient plane
// [T][nmat Op]: matrix m at columns m Op .., zero past O.  bf16 in the order
// of the transposing reads (position 8h + e of 32 is row 4h + (e & 3) +
// 16 (e >> 2)), f32 in order.
template <bool F32>
__global__ __launch_bounds__(256) void grad_plane_kernel(const GradSrc src, int64_t Op,
                                                         void* __restrict__ P) {
    const int64_t per = Op / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= src.T * per) return;
    const int64_t t = i / per, p0 = (i - t * per) * 8;
    float v[2][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int64_t o =
            F32 ? p0 + e : (p0 & ~31LL) + ((p0 & 31) >> 1) + (e & 3) + 16 * (e >> 2);
        v[0][e] = v[1][e] = 0.0f;
        if (o < src.O) {
            const int64_t at = t * src.O + o;
            const float d = load_dy(src, at);
            if (src.nmat == 1)
                v[0][e] = d;
            else
                act_grads(src.pre[at], src.pre[src.T * src.O + at], d, src.act, v[0][e], v[1][e]);
        }
    }
    for (int m = 0; m < src.nmat; ++m) {
        const int64_t at = t * src.nmat * Op + m * Op + p0;
        if constexpr (F32) {
            f32x4_t* d = reinterpret_cast<f32x4_t*>(static_cast<float*>(P) + at);
            d[0] = f32x4_t{v[m][0], v[m][1], v[m][2], v[m][3]};
            d[1] = f32x4_t{v[m][4], v[m][5], v[m][6], v[m][7]};
        } else {
            *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(P) + at) =
                u32x4_t{bf16_pair(v[m][0], v[m][1]), bf16_pair(v[m][2], v[m][3]),
                        bf16_pair(v[m][4], v[m][5]), bf16_pair(v[m][6], v[m][7])};
        }
    }
}

// ------------------------------------------------------------ input gradient
struct DxArgs {
    QMat mat[2];
    int64_t O, Op, I, G, T, K;  // K = nmat Op
    const void* A;              // gradient plane [T][K]
    int splits;
    int64_t mblk, nblk;
    void* dX;
    float* part;                // [splits][T][I], splits > 1
};

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

template <bool F32, int MT>
__global__ __launch_bounds__(kThreads) void dx_tile_kernel(const DxArgs a) {
    // LDS rows of 128 columns; bf16: 288 bytes, so that four rows of 16
    // columns lie in distinct banks; f32: 528 bytes
    constexpr int kRow = F32 ? kTileN * 4 + 16 : kTileN * 2 + 32;
    __shared__ __attribute__((aligned(16))) uint8_t ws[2][kTileK * kRow];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h4 = lane >> 4, l16 = lane & 15;
    const int64_t tile = xcd_range(blockIdx.x, gridDim.x);
    const int64_t n = tile % a.nblk, mm = tile / a.nblk;
    const int64_t m0 = (mm % a.mblk) * (128 * MT);
    const int sp = (int)(mm / a.mblk);
    const int steps = (int)(a.K / kTileK), half = (int)(a.Op / kTileK);
    const int k0 = (int)((int64_t)steps * sp / a.splits);
    const int k1 = (int)((int64_t)steps * (sp + 1) / a.splits);

    // ---- weights: wave w unpacks rows 8w .. 8w+7 of a step, a lane one
    // quarter of one row; groups past G read a valid group (not stored), rows
    // past O a valid row (their dY is zero)
    const int q8 = lane & 7, q = q8 & 3;
    const int64_t grp = std::min<int64_t>(n * 2 + (q8 >> 2), a.G - 1);
    const int rl = 8 * wave + (lane >> 3);
    struct Raw {
        Quarter w;
        float s;
    };
    auto load_raw = [&](int k, Raw& r) {
        const int m = k >= half;  // uniform
        const QMat& mat = a.mat[m];
        const int64_t row =
            std::min<int64_t>((int64_t)(k - m * half) * kTileK + rl, a.O - 1);
        const int64_t at = row * a.G + grp;
        r.w = load_quarter(mat.packed + at * (mat.bits == 3 ? kGroupBytes : kGroupBytesI4), q,
                           mat.bits);
        r.s = mat.scales[at];
    };
    auto unpack = [&](int buf, int k, const Raw& r) {
        const int bits = a.mat[k >= half].bits;
        uint8_t* d = &ws[buf][rl * kRow + q8 * (F32 ? 64 : 32)];
        if constexpr (F32) {
            float v[16];
            scaled_quarter_f32(r.w, q, bits, r.s, v);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                reinterpret_cast<f32x4_t*>(d)[i] =
                    f32x4_t{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
        } else {
            u32x4_t lo8, hi8;
            scaled_quarter(r.w, q, bits, r.s, lo8, hi8);
            reinterpret_cast<u32x4_t*>(d)[0] = lo8;
            reinterpret_cast<u32x4_t*>(d)[1] = hi8;
        }
    };

    // ---- dY: eight inner elements of the lane's tokens
    constexpr int ESZ = F32 ? 4 : 2;
    const char* ap[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        ap[mt] = static_cast<const char*>(a.A) +
                 (std::min<int64_t>(m0 + wave * (16 * MT) + mt * 16 + l16, a.T - 1) * a.K + 8 * h4) *
                     ESZ;
    struct In {
        u32x4_t v[MT][2][F32 ? 2 : 1];
    };
    auto load_a = [&](int k, In& x) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int p = 0; p < (F32 ? 2 : 1); ++p)
                    x.v[mt][ks][p] = *reinterpret_cast<const u32x4_t*>(
                        ap[mt] + ((int64_t)k * kTileK + 32 * ks) * ESZ + 16 * p);
    };

    f32x4_t acc[MT][kNT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) acc[mt][nt] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // weights first: register r of lane l is input 4 (l / 16) + r, token l % 16
    auto step = [&](int buf, const In& x) {
        if constexpr (F32) {
            const uint8_t* b0 = &ws[buf][8 * h4 * kRow + l16 * 4];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    float b[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        b[e] = *reinterpret_cast<const float*>(b0 + (32 * ks + e) * kRow + nt * 64);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            acc[mt][nt] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                b[e], __uint_as_float(x.v[mt][ks][F32 ? (e >> 2) : 0][e & 3]),
                                acc[mt][nt], 0, 0, 0);
                }
        } else {
            const uint8_t* b0 = &ws[buf][(4 * h4 + (l16 >> 2)) * kRow + 8 * (l16 & 3)];
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    struct {
                        s16x4_t lo, hi;
                    } b;
                    const uint8_t* at = b0 + 32 * ks * kRow + nt * 32;
                    b.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
                    b.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 16 * kRow));
                    const bf16x8_t bv = __builtin_bit_cast(bf16x8_t, b);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        acc[mt][nt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            bv, __builtin_bit_cast(bf16x8_t, x.v[mt][ks][0]), acc[mt][nt], 0, 0, 0);
                }
        }
    };

    In x0, x1;
    Raw r0, r1;
    const int last = k1 - 1;
    load_raw(k0, r0);
    load_a(k0, x0);
    load_raw(std::min(k0 + 1, last), r1);
    unpack(0, k0, r0);
    lds_barrier();
    auto body = [&](int k, int buf, const In& xc, In& xn, Raw& rl_, const Raw& ru) {
        load_a(std::min(k + 1, last), xn);
        load_raw(std::min(k + 2, last), rl_);
        step(buf, xc);
        unpack(1 - buf, std::min(k + 1, last), ru);
        lds_barrier();
        return k + 1 >= k1;
    };
    for (int k = k0;; k += 2) {
        if (body(k, 0, x0, x1, r0, r1)) break;
        if (body(k + 1, 1, x1, x0, r1, r0)) break;
    }

#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int64_t t = m0 + wave * (16 * MT) + mt * 16 + l16;
        if (t >= a.T) continue;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            const int64_t i = n * kTileN + nt * 16 + 4 * h4;
            const int64_t left = a.I - i, o = t * a.I + i;
            if (left <= 0) continue;
            const f32x4_t v = acc[mt][nt];
            if (a.splits > 1 || F32) {
                float* p = a.splits > 1 ? a.part + (int64_t)sp * a.T * a.I + o
                                        : static_cast<float*>(a.dX) + o;
                if (left >= 4) *reinterpret_cast<f32x4_u*>(p) = v;
                else
                    for (int r = 0; r < left; ++r) p[r] = v[r];
            } else {
                __bf16* p = static_cast<__bf16*>(a.dX) + o;
                if (left >= 4)
                    *reinterpret_cast<u32x2_u*>(p) =
                        u32x2_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
                else
                    for (int r = 0; r < left; ++r) p[r] = (__bf16)v[r];
            }
        }
    }
}

// out[i] = sum over the splits in split order (+ out[i] if accumulate).
template <bool BF16>
__global__ __launch_bounds__(256) void sum_parts_kernel(const float* __restrict__ part,
                                                        int64_t stride, int splits, int64_t n,
                                                        int accumulate, void* out) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    const int64_t left = n - i;
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < splits; ++s) {
        const float* p = part + s * stride + i;
        if (left >= 4) v += *reinterpret_cast<const f32x4_u*>(p);
        else
            for (int r = 0; r < left; ++r) v[r] += p[r];
    }
    if constexpr (BF16) {
        __bf16* o = static_cast<__bf16*>(out) + i;
        if (left >= 4)
            *reinterpret_cast<u32x2_u*>(o) = u32x2_t{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
        else
            for (int r = 0; r < left; ++r) o[r] = (__bf16)v[r];
    } else {
        float* o = static_cast<float*>(out) + i;
        if (left >= 4) {
            if (accumulate) v = *reinterpret_cast<const f32x4_u*>(o) + v;
            *reinterpret_cast<f32x4_u*>(o) = v;
        } else {
            for (int r = 0; r < left; ++r) o[r] = accumulate ? o[r] + v[r] : v[r];
        }
    }
}

// ------------------------------------------------------------ scale gradient
struct DsArgs {
    QMat mat[2];
    GradSrc src;
    int64_t G, ld;
    const uint16_t* X;   // planes [NP][T][ld]
    int splits, accumulate;
    int64_t tblk, oblk;  // token blocks, 128-row blocks of one matrix
    float* out[2];       // dscales [O x G] of each matrix (one token block), or
    float* part;         // [tblk][nmat][O][G]
};

template <int NP, int MT>
__global__ __launch_bounds__(kThreads) void ds_tile_kernel(const DsArgs a) {
    __shared__ __attribute__((aligned(16))) u32x4_t ws[2][kNT * 2 * 64];
    __shared__ float red[2][8][kTileN];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h4 = lane >> 4, l16 = lane & 15;
    const int64_t T = a.src.T, O = a.src.O;
    // row blocks of both matrices run fastest: their token block's inputs are
    // shared in the XCD's L2
    int64_t tile = xcd_range(blockIdx.x, gridDim.x);
    const int64_t ob = tile % a.oblk;
    tile /= a.oblk;
    const int m = (int)(tile % a.src.nmat);
    tile /= a.src.nmat;
    const int64_t tb = tile % a.tblk;
    const int sp = (int)(tile / a.tblk);
    const int64_t o0 = ob * kTileN, t0 = tb * (128 * MT) + wave * (16 * MT);
    const int g0 = (int)(a.G * sp / a.splits), g1 = (int)(a.G * (sp + 1) / a.splits);
    const QMat mat = a.mat[m];

    const int q = h4;
    const int64_t wrow = std::min<int64_t>(o0 + wave * 16 + l16, O - 1);
    const int gby = mat.bits == 3 ? kGroupBytes : kGroupBytesI4;
    const uint8_t* wp = mat.packed + wrow * a.G * gby;
    auto load_raw = [&](int g, Quarter& r) {
        r = load_quarter(wp + (int64_t)g * gby, q, mat.bits);
    };
    auto unpack = [&](int buf, const Quarter& r) {
        u32x4_t lo8, hi8;
        exact_quarter(r, q, mat.bits, lo8, hi8);
        u32x4_t* d = &ws[buf][(2 * wave + (q >> 1)) * 64 + 32 * (q & 1) + l16];
        d[0] = lo8;
        d[16] = hi8;
    };
    const uint16_t* xp[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        xp[mt] = a.X + std::min<int64_t>(t0 + mt * 16 + l16, T - 1) * a.ld + 8 * h4;
    const int64_t plane = T * a.ld;
    struct In {
        u32x4_t v[NP][MT][2];
    };
    auto load_x = [&](int g, In& x) {
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
                    x.v[p][mt][ks] = *reinterpret_cast<const u32x4_t*>(
                        xp[mt] + p * plane + (int64_t)g * kGroup + 32 * ks);
    };

    // dY of the tile, where the products will lie: register r of lane l is
    // token 4 (l / 16) + r, row l % 16; zero past T and O
    f32x4_t dy[MT][kNT];
    const float unit = code_unit(mat.bits);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int64_t t = t0 + mt * 16 + 4 * h4 + r, o = o0 + nt * 16 + l16;
                dy[mt][nt][r] = t < T && o < O ? grad_at(a.src, m, t, o) * unit : 0.0f;
            }

    // the tile's sums of one group: per wave over its tokens (lane row h ends
    // with row tiles h and 4 + h ... as the swaps leave them), then the waves
    auto step = [&](int buf, const In& x) {
        float v[kNT];
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            bf16x8_t b[2];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
                b[ks] = __builtin_bit_cast(bf16x8_t, ws[buf][(2 * nt + ks) * 64 + lane]);
            float sum = 0.0f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                f32x4_t p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int pc = 0; pc < NP; ++pc)
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks)
                        p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8_t, x.v[pc][mt][ks]), b[ks], p, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < 4; ++r) sum = __builtin_fmaf(p[r], dy[mt][nt][r], sum);
            }
            v[nt] = sum;
        }
        // sums over the four lane rows: two values' halves are swapped and
        // added, then their quarters; lane row h ends with value 2 (h & 1) +
        // (h >> 1) of each four
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            float w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const auto s = __builtin_amdgcn_permlane32_swap(
                    __float_as_uint(v[4 * f + 2 * i]), __float_as_uint(v[4 * f + 2 * i + 1]), false,
                    false);
                w[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
            }
            const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(w[0]),
                                                            __float_as_uint(w[1]), false, false);
            const int nt = 4 * f + 2 * (h4 & 1) + (h4 >> 1);
            red[buf][wave][nt * 16 + l16] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
        }
    };
    // the waves' sums of group g in wave order (after the barrier)
    auto finish = [&](int buf, int g) {
        if (tid < kTileN && o0 + tid < O) {
            float s = red[buf][0][tid];
#pragma unroll
            for (int w = 1; w < 8; ++w) s += red[buf][w][tid];
            const int64_t at = (o0 + tid) * a.G + g;
            if (a.tblk > 1) {
                a.part[(tb * a.src.nmat + m) * O * a.G + at] = s;
            } else {
                float* d = a.out[m] + at;
                *d = a.accumulate ? *d + s : s;
            }
        }
    };

    In x0, x1;
    Quarter r0, r1;
    const int last = g1 - 1;
    load_raw(g0, r0);
    load_x(g0, x0);
    load_raw(std::min(g0 + 1, last), r1);
    unpack(0, r0);
    lds_barrier();
    auto group = [&](int g, int buf, const In& xc, In& xn, Quarter& rl, const Quarter& ru) {
        load_x(std::min(g + 1, last), xn);
        load_raw(std::min(g + 2, last), rl);
        step(buf, xc);
        unpack(1 - buf, ru);
        lds_barrier();
        finish(buf, g);
        return g + 1 >= g1;
    };
    for (int g = g0;; g += 2) {
        if (group(g, 0, x0, x1, r0, r1)) break;
        if (group(g + 1, 1, x1, x0, r1, r0)) break;
    }
}

template <bool F32, int MT>
hipError_t run_dx(const DxArgs& a, hipStream_t s) {
    const int64_t nb = a.mblk * a.nblk * a.splits;
    if (nb > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL((dx_tile_kernel<F32, MT>), dim3((unsigned)nb), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}
template <int NP, int MT>
hipError_t run_ds(const DsArgs& a, hipStream_t s) {
    const int64_t nb = a.oblk * a.src.nmat * a.tblk * a.splits;
    if (nb > 0x7FFFFFFF) return hipErrorInvalidValue;
    hipLaunchKernelGGL((ds_tile_kernel<NP, MT>), dim3((unsigned)nb), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}
hipError_t sum_parts(const float* part, int64_t stride, int splits, int64_t n, int accumulate,
                     bool bf16, void* out, hipStream_t s) {
    const int64_t nb = cdiv(n, 1024);
    if (nb > 0x7FFFFFFF) return hipErrorInvalidValue;
    if (bf16)
        hipLaunchKernelGGL((sum_parts_kernel<true>), dim3((unsigned)nb), dim3(256), 0, s, part,
                           stride, splits, n, accumulate, out);
    else
        hipLaunchKernelGGL((sum_parts_kernel<false>), dim3((unsigned)nb), dim3(256), 0, s, part,
                           stride, splits, n, accumulate, out);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_bwd(const BwdArgs& a, void* workspace, hipStream_t s) {
    const bool want_dx = a.dX != nullptr, want_ds = a.dscales[0] != nullptr;
    const BwdPlan p = bwd_plan(a.T, a.I, a.O, a.nmat, a.bf16, want_dx, want_ds);
    char* w = static_cast<char*>(workspace);
    const int64_t G = cdiv(a.I, kGroup), Op = pad_to(a.O, kTileK);
    const GradSrc src{a.nmat, a.act, a.dy_bf16, a.dY, a.pre, a.T, a.O};
    hipError_t e;
    if (want_dx) {
        const int64_t nb = cdiv(a.T * (Op / 8), 256);
        if (nb > 0x7FFFFFFF) return hipErrorInvalidValue;
        void* A = w + p.grad_off;
        if (a.bf16)
            hipLaunchKernelGGL((grad_plane_kernel<false>), dim3((unsigned)nb), dim3(256), 0, s, src,
                               Op, A);
        else
            hipLaunchKernelGGL((grad_plane_kernel<true>), dim3((unsigned)nb), dim3(256), 0, s, src,
                               Op, A);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        const DxArgs d{{a.mat[0], a.mat[1]}, a.O, Op, a.I, G, a.T, a.nmat * Op, A, p.dx_splits,
                       cdiv(a.T, 128 * p.dx_mt), cdiv(a.I, kTileN), a.dX,
                       reinterpret_cast<float*>(w + p.dxpart_off)};
        if (a.bf16)
            e = p.dx_mt == 1 ? run_dx<false, 1>(d, s) : p.dx_mt == 2 ? run_dx<false, 2>(d, s)
                                                                     : run_dx<false, 4>(d, s);
        else
            e = p.dx_mt == 1 ? run_dx<true, 1>(d, s) : run_dx<true, 2>(d, s);
        if (e != hipSuccess) return e;
        if (p.dx_splits > 1) {
            e = sum_parts(d.part, a.T * a.I, p.dx_splits, a.T * a.I, 0, a.bf16, a.dX, s);
            if (e != hipSuccess) return e;
        }
    }
    if (want_ds) {
        const uint16_t* X = static_cast<const uint16_t*>(a.X);
        if (p.planes) {
            uint16_t* planes = reinterpret_cast<uint16_t*>(w + p.planes_off);
            e = launch_x_planes(a.X, a.bf16, a.T, a.I, planes, s);
            if (e != hipSuccess) return e;
            X = planes;
        }
        const DsArgs d{{a.mat[0], a.mat[1]}, src, G, G * kGroup, X, p.ds_splits, a.accumulate,
                       p.ds_tb, cdiv(a.O, kTileN), {a.dscales[0], a.dscales[1]},
                       reinterpret_cast<float*>(w + p.dspart_off)};
        if (a.bf16)
            e = p.ds_mt == 1 ? run_ds<1, 1>(d, s) : p.ds_mt == 2 ? run_ds<1, 2>(d, s)
                                                                 : run_ds<1, 4>(d, s);
        else
            e = p.ds_mt == 1 ? run_ds<3, 1>(d, s) : run_ds<3, 2>(d, s);
        if (e != hipSuccess) return e;
        for (int m = 0; m < a.nmat && p.ds_tb > 1; ++m) {
            e = sum_parts(d.part + m * a.O * G, a.nmat * a.O * G, p.ds_tb, a.O * G, a.accumulate,
                          false, a.dscales[m], s);
            if (e != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

}  // namespace qt
