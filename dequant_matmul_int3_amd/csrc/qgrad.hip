// Backward passes through packed weights: the gradient of the input and of
// the group scales, of a linear layer (one matrix) or of the gated
// feed-forward block (two).
//   dX[t,i]  = sum_m sum_o dY_m[t,o] s_m[o,g(i)] v_m[o,i]
//   ds_m[o,g] = sum_t dY_m[t,o] sum_{j<64} v_m[o,64g+j] X[t,64g+j]
// For the block dY_0 = dH u act'(g) and dY_1 = dH act(g), from the
// pre-activations g, u that the forward pass kept in f32.
//
// Input gradient.  A matrix product with the weights' rows as its inner axis:
// a block of 8 waves owns 128 MT tokens x 128 inputs (MT 1 or 2: with 4 the
// registers have no room for the weights' loads four steps ahead, 1.65 against
// 1.50 ms) and walks the rows of both matrices 64 at a time.  dY is first
// written as one padded plane in operand blocks; the weights are unpacked once
// per block into LDS row by row and read back as matrix operands.
//   bf16: both operands are rounded to f16, whose eight times finer step keeps
//   the result within its own bf16 rounding (1.69e-3 off in norm, of which the
//   rounding alone makes 1.66e-3; operands in bf16 left it 1.7 times as far off).  Exact powers of two bring them into f16's range and are taken
//   back from the sums: every token's dY is scaled by its largest magnitude to
//   2^14 .. 2^15, the scales of both matrices by the largest of them to 2^11 ..
//   2^12.  Gradients within 2^28 of their token's largest and scales within 2^25
//   of the largest keep all 11 bits, smaller ones an absolute error of 2^-39 and
//   2^-36 of the largest.  The operands come out of LDS through the transposing
//   reads of gfx950, four rows of 16 columns at a time: a lane's eight inner
//   elements are rows 4h .. 4h+3 and 16+4h .. 16+4h+3 of a 32-row step, and the
//   dY plane is written in that order.
//   f32: both stay f32, on the f32 matrix instructions.
// 4096 tokens, 2 x 17408 rows of 5120: 1.92 ms, of which the plane takes 0.38
// and the tiles about 1.5 (1.62 under a kernel trace).
//
// Scale gradient.  The forward product once more, group by group: the exact
// codes times the inputs (three exact bf16 pieces of an f32 input) give each
// token's sum over the group in f32, which is multiplied by dY[t,o] in f32 and
// summed over the tokens.  dY is held in registers for the whole walk over the
// groups.  Nothing is rounded below f32, and the weights' gradient never
// exists.  Token blocks leave partial sums that a last launch adds in order.
// The same shape: 1.71 ms for both matrices (860 TFLOP/s; each 0.87 ms under a
// kernel trace), bound as the forward tile by the FMAs and the unpacking beside
// the matrix instructions.
#include <algorithm>

#include "lds_barrier.h"
#include "tune.h"
#include "unpack.h"
#include "wave_reduce.h"

namespace qt {
namespace {

constexpr int kThreads = kTileThreads;
constexpr int kNT = kTileN / 16;

typedef f32x4_t f32x4_u __attribute__((aligned(4)));
typedef u32x2_t u32x2_u __attribute__((aligned(2)));

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
// ----------------------------------------------------------- gradient plane
// Operand blocks [T16][K / 32][16 tokens][32], K = nmat Op, matrix m at inner
// elements m Op .., zero past O.  bf16 calls: f16 times the token's power of
// two, position 8h + e of a block is row 4h + (e & 3) + 16 (e >> 2); f32 calls:
// f32 in order.  A block writes TOK tokens, 256 threads each, whose rows lie next
// to each other in the blocks: four from 1024 tokens on (one token's 64 bytes
// leave lines half written: 0.39 against 0.45 ms for 4096 tokens of 2 x 17408,
// 82 against 115 us for 1024 tokens of 50257), else one, for the sake of more
// blocks (8 against 15 us for 200 tokens of 2 x 2048).  kMaxParts further
// blocks leave the largest magnitude of their part of the scales (bf16 calls).
constexpr int kMaxParts = 64;

// 2^(top - floor(log2 m)), and 1 for m = 0; the exponent is kept where the
// factor and its inverse are normal numbers.
__device__ __forceinline__ float range_factor(float m, int top) {
    const int e = (int)(__float_as_uint(m) >> 23) & 0xFF;
    const int x = m == 0.0f ? 0 : top - (e - 127);
    return __uint_as_float((uint32_t)(127 + std::min(std::max(x, -125), 125)) << 23);
}

// x of a factor 2^x
__device__ __forceinline__ int factor_exp(float f) { return (int)(__float_as_uint(f) >> 23) - 127; }

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
__device__ __forceinline__ uint32_t f16_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)a, (_Float16)b});
}

template <bool F32, int TOK>
__global__ __launch_bounds__(TOK * 256) void grad_plane_kernel(
    const GradSrc src, int64_t Op, void* __restrict__ P, float* __restrict__ factor,
    const float* __restrict__ s0, const float* __restrict__ s1, int64_t nscales,
    float* __restrict__ smax) {
    constexpr int kPlaneThreads = TOK * 256, kPlaneTok = TOK;
    __shared__ float wm[kPlaneThreads / 64][kPlaneTok];
    const int tid = threadIdx.x;
    const int64_t tblocks = (src.T + kPlaneTok - 1) / kPlaneTok;
    if (!F32 && blockIdx.x >= tblocks) {
        const int part = (int)(blockIdx.x - tblocks);
        float m = 0.0f;
        for (int64_t i = (int64_t)part * kPlaneThreads + tid; i < nscales;
             i += kMaxParts * kPlaneThreads)
            m = fmaxf(m, fmaxf(fabsf(s0[i]), s1 ? fabsf(s1[i]) : 0.0f));
        m = wave_max(m);
        if ((tid & 63) == 0) wm[tid >> 6][0] = m;
        __syncthreads();
        if (tid == 0) {
#pragma unroll
            for (int w = 1; w < kPlaneThreads / 64; ++w) m = fmaxf(m, wm[w][0]);
            smax[part] = m;
        }
        return;
    }
    // four threads take a token's 32 inner elements, the next four the next
    // token's; tokens past T read a valid one and write nothing
    const int tk = (tid >> 2) % kPlaneTok;
    const int64_t c0 = tid / (4 * kPlaneTok) * 4 + (tid & 3);
    constexpr int kStep = kPlaneThreads / kPlaneTok;
    const int64_t tw = (int64_t)blockIdx.x * kPlaneTok + tk;
    const bool live = tw < src.T;
    const int64_t t = live ? tw : src.T - 1;
    const int64_t per = Op / 8;
    // what the eight gradients of chunk c are formed from, zero past O
    auto fetch = [&](int64_t c, float (&d)[8], float (&g)[8], float (&u)[8]) {
        const int64_t p0 = c * 8;
        const int64_t o0 = F32 ? p0 : (p0 & ~31LL) + ((p0 & 31) >> 1);
        auto get4 = [&](int k, int64_t o) {  // elements k .. k+3 from row o
            const int64_t at = t * src.O + o;
            if (o + 4 <= src.O) {
                if (src.dy_bf16) {
                    const u32x2_t w = *reinterpret_cast<const u32x2_u*>(
                        static_cast<const uint16_t*>(src.dY) + at);
                    d[k] = __uint_as_float(w.x << 16);
                    d[k + 1] = __uint_as_float(w.x & 0xFFFF0000u);
                    d[k + 2] = __uint_as_float(w.y << 16);
                    d[k + 3] = __uint_as_float(w.y & 0xFFFF0000u);
                } else {
                    const f32x4_t w =
                        *reinterpret_cast<const f32x4_u*>(static_cast<const float*>(src.dY) + at);
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[k + e] = w[e];
                }
                if (src.nmat == 2) {
                    const f32x4_t a = *reinterpret_cast<const f32x4_u*>(src.pre + at);
                    const f32x4_t b =
                        *reinterpret_cast<const f32x4_u*>(src.pre + src.T * src.O + at);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        g[k + e] = a[e];
                        u[k + e] = b[e];
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool in = o + e < src.O;
                    d[k + e] = in ? load_dy(src, at + e) : 0.0f;
                    g[k + e] = in && src.nmat == 2 ? src.pre[at + e] : 0.0f;
                    u[k + e] = in && src.nmat == 2 ? src.pre[src.T * src.O + at + e] : 0.0f;
                }
            }
        };
        get4(0, o0);
        get4(4, o0 + (F32 ? 4 : 16));
    };
    // the gradients themselves, one matrix's after the other's
    auto form = [&](const float (&d)[8], const float (&g)[8], const float (&u)[8],
                    float (&v)[2][8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (src.nmat == 1) {
                v[0][e] = d[e];
                v[1][e] = 0.0f;
            } else {
                act_grads(g[e], u[e], d[e], src.act, v[0][e], v[1][e]);
            }
        }
    };
    // The factor comes from the largest gradient, not from a bound of it (such
    // as |dH| (|g| + 0.3)): behind a closed gate (g = -30, say) the gradients
    // are 2^-40 of that bound and would all become 0.
    float f = 1.0f;
    if constexpr (!F32) {
        float m = 0.0f;
        for (int64_t c = c0; c < per; c += kStep) {
            float d[8], g[8], u[8], v[2][8];
            fetch(c, d, g, u);
            form(d, g, u, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) m = fmaxf(m, fmaxf(fabsf(v[0][e]), fabsf(v[1][e])));
        }
        // over the lanes of the token, then the waves
#pragma unroll
        for (int d = 32; d > 0; d >>= 1)
            if (d < 4 || d >= 4 * kPlaneTok) m = fmaxf(m, __shfl_xor(m, d));
        if ((tid & 63) < 4 * kPlaneTok && (tid & 3) == 0) wm[tid >> 6][tk] = m;
        __syncthreads();
        m = wm[0][tk];
#pragma unroll
        for (int w = 1; w < kPlaneThreads / 64; ++w) m = fmaxf(m, wm[w][tk]);
        f = range_factor(m, 14);
        if (tid < 4 * kPlaneTok && (tid & 3) == 0 && live) factor[t] = f;
    }
    const int64_t row = (t >> 4) * (src.nmat * Op) * 16 + (t & 15) * 32;  // block 0, this token
    for (int64_t c = c0; c < per; c += kStep) {
        float d[8], g[8], u[8], v[2][8];
        fetch(c, d, g, u);
        form(d, g, u, v);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            if (m >= src.nmat || !live) break;
            const int64_t at = row + ((m * Op + c * 8) >> 5) * 512 + (c & 3) * 8;
            if constexpr (F32) {
                f32x4_t* d = reinterpret_cast<f32x4_t*>(static_cast<float*>(P) + at);
                d[0] = f32x4_t{v[m][0], v[m][1], v[m][2], v[m][3]};
                d[1] = f32x4_t{v[m][4], v[m][5], v[m][6], v[m][7]};
            } else {
                *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(P) + at) = u32x4_t{
                    f16_pair(v[m][0] * f, v[m][1] * f), f16_pair(v[m][2] * f, v[m][3] * f),
                    f16_pair(v[m][4] * f, v[m][5] * f), f16_pair(v[m][6] * f, v[m][7] * f)};
            }
        }
    }
}

// ------------------------------------------------------------ input gradient
struct DxArgs {
    QMat mat[2];
    int64_t O, Op, I, G, T, K;  // K = nmat Op
    const void* A;              // gradient plane
    const float* factor;        // [T] powers of two of the plane's tokens (bf16)
    const float* smax;          // [kMaxParts] largest scales (bf16)
    int splits;
    int64_t mblk, nblk;
    void* dX;
    float* part;                // [splits][T][I], splits > 1
};

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

template <bool F32, int MT>
__global__ __launch_bounds__(kThreads) void dx_tile_kernel(const DxArgs a) {
    // LDS rows of 128 columns; 16-bit: 288 bytes, so that four rows of 16
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
    const int steps = (int)(a.K / kTileK), half = (int)(a.Op / kTileK);  // multiples of 4
    const int k0 = (int)((int64_t)(steps / 4) * sp / a.splits) * 4;
    const int k1 = (int)((int64_t)(steps / 4) * (sp + 1) / a.splits) * 4;

    float sf = 1.0f;  // the scales' power of two
    if constexpr (!F32) sf = range_factor(wave_max(a.smax[lane]), 11);

    // ---- weights: wave w unpacks rows 8w .. 8w+7 of a step, a lane one
    // quarter of one row; groups past G read a valid group (not stored), rows
    // past O a valid row (their dY is zero)
    const int q8 = lane & 7, q = q8 & 3;
    const uint32_t grp = (uint32_t)std::min<int64_t>(n * 2 + (q8 >> 2), a.G - 1);
    const int rl = 8 * wave + (lane >> 3);
    struct Raw {
        Quarter w;
        float s;
    };
    auto load_raw = [&](int k, Raw& r) {
        k = std::min(k, steps - 1);
        const int m = k >= half;  // uniform
        const QMat& mat = a.mat[m];
        const int64_t r0 = (int64_t)(k - m * half) * kTileK;
        // the step's first row is uniform, the lane's row in it at most 63
        // further: 32-bit offsets
        const uint32_t row = (uint32_t)std::min<int64_t>(rl, std::max<int64_t>(a.O - 1 - r0, 0));
        const int64_t base = std::min<int64_t>(r0, a.O - 1) * a.G;
        const uint32_t at = row * (uint32_t)a.G + grp;
        if (mat.bits == 3) {
            const uint8_t* p = mat.packed + base * kGroupBytes;
            r.w.a = *reinterpret_cast<const uint32_t*>(p + (at * (uint32_t)kGroupBytes + 4 * q));
            r.w.b = *reinterpret_cast<const uint32_t*>(
                p + (at * (uint32_t)kGroupBytes + 16 + 4 * (q >> 1)));
        } else {
            const u32x2_t w = *reinterpret_cast<const u32x2_t*>(
                mat.packed + base * kGroupBytesI4 + (at * (uint32_t)kGroupBytesI4 + 8 * q));
            r.w.a = w.x;
            r.w.b = w.y;
        }
        r.s = (mat.scales + base)[at];
    };
    auto unpack = [&](int buf, int k, const Raw& r) {
        const int bits = a.mat[std::min(k, steps - 1) >= half].bits;
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
            scaled_quarter_f16(r.w, q, bits, r.s * sf, lo8, hi8);
            reinterpret_cast<u32x4_t*>(d)[0] = lo8;
            reinterpret_cast<u32x4_t*>(d)[1] = hi8;
        }
    };

    // ---- dY: eight inner elements of the lane's tokens; token tiles past T
    // read a valid one
    constexpr int ESZ = F32 ? 4 : 2;
    const char* ap[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        ap[mt] = static_cast<const char*>(a.A) +
                 (std::min<int64_t>(m0 / 16 + wave * MT + mt, (a.T - 1) / 16) * a.K * 16 +
                  l16 * 32 + h4 * 8) *
                     ESZ;
    struct In {
        u32x4_t v[MT][2][F32 ? 2 : 1];
    };
    auto load_a = [&](int k, In& x) {
        k = std::min(k, steps - 1);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int p = 0; p < (F32 ? 2 : 1); ++p)
                    x.v[mt][ks][p] = *reinterpret_cast<const u32x4_t*>(
                        ap[mt] + (int64_t)(2 * k + ks) * (512 * ESZ) + 16 * p);
    };

    f32x4_t acc[MT][kNT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) acc[mt][nt] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // One step: products of x and LDS buffer buf, and the unpacking of the next
    // step's weights into the other.  Weights first: register r of lane l is
    // input 4 (l / 16) + r, token l % 16.
    auto step = [&](int buf, const In& x, int knext, const Raw& ru) {
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
            unpack(1 - buf, knext, ru);
        } else {
            const uint8_t* b0 = &ws[buf][(4 * h4 + (l16 >> 2)) * kRow + 8 * (l16 & 3)];
            f16x8_t b[2][2];
            auto read_b = [&](int nt) {
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    struct {
                        s16x4_t lo, hi;
                    } w;
                    const uint8_t* at = b0 + 32 * ks * kRow + nt * 32;
                    w.lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
                    w.hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 16 * kRow));
                    b[nt & 1][ks] = __builtin_bit_cast(f16x8_t, w);
                }
            };
            read_b(0);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
                if (nt + 1 < kNT) read_b(nt + 1);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks)
                        acc[mt][nt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                            b[nt & 1][ks], __builtin_bit_cast(f16x8_t, x.v[mt][ks][0]), acc[mt][nt],
                            0, 0, 0);
                if (nt == kNT / 2) unpack(1 - buf, knext, ru);
            }
#pragma unroll
            for (int i = 0; i < 2 * kNT * MT; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                __builtin_amdgcn_sched_group_barrier(0x2, 2, 0);
            }
        }
    };

    // weights four steps ahead in registers (every step reads new rows: two
    // steps ahead left a quarter of the time waiting for them), dY one; past
    // the last step of the plane the loads repeat it
    In x0, x1;
    Raw raw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) load_raw(k0 + j, raw[j]);
    load_a(k0, x0);
    unpack(0, k0, raw[0]);
    lds_barrier();
    auto body = [&](int k, int j, const In& xc, In& xn) {
        load_a(k + 1, xn);
        load_raw(k + 4, raw[j]);
        step(j & 1, xc, k + 1, raw[(j + 1) & 3]);
        lds_barrier();
    };
    for (int k = k0; k < k1; k += 4) {
        body(k, 0, x0, x1);
        body(k + 1, 1, x1, x0);
        body(k + 2, 2, x0, x1);
        body(k + 3, 3, x1, x0);
    }

#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int64_t t = m0 + wave * (16 * MT) + mt * 16 + l16;
        if (t >= a.T) continue;
        // takes both powers of two back; one exponent, since their product may
        // be no f32 number where the result is one
        int un = 0;
        if constexpr (!F32) un = -factor_exp(a.factor[t]) - factor_exp(sf);
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt) {
            const int64_t i = n * kTileN + nt * 16 + 4 * h4;
            const int64_t left = a.I - i, o = t * a.I + i;
            if (left <= 0) continue;
            f32x4_t v = acc[mt][nt];
            if constexpr (!F32) {
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = __builtin_ldexpf(v[r], un);
            }
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
    int64_t G;
    const uint16_t* X;   // blocked planes [NP][T16][2 G] of 1 KB
    int splits, accumulate;
    int64_t tblk, oblk;  // token blocks, row blocks of one matrix
    float* out[2];       // dscales [O x G] of each matrix (one token block), or
    float* part;         // [tblk][nmat][O][G]
};

// M: the matrix; NP pieces per input, MT 16-token tiles per wave, NT weight
// tiles per block
template <int BITS, int NP, int MT, int NT>
__global__ __launch_bounds__(kThreads) void ds_tile_kernel(const DsArgs a, const int m) {
    constexpr int kRows = 16 * NT;
    __shared__ __attribute__((aligned(16))) u32x4_t ws[2][8 * 2 * 64];  // as ffn.hip
    __shared__ float red[2][4][8][kRows];  // [turn][group][wave][row]
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h4 = lane >> 4, l16 = lane & 15;
    const int64_t T = a.src.T, O = a.src.O;
    // row blocks run fastest: their token block's inputs are shared in the
    // XCD's L2
    int64_t tile = xcd_range(blockIdx.x, gridDim.x);
    const int64_t ob = tile % a.oblk;
    tile /= a.oblk;
    const int64_t tb = tile % a.tblk;
    const int sp = (int)(tile / a.tblk);
    const int64_t o0 = ob * kRows, t0 = tb * (128 * MT) + wave * (16 * MT);
    const int G = (int)a.G;
    const int g0 = split_begin(G, sp, a.splits), g1 = split_begin(G, sp + 1, a.splits);

    RowFeed<BITS, BITS> feed;
    feed.init(a.mat[m], a.mat[m], false, std::min<int64_t>(o0 + wave * 16 + l16, O - 1), G, h4);
    feed.load(g0);
    auto unpack = [&](int buf, int j) {
        u32x4_t lo8, hi8;
        feed.exact(j, h4, lo8, hi8);
        u32x4_t* d = &ws[buf][(2 * wave + (h4 >> 1)) * 64 + 32 * (h4 & 1) + l16];
        d[0] = lo8;
        d[16] = hi8;
    };
    const int64_t t16 = (T + 15) / 16, plane = t16 * 2 * G * 512;
    const uint16_t* xp[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
        xp[mt] = a.X + std::min<int64_t>(t0 / 16 + mt, t16 - 1) * (2 * G * 512) + 8 * lane;
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
                        xp[mt] + p * plane + (int64_t)(2 * g + ks) * 512);
    };

    // dY of the tile, where the products will lie: register r of lane l is
    // token 4 (l / 16) + r, row l % 16; zero past T and O.  Loads without
    // branches (past the ends a valid element), a token tile's all in flight.
    f32x4_t dy[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        auto each = [&](auto load) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int64_t t = t0 + mt * 16 + 4 * h4 + r, o = o0 + nt * 16 + l16;
                    load(nt, r, std::min(t, T - 1) * O + std::min(o, O - 1), t < T && o < O);
                }
        };
        float d[NT][4];
        if (a.src.dy_bf16)
            each([&](int nt, int r, int64_t at, bool) {
                d[nt][r] = __uint_as_float(
                    (uint32_t) static_cast<const uint16_t*>(a.src.dY)[at] << 16);
            });
        else
            each([&](int nt, int r, int64_t at, bool) {
                d[nt][r] = static_cast<const float*>(a.src.dY)[at];
            });
        if (a.src.nmat == 2) {
            float g[NT][4], u[NT][4];
            each([&](int nt, int r, int64_t at, bool) {
                g[nt][r] = a.src.pre[at];
                u[nt][r] = a.src.pre[T * O + at];
            });
            each([&](int nt, int r, int64_t, bool) {
                float dg, du;
                act_grads(g[nt][r], u[nt][r], d[nt][r], a.src.act, dg, du);
                d[nt][r] = m == 0 ? dg : du;
            });
        }
        each([&](int nt, int r, int64_t, bool in) {
            dy[mt][nt][r] = in ? d[nt][r] * code_unit(BITS) : 0.0f;
        });
    }

    // the tile's sums of one group, per wave over its tokens, and the
    // unpacking of word j of the feed (ordered as in the forward tile)
    auto step = [&](int buf, const In& x, int j, float (&rd)[8][kRows]) {
        float v[NT];
        bf16x8_t b[2][2];
        f32x4_t part[3];
        auto read_b = [&](int nt) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
                b[nt & 1][ks] = __builtin_bit_cast(bf16x8_t, ws[buf][(2 * nt + ks) * 64 + lane]);
        };
        read_b(0);
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
                    v[pn] = pm == 0 && r == 0
                                ? part[(q - 2) % 3][r] * dy[pm][pn][r]
                                : __builtin_fmaf(part[(q - 2) % 3][r], dy[pm][pn][r], v[pn]);
            }
            if (q == NT * MT / 2) unpack(1 - buf, j);
        }
#pragma unroll
        for (int i = 0; i < 2 * NP * NT * MT; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x2, 2, 0);
        }
        // sums over the four lane rows, two values at a time: their halves are
        // swapped and added, then the quarters of two such sums; lane row h
        // ends with value 2 (h & 1) + (h >> 1) of each four (of each two, both
        // lane rows of a half with the same)
        auto half = [&](float p, float q) {
            const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(p), __float_as_uint(q),
                                                            false, false);
            return __uint_as_float(s[0]) + __uint_as_float(s[1]);
        };
        auto quarter = [&](float p, float q) {
            const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(p), __float_as_uint(q),
                                                            false, false);
            return __uint_as_float(s[0]) + __uint_as_float(s[1]);
        };
#pragma unroll
        for (int f = 0; f + 4 <= NT; f += 4)
            rd[wave][(f + 2 * (h4 & 1) + (h4 >> 1)) * 16 + l16] =
                quarter(half(v[f], v[f + 1]), half(v[f + 2], v[f + 3]));
        if constexpr (NT % 4 == 2) {
            const float w = half(v[NT - 2], v[NT - 1]);
            const float z = quarter(w, w);
            if (!(h4 & 1)) rd[wave][(NT - 2 + (h4 >> 1)) * 16 + l16] = z;
        }
        if constexpr (NT % 4 == 1) {
            const float w = half(v[NT - 1], v[NT - 1]);
            const float z = quarter(w, w);
            if (h4 == 0) rd[wave][(NT - 1) * 16 + l16] = z;
        }
    };
    // four groups' sums over the waves, in wave order, once per turn: thread
    // (row, group)
    const int frow = tid >> 2, fj = tid & 3;
    auto finish = [&](const float (&rd)[4][8][kRows], int g) {
        if (frow < kRows && o0 + frow < O && g + fj < g1) {
            float s = rd[fj][0][frow];
#pragma unroll
            for (int w = 1; w < 8; ++w) s += rd[fj][w][frow];
            const int64_t at = (o0 + frow) * a.G + g + fj;
            if (a.tblk > 1) {
                a.part[(tb * a.src.nmat + m) * O * a.G + at] = s;
            } else {
                float* d = a.out[m] + at;
                *d = a.accumulate ? *d + s : s;
            }
        }
    };

    // the pipeline of the forward tile (ffn.hip)
    In x0, x1;
    load_x(g0, x0);
    feed.take();
    feed.load(g0 + 4);
    unpack(0, 0);
    lds_barrier();
    auto group = [&](int g, int j, const In& xc, In& xn, int turn) {
        load_x(std::min(g + 1, G - 1), xn);
        if (j == 3) {
            feed.take();
            feed.load(g + 5);
        }
        step(j & 1, xc, (j + 1) & 3, red[turn][j]);
        lds_barrier();
    };
    int turn = 0;
    for (int g = g0; g < g1; g += 4) {
        group(g, 0, x0, x1, turn);
        group(g + 1, 1, x1, x0, turn);
        group(g + 2, 2, x0, x1, turn);
        group(g + 3, 3, x1, x0, turn);
        finish(red[turn], g);
        turn ^= 1;  // the next turn writes the other half while this one is summed
    }
}

template <bool F32, int MT>
hipError_t run_dx(const DxArgs& a, hipStream_t s) {
    const int64_t nb = a.mblk * a.nblk * a.splits;
    hipLaunchKernelGGL((dx_tile_kernel<F32, MT>), dim3((unsigned)nb), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}
// one launch per matrix: their bits may differ
template <int NP, int MT, int NT>
hipError_t run_ds(const DsArgs& a, hipStream_t s) {
    const int64_t nb = a.oblk * a.tblk * a.splits;
    for (int m = 0; m < a.src.nmat; ++m) {
        if (a.mat[m].bits == 3)
            hipLaunchKernelGGL((ds_tile_kernel<3, NP, MT, NT>), dim3((unsigned)nb),
                               dim3(kThreads), 0, s, a, m);
        else
            hipLaunchKernelGGL((ds_tile_kernel<4, NP, MT, NT>), dim3((unsigned)nb),
                               dim3(kThreads), 0, s, a, m);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}
hipError_t sum_parts(const float* part, int64_t stride, int splits, int64_t n, int accumulate,
                     bool bf16, void* out, hipStream_t s) {
    const int64_t nb = cdiv(n, 1024);
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
    if (!bwd_fits(p, a.T, a.I, a.O, want_dx, want_ds)) return hipErrorInvalidValue;
    char* w = static_cast<char*>(workspace);
    const int64_t G = cdiv(a.I, kGroup), Op = pad_to(a.O, 4 * kTileK);
    const GradSrc src{a.nmat, a.act, a.dy_bf16, a.dY, a.pre, a.T, a.O};
    hipError_t e;
    if (want_dx) {
        void* A = w + p.grad_off;
        float* factor = reinterpret_cast<float*>(w + p.factor_off);
        float* smax = factor + a.T;
        const float* s1 = a.nmat == 2 ? a.mat[1].scales : nullptr;
        const int64_t maxparts = a.bf16 ? kMaxParts : 0;
#define QT_PLANE(F, N)                                                                       \
    hipLaunchKernelGGL((grad_plane_kernel<F, N>),                                            \
                       dim3((unsigned)(cdiv(a.T, N) + maxparts)), dim3(N * 256), 0, s, src, Op, \
                       A, factor, a.mat[0].scales, s1, a.O * G, smax)
        if (a.bf16) {
            if (a.T >= 1024) QT_PLANE(false, 4);
            else QT_PLANE(false, 1);
        } else {
            if (a.T >= 1024) QT_PLANE(true, 4);
            else QT_PLANE(true, 1);
        }
#undef QT_PLANE
        e = hipGetLastError();
        if (e != hipSuccess) return e;
        const DxArgs d{{a.mat[0], a.mat[1]}, a.O, Op, a.I, G, a.T, a.nmat * Op, A, factor, smax,
                       p.dx_splits, cdiv(a.T, 128 * p.dx_mt), cdiv(a.I, kTileN), a.dX,
                       reinterpret_cast<float*>(w + p.dxpart_off)};
        if (a.bf16)
            e = p.dx_mt == 1 ? run_dx<false, 1>(d, s) : run_dx<false, 2>(d, s);
        else
            e = p.dx_mt == 1 ? run_dx<true, 1>(d, s) : run_dx<true, 2>(d, s);
        if (e != hipSuccess) return e;
        if (p.dx_splits > 1) {
            e = sum_parts(d.part, a.T * a.I, p.dx_splits, a.T * a.I, 0, a.bf16, a.dX, s);
            if (e != hipSuccess) return e;
        }
    }
    if (want_ds) {
        uint16_t* X = reinterpret_cast<uint16_t*>(w + p.planes_off);
        e = launch_x_planes(a.X, a.bf16, true, a.T, a.I, X, s);
        if (e != hipSuccess) return e;
        const DsArgs d{{a.mat[0], a.mat[1]}, src, G, X, p.ds_splits, a.accumulate, p.ds_tb,
                       cdiv(a.O, 16 * p.ds_nt), {a.dscales[0], a.dscales[1]},
                       reinterpret_cast<float*>(w + p.dspart_off)};
        if (a.bf16)
            e = p.ds_mt == 1   ? run_ds<1, 1, 8>(d, s)
                : p.ds_mt == 2 ? run_ds<1, 2, 8>(d, s)
                : p.ds_nt == 5 ? run_ds<1, 4, 5>(d, s)
                               : run_ds<1, 4, 6>(d, s);
        else
            e = p.ds_mt == 1 ? run_ds<3, 1, 8>(d, s) : run_ds<3, 2, 8>(d, s);
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
