// Distillation from a teacher's top-k logits, forward and backward.
//
// Row t of the student's logits z [V], the teacher's entries (idx_j, tl_j),
// j < k, of which those with idx_j in [0, V) count, and a temperature tau:
//   p = softmax over the row's entries of tl_j / tau
//   lse = ln sum_v exp(z_v / tau),  q_v = exp(z_v / tau - lse)
//   loss = tau^2 sum_j p_j (ln p_j - z_{idx_j} / tau + lse)
//        = tau (sum_j p_j (tau ln p_j + r - z_{idx_j}) + (m - r) + tau ln S)
//     with m = max_v z_v, S = sum_v exp((z_v - m) / tau) and any r
//   dz_v = gloss tau (q_v - sum_{j: idx_j = v} p_j)
// A row without entries (or with every entry at -inf) has zero loss and zero
// gradient, whatever its logits hold.
//
// What bounds it: the logits' bytes, read once and (with the gradient)
// written once.  Every value costs about six vector instructions and one
// exp2 per pass, well under the memory time.  2048 rows of 131072 bf16 with
// the gradient: 0.265 ms, 4.0 TB/s of the 5.2 that a copy reaches.
//
// Two forms.
//   * Row form: a block holds a whole row in registers (16-byte vectors, as
//     loaded), so the row is read once for the maximum, the sum and the
//     gradient.  One launch, no workspace.
//   * Split form, for few rows (one block per row would leave most CUs idle)
//     and for rows past the registers: S blocks per row leave the maximum
//     and sum of their chunk in the workspace; a second launch joins the S
//     pairs and writes the gradient, reading its chunk again.
// Sums, maxima and the teacher's softmax are f32.  Exponents are formed from
// differences to the row's maximum (the teacher's, too), and the loss from
// differences to r, the student's largest logit among the teacher's entries,
// so that no term but the entropy's is negative: their rounding does not know
// the level that all of a row's logits share.  (With z / tau and lse in place of
// the differences the loss at tau = 1.5 was 8e-5 off at a level of 300 and 9e-4
// at 3000; it is 1e-6 to 4e-6 off at each.)  The backward call has only lse,
// whose own half step, 2^-24 |lse| at most, enters every probability.  The
// gradient is rounded once, to the logits' type; entries at the teacher's
// indices are formed from their own z and written after the rest of the row.
#include <algorithm>

#include "tune.h"
#include "wave_reduce.h"

namespace qt {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
// the same 16 bytes at the elements' own alignment (the rows of an odd
// vocabulary): gfx950 loads and stores them with the same instructions
typedef u32x4_t u32x4_u __attribute__((aligned(2)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kMaxK = kDistillMaxK;

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// 16 bytes of a row: 8 bf16 or 4 f32 values
template <bool BF16>
struct Vec {
    static constexpr int E = BF16 ? 8 : 4;
    static constexpr int kBytes = BF16 ? 2 : 4;
    static __device__ __forceinline__ float get(const u32x4_t& v, int e) {
        if constexpr (BF16)
            return __uint_as_float((e & 1) ? (v[e >> 1] & 0xFFFF0000u) : (v[e >> 1] << 16));
        else
            return __uint_as_float(v[e]);
    }
    static __device__ __forceinline__ float load1(const void* p, int64_t i) {
        if constexpr (BF16)
            return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << 16);
        else
            return reinterpret_cast<const float*>(p)[i];
    }
    static __device__ __forceinline__ void store1(void* p, int64_t i, float f) {
        if constexpr (BF16)
            reinterpret_cast<__bf16*>(p)[i] = (__bf16)f;
        else
            reinterpret_cast<float*>(p)[i] = f;
    }
    // vector i of a row of V values; values past the row read as -inf
    static __device__ __forceinline__ u32x4_t load(const void* row, int64_t i, int64_t V) {
        const int64_t e0 = i * E;
        u32x4_t v;
        if (e0 + E <= V) {
            v = *reinterpret_cast<const u32x4_u*>(reinterpret_cast<const char*>(row) + e0 * kBytes);
        } else {
            const uint32_t pad = BF16 ? 0xFF80FF80u : 0xFF800000u;
            v = u32x4_t{pad, pad, pad, pad};
            if constexpr (BF16) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (e0 + e < V) {
                        const uint32_t b = reinterpret_cast<const uint16_t*>(row)[e0 + e];
                        v[e >> 1] = (e & 1) ? (v[e >> 1] & 0xFFFFu) | (b << 16)
                                            : (v[e >> 1] & 0xFFFF0000u) | b;
                    }
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    if (e0 + e < V) v[e] = reinterpret_cast<const uint32_t*>(row)[e0 + e];
            }
        }
        return v;
    }
    static __device__ __forceinline__ void store(void* row, int64_t i, int64_t V,
                                                 const float (&f)[E]) {
        const int64_t e0 = i * E;
        if (e0 + E <= V) {
            u32x4_t v;
            if constexpr (BF16) {
                typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    v[e >> 1] = __builtin_bit_cast(uint32_t, bf2{(__bf16)f[e], (__bf16)f[e + 1]});
            } else {
#pragma unroll
                for (int e = 0; e < E; ++e) v[e] = __float_as_uint(f[e]);
            }
            *reinterpret_cast<u32x4_u*>(reinterpret_cast<char*>(row) + e0 * kBytes) = v;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (e0 + e < V) store1(row, e0 + e, f[e]);
        }
    }
};

// fmaxf drops a NaN; the sum over the row brings it back, since
// exp2(NaN - m) is NaN.  m = -inf (nothing but -inf seen so far) is replaced
// by 0 where differences to it are formed, so that those exponentials are 0;
// a row that holds nothing but -inf ends with the sum 0 and lse = -inf.
__device__ __forceinline__ float finite_max(float m) { return m == neg_inf() ? 0.0f : m; }

// (m, s) of sum exp2((z - m) c) joined with another pair.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2, float c) {
    const float M = fmaxf(m, m2), f = finite_max(M);
    s = s * exp2_((m - f) * c) + s2 * exp2_((m2 - f) * c);
    m = M;
}

// The teacher's entries of a row: p_j and idx_j (-1 where the entry does not
// count) in LDS, and z_j, the student's logits there, where `student` reads
// them; the result says whether any entry counts.  One wave, every lane calls.
struct Teacher {
    float p[kMaxK];
    float z[kMaxK];
    int32_t idx[kMaxK];
};
template <typename Z, typename F>
__device__ __forceinline__ bool teacher_softmax(Teacher& th, const int32_t* __restrict__ idx,
                                                const float* __restrict__ tl, int k, int64_t V,
                                                float itau, int lane, Z student, F term) {
    float m = neg_inf(), bad = 0.0f;
    for (int j = lane; j < k; j += 64) {
        const int32_t id = idx[j];
        const bool ok = id >= 0 && id < V;
        const float x = ok ? tl[j] : neg_inf();
        th.idx[j] = ok ? id : -1;
        th.p[j] = x;
        student(j, ok ? id : -1);
        m = fmaxf(m, x);
        bad += x != x ? 1.0f : 0.0f;
    }
    m = wave_max(m);
    // nothing but NaN or -inf: no mass unless a NaN asks to be seen
    const bool mass = m > neg_inf() || wave_sum(bad) > 0.0f;
    const float f = finite_max(m);
    float s = 0.0f;
    for (int j = lane; j < k; j += 64) s += expf((th.p[j] - f) * itau);
    s = wave_sum(s);
    const float ls = logf(s), is = 1.0f / s;
    for (int j = lane; j < k; j += 64) {
        const float d = (th.p[j] - f) * itau;
        const float p = mass ? expf(d) * is : 0.0f;
        if (th.idx[j] >= 0 && p != 0.0f) term(j, p, d - ls);  // NaN included
        th.p[j] = p;
    }
    return mass;
}

// The teacher's side of the loss: a = sum_j p_j (tau ln p_j + r - z_j) over the
// entries with p_j > 0 and r, their largest finite z_j (0: none).
struct TeacherLoss {
    float a, r;
    bool mass;
};
template <bool BF16>
__device__ __forceinline__ TeacherLoss teacher_loss(Teacher& th, const int32_t* __restrict__ idx,
                                                    const float* __restrict__ tl, int k, int64_t V,
                                                    float tau, float itau, int lane,
                                                    const char* row) {
    float ent = 0.0f, r = neg_inf();
    TeacherLoss t;
    t.mass = teacher_softmax(
        th, idx, tl, k, V, itau, lane,
        [&](int j, int32_t id) { th.z[j] = id >= 0 ? Vec<BF16>::load1(row, id) : 0.0f; },
        [&](int j, float p, float lp) {
            ent += p * lp;
            r = fmaxf(r, th.z[j]);
        });
    t.r = finite_max(wave_max(r));
    float d = 0.0f;
    for (int j = lane; j < k; j += 64)
        if (th.p[j] != 0.0f) d += th.p[j] * (t.r - th.z[j]);
    t.a = wave_sum(tau * ent + d);
    return t;
}
// m, s: the row's maximum and sum.  A row with a NaN, a +inf or nothing but -inf
// gives NaN, mass on a logit of -inf gives +inf.
__device__ __forceinline__ float loss_value(float a, float r, float m, float s, float tau) {
    return tau * (a + (m - r) + tau * logf(s));
}

// ---------------------------------------------------------------- row form
template <bool BF16, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void distill_row_kernel(
    const void* logits, int64_t T, int64_t V, int64_t ld, const int32_t* __restrict__ idx,
    const float* __restrict__ tl, int k, float tau, float* __restrict__ loss,
    float* __restrict__ lse, const float* __restrict__ gloss, void* dlogits, int64_t ldd) {
    typedef Vec<BF16> X;
    constexpr int W = THREADS / 64;
    __shared__ Teacher th;
    __shared__ float wm[W], wsum[W];
    __shared__ int has;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    if (t >= T) return;
    const char* row = static_cast<const char*>(logits) + t * ld * X::kBytes;
    const float itau = 1.0f / tau, c = itau * kLog2e;

    u32x4_t v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = X::load(row, i * THREADS + tid, V);

    // the last wave also takes the teacher's entries and the student's
    // logits at them (before anything is written: dlogits may be logits)
    TeacherLoss tls{0.0f, 0.0f, false};
    if (wave == W - 1) {
        tls = teacher_loss<BF16>(th, idx + t * k, tl + t * k, k, V, tau, itau, lane, row);
        if (lane == 0) has = tls.mass;
    }

    // The row stays as loaded between the passes: without this the compiler
    // keeps its f32 values for the next pass and spills them (0.80 against
    // 0.27 ms for 2048 rows of 131072).
    auto keep_raw = [&]() {
#pragma unroll
        for (int i = 0; i < NV; ++i) asm volatile("" : "+v"(v[i]));
    };
    float m = neg_inf();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < X::E; ++e) m = fmaxf(m, X::get(v[i], e));
    m = wave_max(m);
    const float f = finite_max(m);
    float s = 0.0f;
    keep_raw();
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < X::E; ++e) s += exp2_((X::get(v[i], e) - f) * c);
    s = wave_sum(s);
    if (lane == 0) {
        wm[wave] = m;
        wsum[wave] = s;
    }
    __syncthreads();
    m = wm[0];
    s = wsum[0];
#pragma unroll
    for (int w = 1; w < W; ++w) join(m, s, wm[w], wsum[w], c);
    const bool mass = has != 0;
    if (tid == THREADS - 64) {  // first lane of the last wave
        lse[t] = m * itau + logf(s);
        loss[t] = mass ? loss_value(tls.a, tls.r, m, s, tau) : 0.0f;
    }
    if (!dlogits) return;

    const float g = (gloss ? gloss[t] : 1.0f) * tau;
    const float is = 1.0f / s, fm = finite_max(m);
    char* drow = static_cast<char*>(dlogits) + t * ldd * X::kBytes;
    keep_raw();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int64_t vi = i * THREADS + tid;
        if (vi * X::E < V) {
            float o[X::E];
#pragma unroll
            for (int e = 0; e < X::E; ++e) {
                const float q = exp2_((X::get(v[i], e) - fm) * c) * is;
                o[e] = mass ? q * g : 0.0f;
            }
            X::store(drow, vi, V, o);
        }
    }
    __syncthreads();
    // the teacher's indices, each written by the first entry that names it
    if (mass)
        for (int j = tid; j < k; j += THREADS) {
            const int32_t id = th.idx[j];
            if (id < 0) continue;
            float p = 0.0f;
            bool first = true;
            for (int i = 0; i < k; ++i)
                if (th.idx[i] == id) {
                    first = first && i >= j;
                    p += th.p[i];
                }
            if (first) X::store1(drow, id, (exp2_((th.z[j] - fm) * c) * is - p) * g);
        }
}

// -------------------------------------------------------------- split form
constexpr int kSplitThreads = 256;

struct SplitWs {
    float* part;  // [T][S][2]: maximum and sum of each chunk
    float* row;   // [T][3]: a and r of TeacherLoss, and whether there is mass
};

__device__ __host__ inline int64_t split_chunk(int64_t V, int S, int E) {
    const int64_t vecs = (V + E - 1) / E;
    return (vecs + S - 1) / S * E;  // values per chunk, whole vectors
}

template <bool BF16>
__global__ __launch_bounds__(kSplitThreads) void distill_stats_kernel(
    const void* __restrict__ logits, int64_t V, int64_t ld, const int32_t* __restrict__ idx,
    const float* __restrict__ tl, int k, float tau, int S, SplitWs ws) {
    typedef Vec<BF16> X;
    constexpr int W = kSplitThreads / 64;
    __shared__ Teacher th;
    __shared__ float wm[W], wsum[W];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t = blockIdx.x / S;
    const int sp = blockIdx.x % S;
    const char* row = static_cast<const char*>(logits) + t * ld * X::kBytes;
    const float itau = 1.0f / tau, c = itau * kLog2e;
    const int64_t chunk = split_chunk(V, S, X::E);
    const int64_t v0 = sp * chunk / X::E;
    const int64_t v1 = std::min<int64_t>(v0 + chunk / X::E, (V + X::E - 1) / X::E);

    if (sp == 0 && wave == W - 1) {
        const TeacherLoss tls =
            teacher_loss<BF16>(th, idx + t * k, tl + t * k, k, V, tau, itau, lane, row);
        if (lane == 0) {
            ws.row[3 * t] = tls.a;
            ws.row[3 * t + 1] = tls.r;
            ws.row[3 * t + 2] = tls.mass ? 1.0f : 0.0f;
        }
    }
    // four vectors at a time: their loads are in flight together
    float m = neg_inf(), s = 0.0f;
    for (int64_t i = v0 + tid; i < v1; i += 4 * kSplitThreads) {
        u32x4_t v[4];
        float bm = neg_inf();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t iq = i + q * kSplitThreads;
            const uint32_t pad = BF16 ? 0xFF80FF80u : 0xFF800000u;
            v[q] = iq < v1 ? X::load(row, iq, V) : u32x4_t{pad, pad, pad, pad};
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < X::E; ++e) bm = fmaxf(bm, X::get(v[q], e));
        const float f = finite_max(bm);
        float bs = 0.0f;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < X::E; ++e) bs += exp2_((X::get(v[q], e) - f) * c);
        join(m, s, bm, bs, c);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) join(m, s, __shfl_xor(m, d), __shfl_xor(s, d), c);
    if (lane == 0) {
        wm[wave] = m;
        wsum[wave] = s;
    }
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < W; ++w) join(m, s, wm[w], wsum[w], c);
        ws.part[2 * (t * S + sp)] = m;
        ws.part[2 * (t * S + sp) + 1] = s;
    }
}

// Second launch of the split form (FROM_LSE false: joins the chunks' pairs,
// writes loss and lse) and the backward pass (FROM_LSE true).  Blocks write
// the gradient of chunk sp of row t; without dlogits one block per row only
// joins.
template <bool BF16, bool FROM_LSE>
__global__ __launch_bounds__(kSplitThreads) void distill_grad_kernel(
    const void* logits, int64_t V, int64_t ld, const int32_t* __restrict__ idx,
    const float* __restrict__ tl, int k, float tau, int S, int nblk, SplitWs ws,
    float* __restrict__ loss, float* __restrict__ lse, const float* __restrict__ gloss,
    void* dlogits, int64_t ldd) {
    typedef Vec<BF16> X;
    __shared__ Teacher th;
    __shared__ int has;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t = blockIdx.x / nblk;
    const int sp = blockIdx.x % nblk;
    const float itau = 1.0f / tau;
    const char* row = static_cast<const char*>(logits) + t * ld * X::kBytes;
    // q_v = exp2((z_v - off) c - l2): off = the row's maximum and l2 = log2 of
    // the sum where the pairs are joined; off = 0 and l2 = lse log2(e) where
    // lse is given
    float fm = 0.0f, is = 1.0f, l = 0.0f;
    const float c = itau * kLog2e;
    if constexpr (!FROM_LSE) {
        float m = ws.part[2 * t * S], s = ws.part[2 * t * S + 1];
        for (int q = 1; q < S; ++q)
            join(m, s, ws.part[2 * (t * S + q)], ws.part[2 * (t * S + q) + 1], c);
        fm = finite_max(m);
        is = 1.0f / s;
        if (sp == 0 && tid == 0) {
            lse[t] = m * itau + logf(s);
            const float* r = ws.row + 3 * t;
            loss[t] = r[2] != 0.0f ? loss_value(r[0], r[1], m, s, tau) : 0.0f;
        }
    } else {
        l = lse[t];
    }
    if (!dlogits) return;
    auto prob = [&](float z) {
        if constexpr (FROM_LSE)
            return exp2_(__builtin_fmaf(z, itau, -l) * kLog2e);
        else
            return exp2_((z - fm) * c) * is;
    };
    if (wave == 0) {
        const bool mass = teacher_softmax(th, idx + t * k, tl + t * k, k, V, itau, lane,
                                          [](int, int32_t) {}, [](int, float, float) {});
        if (lane == 0) has = mass;
    }
    __syncthreads();
    const int64_t chunk = split_chunk(V, S, X::E);
    const int64_t v0 = sp * chunk / X::E;
    const int64_t v1 = std::min<int64_t>(v0 + chunk / X::E, (V + X::E - 1) / X::E);
    const int64_t e0 = v0 * X::E, e1 = std::min<int64_t>(v1 * X::E, V);
    const bool mass = has != 0;
    const float g = (gloss ? gloss[t] : 1.0f) * tau;
    for (int j = tid; j < k; j += kSplitThreads) {
        const int32_t id = th.idx[j];
        th.z[j] = id >= e0 && id < e1 ? X::load1(row, id) : 0.0f;
    }
    __syncthreads();  // the logits at the teacher's indices are read: dlogits may be logits
    char* drow = static_cast<char*>(dlogits) + t * ldd * X::kBytes;
    for (int64_t i = v0 + tid; i < v1; i += 4 * kSplitThreads) {
        u32x4_t v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t iq = i + q * kSplitThreads;
            if (iq < v1) v[q] = X::load(row, iq, V);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int64_t iq = i + q * kSplitThreads;
            if (iq < v1) {
                float o[X::E];
#pragma unroll
                for (int e = 0; e < X::E; ++e)
                    o[e] = mass ? prob(X::get(v[q], e)) * g : 0.0f;
                X::store(drow, iq, V, o);
            }
        }
    }
    __syncthreads();
    if (mass)
        for (int j = tid; j < k; j += kSplitThreads) {
            const int32_t id = th.idx[j];
            if (id < e0 || id >= e1) continue;
            float p = 0.0f;
            bool first = true;
            for (int i = 0; i < k; ++i)
                if (th.idx[i] == id) {
                    first = first && i >= j;
                    p += th.p[i];
                }
            if (first) X::store1(drow, id, (prob(th.z[j]) - p) * g);
        }
}

template <bool BF16, int THREADS, int NV>
void run_row(const DistillArgs& a, float* loss, float* lse, void* dlogits, int64_t ldd,
             hipStream_t s) {
    const GridRows g = grid_rows(a.T, THREADS);
    hipLaunchKernelGGL((distill_row_kernel<BF16, THREADS, NV>), dim3(g.x, g.y),
                       dim3(THREADS), 0, s, a.logits, a.T, a.V, a.ld, a.idx, a.tl, a.k, a.tau, loss,
                       lse, a.gloss, dlogits, ldd);
}

template <bool BF16>
hipError_t run_distill(const DistillArgs& a, float* loss, float* lse, void* dlogits, int64_t ldd,
                       void* workspace, hipStream_t s) {
    const int S = distill_splits(a.T, a.V, BF16);
    if (S == 0) {
        const int64_t vecs = (a.V + Vec<BF16>::E - 1) / Vec<BF16>::E;
        if (vecs <= 256 * 2) run_row<BF16, 256, 2>(a, loss, lse, dlogits, ldd, s);
        else if (vecs <= 256 * 8) run_row<BF16, 256, 8>(a, loss, lse, dlogits, ldd, s);
        else if (vecs <= 1024 * 4) run_row<BF16, 1024, 4>(a, loss, lse, dlogits, ldd, s);
        else if (vecs <= 1024 * 8) run_row<BF16, 1024, 8>(a, loss, lse, dlogits, ldd, s);
        else run_row<BF16, 1024, 16>(a, loss, lse, dlogits, ldd, s);
        return hipGetLastError();
    }
    SplitWs ws{static_cast<float*>(workspace), static_cast<float*>(workspace) + 2 * a.T * S};
    hipLaunchKernelGGL((distill_stats_kernel<BF16>), dim3((unsigned)(a.T * S)),
                       dim3(kSplitThreads), 0, s, a.logits, a.V, a.ld, a.idx, a.tl, a.k, a.tau, S,
                       ws);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int nblk = dlogits ? S : 1;
    hipLaunchKernelGGL((distill_grad_kernel<BF16, false>), dim3((unsigned)(a.T * nblk)),
                       dim3(kSplitThreads), 0, s, a.logits, a.V, a.ld, a.idx, a.tl, a.k, a.tau, S,
                       nblk, ws, loss, lse, a.gloss, dlogits, ldd);
    return hipGetLastError();
}

template <bool BF16>
hipError_t run_bwd(const DistillArgs& a, const float* lse, void* dlogits, int64_t ldd,
                   hipStream_t s) {
    const int S = distill_bwd_splits(a.T, a.V, BF16);
    hipLaunchKernelGGL((distill_grad_kernel<BF16, true>), dim3((unsigned)(a.T * S)),
                       dim3(kSplitThreads), 0, s, a.logits, a.V, a.ld, a.idx, a.tl, a.k, a.tau, S,
                       S, SplitWs{nullptr, nullptr}, nullptr, const_cast<float*>(lse), a.gloss,
                       dlogits, ldd);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_distill(const DistillArgs& a, float* loss, float* lse, void* dlogits,
                          int64_t ldd, void* workspace, hipStream_t s) {
    return a.bf16 ? run_distill<true>(a, loss, lse, dlogits, ldd, workspace, s)
                  : run_distill<false>(a, loss, lse, dlogits, ldd, workspace, s);
}

hipError_t launch_distill_bwd(const DistillArgs& a, const float* lse, void* dlogits, int64_t ldd,
                              hipStream_t s) {
    return a.bf16 ? run_bwd<true>(a, lse, dlogits, ldd, s) : run_bwd<false>(a, lse, dlogits, ldd, s);
}

}  // namespace qt
