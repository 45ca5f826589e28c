// Attention over the quantized cache (attn.h): bf16 queries, and the join of
// the chunks' parts.
#include "attn.h"

namespace qt {
namespace {

// One block per (sequence, query head): the chunks' bases, sums and value
// sums, 4 values a thread, the chunks dealt to 256 / (W / 4) threads each and
// joined in LDS, always in the same order.
template <int G, bool F32>
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnKernelArgs x) {
    constexpr int W = G * kGroup, COLS = W / 4, ROWS = 256 / COLS;
    const AttnArgs& a = x.a;
    const int64_t row = blockIdx.x;
    const int b = (int)(row / a.q_heads);
    const int64_t reach = a.table_pages * a.c.page;
    const int n = (int)min<int64_t>(max(a.lens[b], 0), reach);
    const int lo = a.window > 0 && a.window < n ? (int)(n - a.window) : 0;
    const int first = lo & ~(kAttnTile - 1);
    // the first chunk is there even when empty
    const int parts = max(1, (int)(((int64_t)n - first + x.chunk - 1) / x.chunk));
    const float* part = x.part + row * x.splits * (W + 4);
    const int tid = threadIdx.x, col = tid % COLS, who = tid / COLS;

    __shared__ float wmax[4];
    float mx = -INFINITY;
    for (int i = tid; i < parts; i += 256) mx = fmaxf(mx, part[(int64_t)i * (W + 4) + W]);
    mx = wave_max(mx);
    if ((tid & 63) == 0) wmax[tid >> 6] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3]));
    const float base = mx == -INFINITY ? 0.0f : mx;

    __shared__ float red[ROWS][W + 1];
    float v[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.0f;
    if (who < ROWS) {
#pragma unroll 4
        for (int i = who; i < parts; i += ROWS) {
            const float* p = part + (int64_t)i * (W + 4);
            const float e = __builtin_amdgcn_exp2f(p[W] - base);
            const f32x4_t z = *reinterpret_cast<const f32x4_t*>(p + 4 * col);
            sum += e * p[W + 1];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = __builtin_fmaf(e, z[k], v[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) red[who][4 * col + k] = v[k];
        if (col == 0) red[who][W] = sum;
    }
    __syncthreads();
    if (tid >= W) return;
    float y = 0.0f;
    sum = 0.0f;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        y += red[r][tid];
        sum += red[r][W];
    }
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
    if (tid < a.c.dim) {
        if constexpr (F32)
            static_cast<float*>(a.out)[row * a.c.dim + tid] = y * inv;
        else
            static_cast<__bf16*>(a.out)[row * a.c.dim + tid] = (__bf16)(y * inv);
    }
    if (tid == 0 && a.lse) a.lse[row] = (mx + __log2f(sum)) * 0.6931471805599453f;
}

template <bool F32>
hipError_t join(const AttnKernelArgs& k, hipStream_t s) {
    const unsigned grid = (unsigned)((int64_t)k.a.B * k.a.q_heads);
    switch (k.a.c.groups) {
        case 1: attn_join_kernel<1, F32><<<grid, 256, 0, s>>>(k); break;
        case 2: attn_join_kernel<2, F32><<<grid, 256, 0, s>>>(k); break;
        case 3: attn_join_kernel<3, F32><<<grid, 256, 0, s>>>(k); break;
        default: attn_join_kernel<4, F32><<<grid, 256, 0, s>>>(k); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_bf16(const AttnKernelArgs& k, hipStream_t s) {
    return attn_bits<kAttnWaves, false>(k, s);
}

hipError_t launch_attn_decode(const AttnArgs& a, void* workspace, hipStream_t s) {
    const AttnPlan p = attn_plan(a.B, a.c.heads, a.q_heads, a.c.dim, a.table_pages, a.c.page,
                                 a.window);
    const int64_t qe = a.bf16 ? 8 : 4;  // elements of 16 bytes
    const bool q_vec = a.c.dim % 8 == 0 && a.ldq % qe == 0 &&
                       (reinterpret_cast<uintptr_t>(a.Q) & 15) == 0;
    const uint32_t rows = (uint32_t)(a.B * a.c.heads);
    AttnKernelArgs k{a, p.chunk, p.splits, (a.q_heads / a.c.heads + 15) / 16,
                     rows, rows * (uint32_t)p.splits,
                     FastDiv::of((uint32_t)a.c.page), q_vec, static_cast<float*>(workspace)};
    hipError_t e = p.waves == kAttnMaxWaves ? launch_attn_short(k, s)
                   : a.bf16                 ? launch_attn_bf16(k, s) : launch_attn_f32(k, s);
    if (e != hipSuccess || p.splits == 1) return e;
    return a.bf16 ? join<false>(k, s) : join<true>(k, s);
}

}  // namespace qt
