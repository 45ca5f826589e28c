// Internal launch interface of the gated feed-forward block, the backward
// passes and the distillation loss, with the host rules that size their
// workspaces.  Arguments here are already validated.  Host-only code apart
// from the launchers' declarations, so that the validation layer builds and
// runs without a GPU compiler.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qt_internal.h"

namespace qt {

constexpr int kCUs = 256;                  // compute units of an MI355X
constexpr int64_t kTuneMaxDim = 1 << 20;   // D, F, O, I of these calls
constexpr int64_t kTuneMaxTokens = 1 << 22;
constexpr int kDistillMaxK = 1024;
// 1 / tau, log2(e) / tau and tau times a sum of logarithms are all f32 numbers
constexpr float kDistillMinTau = 0x1p-100f, kDistillMaxTau = 0x1p100f;
constexpr int64_t kDistillMaxV = 1LL << 31;  // row strides, too

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t pad_to(int64_t a, int64_t b) { return cdiv(a, b) * b; }
// Workspace sections start at multiples of 256 bytes.
inline int64_t sect(int64_t bytes) { return pad_to(bytes, 256); }

// A launch has fewer than 2^32 threads along a dimension.  Kernels that a call of
// documented size may give more blocks than that take them in rows of equal
// length (their last row may be a few blocks too long); the others are checked
// before anything is enqueued.
inline bool launch_fits(int64_t blocks, int64_t threads) { return blocks * threads < (1LL << 32); }
struct GridRows {
    uint32_t x, y;
};
inline GridRows grid_rows(int64_t blocks, int64_t threads) {
    const int64_t rows = cdiv(blocks, ((1LL << 32) - 1) / threads);
    return {(uint32_t)cdiv(blocks, rows), (uint32_t)rows};
}

// A packed matrix and its bits (3 or 4).
struct QMat {
    const uint8_t* packed;
    const float* scales;
    int32_t bits;
};

// ------------------------------------------------------------ forward pass
// Up to this many input rows (bf16 tokens, or three pieces per f32 token)
// take the small kernel; more take the tile.
constexpr int kSmallRows = 64;
// Pieces per input value: an f32 input is split exactly into three bf16.
inline int ffn_pieces(bool bf16) { return bf16 ? 1 : 3; }
inline bool ffn_small(int64_t T, bool bf16) { return T * ffn_pieces(bf16) <= kSmallRows; }

// Bytes of the input's bf16 planes: rows of whole groups (the small form,
// where bf16 rows that are whole groups already are read in place instead), or
// operand blocks of 16 tokens (the tiles).
inline int64_t x_planes_bytes(int64_t T, int64_t D, bool bf16, bool blocked) {
    return sect(ffn_pieces(bf16) * (blocked ? pad_to(T, 16) : T) * pad_to(D, kGroup) * 2);
}

// Blocks of the launch that writes them: 256 threads, eight values each.
inline int64_t x_planes_blocks(int64_t T, int64_t D, bool blocked) {
    return cdiv((blocked ? pad_to(T, 16) : T) * (pad_to(D, kGroup) / 8), 256);
}

constexpr int kTileThreads = 512;  // of every block tile
constexpr int kTileN = 128;  // input columns of a block tile of the input gradient
constexpr int kTileK = 64;   // inner elements of a step
// 16-token tiles per wave of the 8-wave block tile: 1, 2 or 4
inline int tile_mt(int64_t T, int most) {
    int mt = 1;
    while (mt < most && 128 * mt < T) mt *= 2;
    return mt;
}
// Weight tiles (16 rows) per block: 8, and for 64 tokens per wave the 6 that
// the registers hold beside the inputs.
constexpr int tile_nt(int mt) { return mt == 4 ? 6 : 8; }
// The scale gradient takes 5 for 6 where the blocks then fill the CUs better
// (a step takes about 0.25 + 0.2 NT us): 281 against 300 us for 1024 tokens and
// 50257 rows.  In the forward tile it gained nothing (318 against 323 us for
// 512 tokens and 18432 features).
inline int ds_tile_nt(int mt, int64_t token_blocks, int64_t rows) {
    auto cost = [&](int nt) {
        return (double)cdiv(token_blocks * cdiv(rows, 16 * nt), kCUs) * (0.25 + 0.2 * nt);
    };
    return mt == 4 && cost(5) < cost(6) ? 5 : tile_nt(mt);
}

// Splits of the inner axis, so that the blocks fill the CUs: the count (at
// most `most`) with the least estimated time.  A step of a block tile takes
// about step_us; the splits' partial sums (part_bytes each) are written and
// read back at about 4 TB/s by a further launch of 5 us.
inline int inner_splits(int64_t blocks, int64_t steps, int most, double step_us,
                        double part_bytes) {
    int best = 1;
    double cost = 1e30;
    for (int s = 1; s <= most && (s == 1 || steps / s >= 4); ++s) {
        const double c = (double)cdiv(blocks * s, kCUs) * (double)cdiv(steps, s) * step_us +
                         (s > 1 ? 5.0 + 2.0 * s * part_bytes / 4e6 : 0.0);
        if (c < cost) {
            cost = c;
            best = s;
        }
    }
    return best;
}

// First group of split sp of a walk over G groups, which goes four at a time.
__host__ __device__ inline int split_begin(int G, int sp, int splits) {
    const int b = (int)((int64_t)((G + 3) / 4) * sp / splits) * 4;
    return b < G ? b : G;
}

struct FfnPlan {
    bool small;
    bool staged;       // small form: every block copies the rows into LDS
    bool planes;       // X is copied into planes by a launch of its own first
    int mt, nt;        // tile form: 16-token tiles per wave, weight tiles per block
    int splits;        // tile form: splits of the groups
    int64_t planes_off, part_off, bytes;
};
inline FfnPlan ffn_plan(int64_t T, int64_t D, int64_t F, bool bf16) {
    FfnPlan p{};
    p.small = ffn_small(T, bf16);
    // a few rows go through LDS, 16 rows and 48 KB at most (three blocks a CU)
    const int64_t rows = T * ffn_pieces(bf16);
    p.staged = p.small && rows <= 16 && rows * (pad_to(D, kGroup) + 8) * 2 <= 48 * 1024;
    p.planes = !p.staged && (!p.small || !bf16 || D % kGroup != 0);
    p.splits = 1;
    if (!p.small) {
        p.mt = tile_mt(T, bf16 ? 4 : 2);
        p.nt = tile_nt(p.mt);
        p.splits = inner_splits(cdiv(T, 128 * p.mt) * cdiv(F, 8 * p.nt), cdiv(D, kGroup), 8,
                                0.35 * p.mt * (bf16 ? 1 : 3), 2.0 * T * F * 4);
    }
    p.planes_off = 0;
    p.part_off = p.planes ? x_planes_bytes(T, D, bf16, !p.small) : 0;
    p.bytes = p.part_off + (p.splits > 1 ? sect(p.splits * 2 * T * F * 4) : 0);
    return p;
}

inline int64_t ffn_tile_blocks(const FfnPlan& p, int64_t T, int64_t F) {
    return cdiv(T, 128 * p.mt) * cdiv(F, 8 * p.nt) * p.splits;
}
// Launches that join partial sums: four values a thread.
inline bool join_fits(int64_t n) { return launch_fits(cdiv(n, 1024), 256); }
inline bool ffn_fits(const FfnPlan& p, int64_t T, int64_t F) {
    return p.small || (launch_fits(ffn_tile_blocks(p, T, F), kTileThreads) &&
                       (p.splits == 1 || join_fits(T * F)));
}

struct FfnArgs {
    QMat gate, up;
    int64_t F, D;
    int act;
    const void* X;
    bool bf16;
    int64_t T;
    void* H;
    float* pre;  // [2][T][F] or null
};
hipError_t launch_ffn_gated(const FfnArgs& a, void* workspace, hipStream_t s);
// X [T x D] -> padded bf16 planes, rows or operand blocks (ffn.hip).
hipError_t launch_x_planes(const void* X, bool bf16, bool blocked, int64_t T, int64_t D,
                           uint16_t* planes, hipStream_t s);

// ----------------------------------------------------------- backward pass
// dX = sum over the matrices of dY_m W_m; dscales of each matrix.  The
// gradients dY come from pre and dH (the feed-forward block, two matrices) or
// are given (one matrix).
struct BwdArgs {
    int nmat;          // 2: the feed-forward block, 1: a linear layer
    QMat mat[2];
    int64_t O, I, T;
    int act;
    const float* pre;  // nmat == 2: [2][T][O]
    const void* dY;    // dH or dY
    bool dy_bf16;
    const void* X;     // null without dscales
    bool bf16;         // type of X and dX
    void* dX;          // or null
    float* dscales[2]; // or null
    int accumulate;
};
struct BwdPlan {
    int dx_mt, dx_splits;
    int ds_mt, ds_nt, ds_tb, ds_splits;  // as FfnPlan; token blocks, splits of the groups
    int64_t grad_off, factor_off, dxpart_off, planes_off, dspart_off, bytes;
};
inline BwdPlan bwd_plan(int64_t T, int64_t I, int64_t O, int nmat, bool bf16, bool want_dx,
                        bool want_ds) {
    BwdPlan p{};
    const int64_t G = cdiv(I, kGroup);
    int64_t off = 0;
    p.dx_splits = 1;
    if (want_dx) {
        const int64_t K = nmat * pad_to(O, 4 * kTileK);
        p.dx_mt = tile_mt(T, 2);
        p.dx_splits = inner_splits(cdiv(T, 128 * p.dx_mt) * cdiv(I, kTileN), K / kTileK, 16,
                                   (bf16 ? 0.35 : 3.0) * p.dx_mt, 1.0 * T * I * 4);
        p.grad_off = off;
        off += sect(pad_to(T, 16) * K * (bf16 ? 2 : 4));
        p.factor_off = off;
        off += sect((T + 64) * 4);  // the tokens' factors and 64 partial maxima
        p.dxpart_off = off;
        off += p.dx_splits > 1 ? sect(p.dx_splits * T * I * 4) : 0;
    }
    if (want_ds) {
        p.planes_off = off;
        off += x_planes_bytes(T, I, bf16, true);
        p.ds_mt = tile_mt(T, bf16 ? 4 : 2);
        p.ds_tb = (int)cdiv(T, 128 * p.ds_mt);
        // the groups split freely: every block writes its own groups' sums
        p.ds_nt = ds_tile_nt(p.ds_mt, p.ds_tb, O);
        const int64_t blocks = cdiv(O, 16 * p.ds_nt) * p.ds_tb;  // of one launch
        p.ds_splits = 1;
        while (p.ds_splits < 16 && blocks * p.ds_splits < kCUs && G / (2 * p.ds_splits) >= 4)
            p.ds_splits *= 2;
        p.dspart_off = off;
        off += p.ds_tb > 1 ? sect(p.ds_tb * nmat * O * G * 4) : 0;
    }
    p.bytes = off;
    return p;
}
inline int64_t dx_tile_blocks(const BwdPlan& p, int64_t T, int64_t I) {
    return cdiv(T, 128 * p.dx_mt) * cdiv(I, kTileN) * p.dx_splits;
}
inline int64_t ds_tile_blocks(const BwdPlan& p, int64_t O) {
    return cdiv(O, 16 * p.ds_nt) * p.ds_tb * p.ds_splits;
}
inline bool bwd_fits(const BwdPlan& p, int64_t T, int64_t I, int64_t O, bool want_dx,
                     bool want_ds) {
    if (want_dx && !(launch_fits(dx_tile_blocks(p, T, I), kTileThreads) &&
                     (p.dx_splits == 1 || join_fits(T * I))))
        return false;
    return !want_ds || (launch_fits(ds_tile_blocks(p, O), kTileThreads) &&
                        (p.ds_tb == 1 || join_fits(O * cdiv(I, kGroup))));
}
hipError_t launch_bwd(const BwdArgs& a, void* workspace, hipStream_t s);

// ------------------------------------------------------------ distillation
struct DistillArgs {
    const void* logits;
    bool bf16;
    int64_t T, V, ld;
    const int32_t* idx;
    const float* tl;
    int k;
    float tau;
    const float* gloss;
};
// Blocks per row of the split form; 0: the row form (see distill.hip).
inline int distill_splits(int64_t T, int64_t V, bool bf16) {
    const int64_t vecs = cdiv(V, bf16 ? 8 : 4);
    if (vecs <= 512 || (T >= 128 && vecs <= 16 * 1024)) return 0;
    const int64_t s = vecs / 1024 < cdiv(1024, T) ? vecs / 1024 : cdiv(1024, T);
    return (int)(s < 1 ? 1 : s > 256 ? 256 : s);
}
inline int distill_bwd_splits(int64_t T, int64_t V, bool bf16) {
    const int64_t vecs = cdiv(V, bf16 ? 8 : 4);
    const int64_t s = vecs / 1024 < cdiv(2048, T) ? vecs / 1024 : cdiv(2048, T);
    return (int)(s < 1 ? 1 : s > 256 ? 256 : s);
}
inline int64_t distill_workspace(int64_t T, int64_t V, bool bf16) {
    const int S = distill_splits(T, V, bf16);
    return S == 0 ? 0 : T * (2 * S + 3) * 4;
}
hipError_t launch_distill(const DistillArgs& a, float* loss, float* lse, void* dlogits,
                          int64_t ldd, void* workspace, hipStream_t s);
hipError_t launch_distill_bwd(const DistillArgs& a, const float* lse, void* dlogits, int64_t ldd,
                              hipStream_t s);

}  // namespace qt
