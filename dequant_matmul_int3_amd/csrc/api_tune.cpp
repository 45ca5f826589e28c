// C-ABI layer of the gated feed-forward block, the backward passes and the
// distillation loss: host-side argument validation, then the launches on the
// caller's stream.  See qt.h for the contract of every entry point.
#include "api_util.h"
#include "tune.h"

namespace {

bool dtype_ok(qt_dtype t) { return t == QT_F32 || t == QT_BF16; }
int64_t esize(qt_dtype t) { return t == QT_F32 ? 4 : 2; }
int64_t group_bytes(int32_t bits) { return bits == 3 ? kGroupBytes : kGroupBytesI4; }

bool sizes_ok(int64_t T, int64_t D, int64_t F) {
    return T >= 1 && T <= qt::kTuneMaxTokens && D >= 1 && D <= qt::kTuneMaxDim && F >= 1 &&
           F <= qt::kTuneMaxDim;
}

// A buffer of a call: address and bytes (null: not there).
struct Buf {
    const void* p;
    int64_t n;
};
template <int NO, int NI>
bool any_overlap(const Buf (&out)[NO], const Buf (&in)[NI]) {
    for (int a = 0; a < NO; ++a) {
        for (int b = 0; b < NI; ++b)
            if (overlap(out[a].p, out[a].n, in[b].p, in[b].n)) return true;
        for (int b = a + 1; b < NO; ++b)
            if (overlap(out[a].p, out[a].n, out[b].p, out[b].n)) return true;
    }
    return false;
}

qt_status workspace_ok(const void* workspace, size_t ws_bytes, size_t need) {
    if (need == 0) return QT_OK;
    if (!workspace || ws_bytes < need) return QT_ERR_WORKSPACE;
    return aligned(workspace, 16) ? QT_OK : QT_ERR_ALIGN;
}

// A few bf16 rows of whole groups may be read in place, with 16-byte loads;
// everything else copies X first, from its elements' alignment.
uintptr_t x_alignment(qt_dtype xt, int64_t T, int64_t D) {
    const bool in_place = xt == QT_BF16 && D % kGroup == 0 && qt::ffn_small(T, true);
    return in_place ? 16 : (uintptr_t)esize(xt);
}

}  // namespace

extern "C" {

size_t qt_ffn_gated_workspace_bytes(int64_t T, int64_t D, int64_t F, qt_dtype xt) {
    if (!sizes_ok(T, D, F) || !dtype_ok(xt)) return 0;
    return (size_t)qt::ffn_plan(T, D, F, xt == QT_BF16).bytes;
}

qt_status qt_ffn_gated(const uint8_t* gate_packed, const float* gate_scales, int32_t gate_bits,
                       const uint8_t* up_packed, const float* up_scales, int32_t up_bits,
                       int64_t F, int64_t D, qt_act act, const void* X, qt_dtype xt, int64_t T,
                       void* H, float* pre, void* workspace, size_t ws_bytes, void* stream) {
    if (!gate_packed || !gate_scales || !up_packed || !up_scales || !X || !H) return QT_ERR_NULL;
    if (!dtype_ok(xt)) return QT_ERR_DTYPE;
    if (!sizes_ok(T, D, F)) return QT_ERR_SHAPE;
    if ((gate_bits != 3 && gate_bits != 4) || (up_bits != 3 && up_bits != 4)) return QT_ERR_ARG;
    if (act != QT_ACT_SILU && act != QT_ACT_GELU) return QT_ERR_ARG;
    const size_t need = qt_ffn_gated_workspace_bytes(T, D, F, xt);
    const qt_status st = workspace_ok(workspace, ws_bytes, need);
    if (st != QT_OK) return st;
    if (!aligned(gate_packed, 16) || !aligned(up_packed, 16) || !aligned(gate_scales, 4) ||
        !aligned(up_scales, 4) || !aligned(X, x_alignment(xt, T, D)) ||
        !aligned(H, (uintptr_t)esize(xt)) || !aligned(pre, 4))
        return QT_ERR_ALIGN;
    const int64_t G = qt_groups(D), e = esize(xt);
    const Buf out[3] = {{H, T * F * e}, {pre, 2 * T * F * 4}, {workspace, (int64_t)need}};
    const Buf in[5] = {{gate_packed, F * G * group_bytes(gate_bits)}, {gate_scales, F * G * 4},
                       {up_packed, F * G * group_bytes(up_bits)}, {up_scales, F * G * 4},
                       {X, T * D * e}};
    if (any_overlap(out, in)) return QT_ERR_ALIAS;
    const qt::FfnArgs a{{gate_packed, gate_scales, gate_bits}, {up_packed, up_scales, up_bits},
                        F, D, (int)act, X, xt == QT_BF16, T, H, pre};
    return launched(qt::launch_ffn_gated(a, workspace, as_stream(stream)));
}

size_t qt_ffn_gated_bwd_workspace_bytes(int64_t T, int64_t D, int64_t F, qt_dtype xt,
                                        int32_t want_dx, int32_t want_dscales) {
    if (!sizes_ok(T, D, F) || !dtype_ok(xt)) return 0;
    return (size_t)qt::bwd_plan(T, D, F, 2, xt == QT_BF16, want_dx != 0, want_dscales != 0).bytes;
}

qt_status qt_ffn_gated_bwd(const uint8_t* gate_packed, const float* gate_scales,
                           int32_t gate_bits, const uint8_t* up_packed, const float* up_scales,
                           int32_t up_bits, int64_t F, int64_t D, qt_act act, const float* pre,
                           const void* dH, const void* X, qt_dtype xt, int64_t T, void* dX,
                           float* dgate_scales, float* dup_scales, int32_t accumulate,
                           void* workspace, size_t ws_bytes, void* stream) {
    const bool want_ds = dgate_scales || dup_scales;
    if (!gate_packed || !gate_scales || !up_packed || !up_scales || !pre || !dH) return QT_ERR_NULL;
    if (!dX && !want_ds) return QT_ERR_NULL;
    if (want_ds && (!dgate_scales || !dup_scales || !X)) return QT_ERR_NULL;
    if (!dtype_ok(xt)) return QT_ERR_DTYPE;
    if (!sizes_ok(T, D, F)) return QT_ERR_SHAPE;
    if ((gate_bits != 3 && gate_bits != 4) || (up_bits != 3 && up_bits != 4)) return QT_ERR_ARG;
    if ((act != QT_ACT_SILU && act != QT_ACT_GELU) || (accumulate != 0 && accumulate != 1))
        return QT_ERR_ARG;
    const size_t need = qt_ffn_gated_bwd_workspace_bytes(T, D, F, xt, dX != nullptr, want_ds);
    const qt_status st = workspace_ok(workspace, ws_bytes, need);
    if (st != QT_OK) return st;
    const uintptr_t ea = (uintptr_t)esize(xt);
    if (!aligned(gate_packed, 16) || !aligned(up_packed, 16) || !aligned(gate_scales, 4) ||
        !aligned(up_scales, 4) || !aligned(pre, 4) || !aligned(dH, ea) || !aligned(dX, ea) ||
        !aligned(dgate_scales, 4) || !aligned(dup_scales, 4) ||
        (want_ds && !aligned(X, ea)))
        return QT_ERR_ALIGN;
    const int64_t G = qt_groups(D), e = esize(xt);
    const Buf out[4] = {{dX, T * D * e}, {dgate_scales, F * G * 4}, {dup_scales, F * G * 4},
                        {workspace, (int64_t)need}};
    const Buf in[7] = {{gate_packed, F * G * group_bytes(gate_bits)}, {gate_scales, F * G * 4},
                       {up_packed, F * G * group_bytes(up_bits)}, {up_scales, F * G * 4},
                       {pre, 2 * T * F * 4}, {dH, T * F * e}, {want_ds ? X : nullptr, T * D * e}};
    if (any_overlap(out, in)) return QT_ERR_ALIAS;
    const qt::BwdArgs a{2, {{gate_packed, gate_scales, gate_bits}, {up_packed, up_scales, up_bits}},
                        F, D, T, (int)act, pre, dH, xt == QT_BF16, X, xt == QT_BF16, dX,
                        {dgate_scales, dup_scales}, accumulate};
    return launched(qt::launch_bwd(a, workspace, as_stream(stream)));
}

size_t qt_matmul_bwd_workspace_bytes(int64_t B, int64_t I, int64_t O, qt_dtype xt,
                                     int32_t want_dx, int32_t want_dscales) {
    if (!sizes_ok(B, I, O) || !dtype_ok(xt)) return 0;
    return (size_t)qt::bwd_plan(B, I, O, 1, xt == QT_BF16, want_dx != 0, want_dscales != 0).bytes;
}

qt_status qt_matmul_bwd(const uint8_t* packed, const float* scales, int32_t bits, int64_t O,
                        int64_t I, const void* dY, qt_dtype yt, const void* X, qt_dtype xt,
                        int64_t B, void* dX, float* dscales, int32_t accumulate,
                        void* workspace, size_t ws_bytes, void* stream) {
    if (!packed || !scales || !dY || (!dX && !dscales) || (dscales && !X)) return QT_ERR_NULL;
    if (!dtype_ok(xt) || !dtype_ok(yt)) return QT_ERR_DTYPE;
    if (!sizes_ok(B, I, O)) return QT_ERR_SHAPE;
    if ((bits != 3 && bits != 4) || (accumulate != 0 && accumulate != 1)) return QT_ERR_ARG;
    const size_t need =
        qt_matmul_bwd_workspace_bytes(B, I, O, xt, dX != nullptr, dscales != nullptr);
    const qt_status st = workspace_ok(workspace, ws_bytes, need);
    if (st != QT_OK) return st;
    if (!aligned(packed, 16) || !aligned(scales, 4) || !aligned(dY, (uintptr_t)esize(yt)) ||
        !aligned(dX, (uintptr_t)esize(xt)) || !aligned(dscales, 4) ||
        (dscales && !aligned(X, (uintptr_t)esize(xt))))
        return QT_ERR_ALIGN;
    const int64_t G = qt_groups(I);
    const Buf out[3] = {{dX, B * I * esize(xt)}, {dscales, O * G * 4}, {workspace, (int64_t)need}};
    const Buf in[4] = {{packed, O * G * group_bytes(bits)}, {scales, O * G * 4},
                       {dY, B * O * esize(yt)}, {dscales ? X : nullptr, B * I * esize(xt)}};
    if (any_overlap(out, in)) return QT_ERR_ALIAS;
    const qt::BwdArgs a{1, {{packed, scales, bits}, {nullptr, nullptr, 3}}, O, I, B, 0, nullptr, dY,
                        yt == QT_BF16, X, xt == QT_BF16, dX, {dscales, nullptr}, accumulate};
    return launched(qt::launch_bwd(a, workspace, as_stream(stream)));
}

namespace {

// The checks that both distillation calls share; dlogits null: not wanted.
qt_status distill_ok(const void* logits, qt_dtype lt, int64_t T, int64_t V, int64_t ldl,
                     const int32_t* idx, const float* tlogits, int32_t k, float tau,
                     const float* gloss, const void* dlogits, int64_t ldd) {
    if (!dtype_ok(lt)) return QT_ERR_DTYPE;
    if (T < 1 || T > qt::kTuneMaxTokens || V < 1 || V >= qt::kDistillMaxV || ldl < V ||
        ldl >= qt::kDistillMaxV || (dlogits && (ldd < V || ldd >= qt::kDistillMaxV)))
        return QT_ERR_SHAPE;
    if (k < 1 || k > qt::kDistillMaxK || !(tau >= qt::kDistillMinTau && tau <= qt::kDistillMaxTau))
        return QT_ERR_ARG;
    const uintptr_t e = (uintptr_t)esize(lt);
    if (!aligned(logits, e) || !aligned(dlogits, e) || !aligned(idx, 4) || !aligned(tlogits, 4) ||
        !aligned(gloss, 4))
        return QT_ERR_ALIGN;
    return QT_OK;
}

int64_t row_span(int64_t T, int64_t V, int64_t ld, qt_dtype t) {
    return ((T - 1) * ld + V) * esize(t);
}

}  // namespace

size_t qt_distill_topk_workspace_bytes(int64_t T, int64_t V, qt_dtype lt) {
    if (T < 1 || T > qt::kTuneMaxTokens || V < 1 || V >= qt::kDistillMaxV || !dtype_ok(lt)) return 0;
    return (size_t)qt::distill_workspace(T, V, lt == QT_BF16);
}

qt_status qt_distill_topk(const void* logits, qt_dtype lt, int64_t T, int64_t V, int64_t ldl,
                          const int32_t* idx, const float* tlogits, int32_t k, float tau,
                          float* loss, float* lse, const float* gloss, void* dlogits,
                          int64_t ldd, void* workspace, size_t ws_bytes, void* stream) {
    if (!logits || !idx || !tlogits || !loss || !lse) return QT_ERR_NULL;
    qt_status st = distill_ok(logits, lt, T, V, ldl, idx, tlogits, k, tau, gloss, dlogits, ldd);
    if (st != QT_OK) return st;
    const size_t need = qt_distill_topk_workspace_bytes(T, V, lt);
    st = workspace_ok(workspace, ws_bytes, need);
    if (st != QT_OK) return st;
    if (!aligned(loss, 4) || !aligned(lse, 4)) return QT_ERR_ALIGN;
    const bool in_place = dlogits == logits && (ldd == ldl || T == 1);
    const Buf lg{logits, row_span(T, V, ldl, lt)};
    const Buf out[4] = {{loss, T * 4}, {lse, T * 4}, {workspace, (int64_t)need},
                        {in_place ? nullptr : dlogits, dlogits ? row_span(T, V, ldd, lt) : 0}};
    const Buf in[4] = {lg, {idx, T * k * 4}, {tlogits, T * k * 4}, {gloss, T * 4}};
    if (any_overlap(out, in)) return QT_ERR_ALIAS;
    if (in_place)
        for (int i = 1; i < 4; ++i)
            if (overlap(lg.p, lg.n, in[i].p, in[i].n)) return QT_ERR_ALIAS;
    const qt::DistillArgs a{logits, lt == QT_BF16, T, V, ldl, idx, tlogits, k, tau, gloss};
    return launched(qt::launch_distill(a, loss, lse, dlogits, ldd, workspace, as_stream(stream)));
}

qt_status qt_distill_topk_bwd(const void* logits, qt_dtype lt, int64_t T, int64_t V, int64_t ldl,
                              const int32_t* idx, const float* tlogits, int32_t k, float tau,
                              const float* lse, const float* gloss, void* dlogits, int64_t ldd,
                              void* stream) {
    if (!logits || !idx || !tlogits || !lse || !dlogits) return QT_ERR_NULL;
    const qt_status st =
        distill_ok(logits, lt, T, V, ldl, idx, tlogits, k, tau, gloss, dlogits, ldd);
    if (st != QT_OK) return st;
    if (!aligned(lse, 4)) return QT_ERR_ALIGN;
    const bool in_place = dlogits == logits && (ldd == ldl || T == 1);
    const Buf out[1] = {{dlogits, row_span(T, V, ldd, lt)}};
    const Buf in[5] = {{in_place ? nullptr : logits, row_span(T, V, ldl, lt)}, {idx, T * k * 4},
                       {tlogits, T * k * 4}, {gloss, T * 4}, {lse, T * 4}};
    if (any_overlap(out, in)) return QT_ERR_ALIAS;
    const qt::DistillArgs a{logits, lt == QT_BF16, T, V, ldl, idx, tlogits, k, tau, gloss};
    return launched(qt::launch_distill_bwd(a, lse, dlogits, ldd, as_stream(stream)));
}

}  // extern "C"
