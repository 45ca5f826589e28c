// C-ABI layer of the serving calls (the quantized key-value cache, the
// attention that reads it and the expert layer for a few tokens): host-side argument validation, then the launches
// on the caller's stream.  See qt.h for the contract of every entry point.
#include <cmath>

#include "api_util.h"
#include "serve.h"

namespace {

bool dtype_ok(qt_dtype t) { return t == QT_F32 || t == QT_BF16; }
int64_t esize(qt_dtype t) { return t == QT_F32 ? 4 : 2; }
bool kv_bits_ok(int32_t b) { return b == 4 || b == 8; }

bool kv_sizes_ok(int64_t n_pages, int64_t page, int64_t heads, int64_t dim) {
    return n_pages >= 1 && page >= 16 && page <= qt::kKvMaxPage && page % 16 == 0 &&
           n_pages <= qt::kKvMaxSlots / page && heads >= 1 && heads <= qt::kKvMaxHeads &&
           dim >= 1 && dim <= qt::kKvMaxDim;
}
int64_t groups(int64_t dim) { return (dim + kGroup - 1) / kGroup; }
// bytes of a cache's codes and scales (sizes checked: below 2^31 * 2^10 * 2^8 * 4)
int64_t code_bytes(int64_t n_pages, int64_t page, int64_t heads, int64_t dim, int32_t bits) {
    return n_pages * page * heads * groups(dim) * 8 * bits;
}
int64_t scale_bytes(int64_t n_pages, int64_t page, int64_t heads, int64_t dim) {
    return n_pages * page * heads * groups(dim) * 4;
}

// rows of n elements, ld apart
int64_t span(int64_t rows, int64_t n, int64_t ld, qt_dtype t) {
    return ((rows - 1) * ld + n) * esize(t);
}
// a row distance that no product with a row count overflows
bool ld_ok(int64_t ld, int64_t n) { return ld >= n && ld <= (int64_t(1) << 38); }

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

qt::KvCache cache_of(const uint8_t* kc, const float* ks, int32_t kbits, const uint8_t* vc,
                     const float* vs, int32_t vbits, int64_t n_pages, int64_t page, int64_t heads,
                     int64_t dim) {
    return qt::KvCache{const_cast<uint8_t*>(kc), const_cast<float*>(ks), kbits,
                       const_cast<uint8_t*>(vc), const_cast<float*>(vs), vbits, n_pages,
                       (int)page, (int)heads, (int)dim, (int)groups(dim)};
}

bool cache_aligned(const uint8_t* kc, const float* ks, const uint8_t* vc, const float* vs) {
    return aligned(kc, 16) && aligned(ks, 16) && aligned(vc, 16) && aligned(vs, 16);
}

}  // namespace

extern "C" {

int64_t qt_kv_bytes(int64_t n_pages, int64_t page, int64_t heads, int64_t dim, int32_t bits) {
    if (!kv_sizes_ok(n_pages, page, heads, dim) || !kv_bits_ok(bits)) return 0;
    return code_bytes(n_pages, page, heads, dim, bits);
}

qt_status qt_kv_write(const void* K, int64_t ldk, const void* V, int64_t ldv, qt_dtype xt,
                      int64_t T, const int32_t* slots, uint8_t* k_codes, float* k_scales,
                      int32_t k_bits, uint8_t* v_codes, float* v_scales, int32_t v_bits,
                      int64_t n_pages, int64_t page, int64_t heads, int64_t dim, void* stream) {
    if (!K || !V || !slots || !k_codes || !k_scales || !v_codes || !v_scales) return QT_ERR_NULL;
    if (!dtype_ok(xt)) return QT_ERR_DTYPE;
    if (!kv_sizes_ok(n_pages, page, heads, dim) || T < 1 || T > qt::kServeMaxTokens ||
        !ld_ok(ldk, heads * dim) || !ld_ok(ldv, heads * dim))
        return QT_ERR_SHAPE;
    if (!kv_bits_ok(k_bits) || !kv_bits_ok(v_bits)) return QT_ERR_ARG;
    const uintptr_t e = (uintptr_t)esize(xt);
    if (!cache_aligned(k_codes, k_scales, v_codes, v_scales) || !aligned(K, e) || !aligned(V, e) ||
        !aligned(slots, 4))
        return QT_ERR_ALIGN;
    const int64_t sb = scale_bytes(n_pages, page, heads, dim);
    const Buf out[4] = {{k_codes, code_bytes(n_pages, page, heads, dim, k_bits)}, {k_scales, sb},
                        {v_codes, code_bytes(n_pages, page, heads, dim, v_bits)}, {v_scales, sb}};
    const Buf in[3] = {{K, span(T, heads * dim, ldk, xt)}, {V, span(T, heads * dim, ldv, xt)},
                       {slots, T * 4}};
    if (any_overlap(out, in)) return QT_ERR_ALIAS;
    const qt::KvCache c = cache_of(k_codes, k_scales, k_bits, v_codes, v_scales, v_bits, n_pages,
                                   page, heads, dim);
    const qt::KvRows r{K, ldk, V, ldv, xt == QT_BF16};
    return launched(qt::launch_kv_write(c, r, slots, T, as_stream(stream)));
}

qt_status qt_kv_read(const int32_t* slots, int64_t R, const uint8_t* k_codes,
                     const float* k_scales, int32_t k_bits, const uint8_t* v_codes,
                     const float* v_scales, int32_t v_bits, int64_t n_pages, int64_t page,
                     int64_t heads, int64_t dim, void* K, void* V, qt_dtype xt, void* stream) {
    if (!slots || !k_codes || !k_scales || !v_codes || !v_scales || (!K && !V)) return QT_ERR_NULL;
    if (!dtype_ok(xt)) return QT_ERR_DTYPE;
    if (!kv_sizes_ok(n_pages, page, heads, dim) || R < 1 || R > qt::kServeMaxTokens)
        return QT_ERR_SHAPE;
    if (!kv_bits_ok(k_bits) || !kv_bits_ok(v_bits)) return QT_ERR_ARG;
    const uintptr_t e = (uintptr_t)esize(xt);
    if (!cache_aligned(k_codes, k_scales, v_codes, v_scales) || !aligned(K, e) || !aligned(V, e) ||
        !aligned(slots, 4))
        return QT_ERR_ALIGN;
    const int64_t sb = scale_bytes(n_pages, page, heads, dim), ob = R * heads * dim * esize(xt);
    const Buf out[2] = {{K, ob}, {V, ob}};
    const Buf in[5] = {{k_codes, code_bytes(n_pages, page, heads, dim, k_bits)}, {k_scales, sb},
                       {v_codes, code_bytes(n_pages, page, heads, dim, v_bits)}, {v_scales, sb},
                       {slots, R * 4}};
    if (any_overlap(out, in)) return QT_ERR_ALIAS;
    const qt::KvCache c = cache_of(k_codes, k_scales, k_bits, v_codes, v_scales, v_bits, n_pages,
                                   page, heads, dim);
    return launched(qt::launch_kv_read(c, slots, R, K, V, xt == QT_BF16, as_stream(stream)));
}

}  // extern "C"

namespace {

bool attn_sizes_ok(int64_t B, int64_t q_heads, int64_t heads, int64_t dim, int64_t table_pages,
                   int64_t page, int64_t window) {
    return kv_sizes_ok(1, page, heads, dim) && B >= 1 && B <= qt::kAttnMaxBatch &&
           q_heads >= 1 && q_heads % heads == 0 && q_heads / heads <= qt::kAttnMaxGroupHeads &&
           table_pages >= 1 && table_pages <= qt::kKvMaxSlots / page && window >= 0 &&
           qt::attn_fits(qt::attn_plan(B, heads, q_heads, dim, table_pages, page, window), B,
                         heads, q_heads);
}

}  // namespace

extern "C" {

size_t qt_attn_decode_workspace_bytes(int64_t B, int64_t q_heads, int64_t heads, int64_t dim,
                                      int64_t table_pages, int64_t page, int64_t window) {
    if (!attn_sizes_ok(B, q_heads, heads, dim, table_pages, page, window)) return 0;
    return (size_t)qt::attn_plan(B, heads, q_heads, dim, table_pages, page, window).bytes;
}

qt_status qt_attn_decode(const void* Q, int64_t ldq, qt_dtype xt, int64_t B, int64_t q_heads,
                         const uint8_t* k_codes, const float* k_scales, int32_t k_bits,
                         const uint8_t* v_codes, const float* v_scales, int32_t v_bits,
                         int64_t n_pages, int64_t page, int64_t heads, int64_t dim,
                         const int32_t* page_table, int64_t table_pages, const int32_t* lens,
                         int64_t window, float scale, void* out, float* lse, void* workspace,
                         size_t ws_bytes, void* stream) {
    if (!Q || !k_codes || !k_scales || !v_codes || !v_scales || !page_table || !lens || !out)
        return QT_ERR_NULL;
    if (!dtype_ok(xt)) return QT_ERR_DTYPE;
    if (!kv_sizes_ok(n_pages, page, heads, dim) ||
        !attn_sizes_ok(B, q_heads, heads, dim, table_pages, page, window) ||
        !ld_ok(ldq, q_heads * dim))
        return QT_ERR_SHAPE;
    // the kernel takes powers of two of scale * log2 e, which has to be a number
    if (!kv_bits_ok(k_bits) || !kv_bits_ok(v_bits) || !(std::fabs(scale) <= 0x1p127f))
        return QT_ERR_ARG;
    const size_t need =
        qt_attn_decode_workspace_bytes(B, q_heads, heads, dim, table_pages, page, window);
    if (need && (!workspace || ws_bytes < need)) return QT_ERR_WORKSPACE;
    const uintptr_t e = (uintptr_t)esize(xt);
    if (!cache_aligned(k_codes, k_scales, v_codes, v_scales) || !aligned(Q, e) || !aligned(out, e) ||
        !aligned(lse, 4) || !aligned(page_table, 4) || !aligned(lens, 4) ||
        (need && !aligned(workspace, 16)))
        return QT_ERR_ALIGN;
    const int64_t sb = scale_bytes(n_pages, page, heads, dim);
    const Buf o[3] = {{out, B * q_heads * dim * esize(xt)}, {lse, B * q_heads * 4},
                      {need ? workspace : nullptr, (int64_t)need}};
    const Buf in[7] = {{k_codes, code_bytes(n_pages, page, heads, dim, k_bits)}, {k_scales, sb},
                       {v_codes, code_bytes(n_pages, page, heads, dim, v_bits)}, {v_scales, sb},
                       {Q, span(B, q_heads * dim, ldq, xt)}, {page_table, B * table_pages * 4},
                       {lens, B * 4}};
    if (any_overlap(o, in)) return QT_ERR_ALIAS;
    const qt::AttnArgs a{cache_of(k_codes, k_scales, k_bits, v_codes, v_scales, v_bits, n_pages,
                                  page, heads, dim),
                         Q, ldq, xt == QT_BF16, (int)B, (int)q_heads, page_table, table_pages,
                         lens, window, scale, out, lse};
    return launched(qt::launch_attn_decode(a, workspace, as_stream(stream)));
}

}  // extern "C"

namespace {

bool few_sizes_ok(int64_t T, int32_t k, int32_t E, int64_t D, int64_t F) {
    return T >= 1 && T <= qt::kFewMaxTokens && D >= 1 && D <= qt::kFewMaxDim && F >= 1 &&
           F <= qt::kFewMaxDim && E >= 1 && E <= qt::kFewMaxExperts && k >= 1 &&
           k <= qt::kFewMaxTopK && k <= E;
}

}  // namespace

extern "C" {

size_t qt_moe_decode_workspace_bytes(int64_t T, int32_t k, int32_t E, int64_t D, int64_t F,
                                     qt_dtype xt) {
    if (!few_sizes_ok(T, k, E, D, F) || !dtype_ok(xt)) return 0;
    return (size_t)qt::few_workspace(T, k, E, D, F, xt == QT_BF16);
}

qt_status qt_moe_decode(const void* X, qt_dtype xt, int64_t T, int64_t D, int64_t F,
                        const float* logits, int32_t E, int32_t k, qt_act act,
                        const uint8_t* gate_packed, const float* gate_scales, int32_t gate_bits,
                        const uint8_t* up_packed, const float* up_scales, int32_t up_bits,
                        const uint8_t* down_packed, const float* down_scales, int32_t down_bits,
                        void* out, void* workspace, size_t ws_bytes, void* stream) {
    if (!X || !logits || !gate_packed || !gate_scales || !up_packed || !up_scales ||
        !down_packed || !down_scales || !out)
        return QT_ERR_NULL;
    if (!dtype_ok(xt)) return QT_ERR_DTYPE;
    if (!few_sizes_ok(T, k, E, D, F)) return QT_ERR_SHAPE;
    auto bits_ok = [](int32_t b) { return b == 3 || b == 4; };
    if (!bits_ok(gate_bits) || !bits_ok(up_bits) || !bits_ok(down_bits) ||
        (act != QT_ACT_SILU && act != QT_ACT_GELU))
        return QT_ERR_ARG;
    const size_t need = qt_moe_decode_workspace_bytes(T, k, E, D, F, xt);
    if (!workspace || ws_bytes < need) return QT_ERR_WORKSPACE;
    const uintptr_t e = (uintptr_t)esize(xt);
    if (!aligned(gate_packed, 16) || !aligned(up_packed, 16) || !aligned(down_packed, 16) ||
        !aligned(gate_scales, 4) || !aligned(up_scales, 4) || !aligned(down_scales, 4) ||
        !aligned(X, e) || !aligned(out, e) || !aligned(logits, 4) || !aligned(workspace, 16))
        return QT_ERR_ALIGN;
    auto gb = [](int32_t b) -> int64_t { return b == 3 ? kGroupBytes : kGroupBytesI4; };
    const int64_t up_groups = E * F * groups(D), down_groups = E * D * groups(F);
    const Buf o[2] = {{out, T * D * esize(xt)}, {workspace, (int64_t)need}};
    const Buf in[8] = {{X, T * D * esize(xt)}, {logits, T * E * 4},
                       {gate_packed, up_groups * gb(gate_bits)}, {gate_scales, up_groups * 4},
                       {up_packed, up_groups * gb(up_bits)}, {up_scales, up_groups * 4},
                       {down_packed, down_groups * gb(down_bits)}, {down_scales, down_groups * 4}};
    if (any_overlap(o, in)) return QT_ERR_ALIAS;
    const qt::FewArgs a{X, xt == QT_BF16, (int)T, E, k, (int)act, D, F, logits,
                        {gate_packed, gate_scales, gate_bits}, {up_packed, up_scales, up_bits},
                        {down_packed, down_scales, down_bits}, out};
    return launched(qt::launch_moe_few(a, workspace, as_stream(stream)));
}

}  // extern "C"
