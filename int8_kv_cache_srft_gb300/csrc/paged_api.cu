// paged_api.cu -- the C entry points of the paged cache: argument checks and
// the calls' parameter blocks.  Declared and documented in include/srftkv.h.
#include <climits>
#include <cmath>
#include <cstring>

#include "paged.h"

namespace srftkv {

static int bad(const char* fn, const char* msg) {
    set_error("%s: %s", fn, msg);
    return SRFTKV_ERR_INVALID;
}
static bool pow2(int v) { return v > 0 && (v & (v - 1)) == 0; }
static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
static int ilog2(int v) {
    int n = 0;
    while ((1 << n) < v) ++n;
    return n;
}

static int check_pages(const char* fn, const srftkv_pages* p) {
    if (p->d != 64 && p->d != 128 && p->d != 256) return bad(fn, "d must be 64, 128 or 256");
    if (!pow2(p->group) || p->group < 16 || p->group > p->d)
        return bad(fn, "group must be a power of two with 16 <= group <= d");
    if (!pow2(p->page_size) || p->page_size < 16 || p->page_size > 256)
        return bad(fn, "page_size must be a power of two with 16 <= page_size <= 256");
    if (p->n_pages <= 0 || p->H <= 0 || p->H > 65535) return bad(fn, "need n_pages > 0 and 0 < H <= 65535");
    if ((long long)p->n_pages * p->H > INT_MAX) return bad(fn, "n_pages * H must be below 2^31");
    if (p->bits != 4 && p->bits != 8) return bad(fn, "bits must be 4 or 8");
    if (p->transform != SRFTKV_TRANSFORM_SRFT && p->transform != SRFTKV_TRANSFORM_SRHT)
        return bad(fn, "transform must be SRFTKV_TRANSFORM_SRFT or SRFTKV_TRANSFORM_SRHT");
    if (p->scale_format != SRFTKV_SCALE_FP32 && p->scale_format != SRFTKV_SCALE_FP16 &&
        p->scale_format != SRFTKV_SCALE_E8M0)
        return bad(fn, "scale_format must be SRFTKV_SCALE_FP32, _FP16 or _E8M0");
    if (!p->codes || !p->scales) return bad(fn, "codes and scales must not be NULL");
    if (!aligned16(p->codes) || !aligned16(p->scales) || !aligned16(p->lambda))
        return bad(fn, "codes, scales and lambda must be 16-byte aligned");
    return SRFTKV_OK;
}
static int check_pair(const char* fn, const srftkv_pages* k, const srftkv_pages* v) {
    if (k->n_pages != v->n_pages || k->H != v->H || k->page_size != v->page_size || k->d != v->d || k->group != v->group)
        return bad(fn, "k and v must share n_pages, H, page_size, d and group");
    return SRFTKV_OK;
}
// a row stride in elements: 0 (dense) or a multiple of 8 of at least the row
static bool stride_ok(int64_t s, int64_t row) { return s == 0 || (s >= row && s % 8 == 0); }

static int paged_codec(const char* fn, const srftkv_pages* k, void* xk, int64_t xks, const srftkv_pages* v, void* xv,
                       int64_t xvs, const int64_t* slots, int n_tokens, int dtype, uint64_t seed, void* stream,
                       bool quantize) {
    if (!k && !v) return bad(fn, "at least one of k, v must be given");
    const srftkv_pages* sides[2] = {k, v};
    void* xs[2] = {xk, xv};
    const int64_t strides[2] = {xks, xvs};
    if (dtype != SRFTKV_DTYPE_FP16 && dtype != SRFTKV_DTYPE_BF16)
        return bad(fn, "dtype must be SRFTKV_DTYPE_FP16 or SRFTKV_DTYPE_BF16");
    if (n_tokens < 0) return bad(fn, "n_tokens must be >= 0");
    PagedCodecCall c;
    std::memset(&c, 0, sizeof(c));
    for (int i = 0; i < 2; ++i) {
        const srftkv_pages* p = sides[i];
        if (!p) continue;
        const int rc = check_pages(fn, p);
        if (rc) return rc;
        const int64_t row = (int64_t)p->H * p->d;
        if (n_tokens && (!xs[i] || !aligned16(xs[i]))) return bad(fn, "x must be a 16-byte aligned device pointer");
        if (!stride_ok(strides[i], row)) return bad(fn, "a token stride must be 0 or a multiple of 8 of at least H * d");
        PagedSideK& s = c.P.side[c.P.n_sides++];
        s.x = xs[i];
        s.x_stride = strides[i] ? strides[i] : row;
        s.codes = static_cast<uint8_t*>(p->codes);
        s.scales = static_cast<uint8_t*>(p->scales);
        s.lambda = p->lambda;
        s.bits = p->bits;
        s.transform = p->transform;
        s.sfmt = p->scale_format;
    }
    if (k && v) {
        const int rc = check_pair(fn, k, v);
        if (rc) return rc;
    }
    const srftkv_pages* p = k ? k : v;
    if (n_tokens && (!slots || (reinterpret_cast<uintptr_t>(slots) & 7)))
        return bad(fn, "slots must be an 8-byte aligned device pointer");
    if ((long long)n_tokens * p->H * 2 > INT_MAX) return bad(fn, "n_tokens * H must be below 2^30");
    if (n_tokens == 0) return SRFTKV_OK;
    const int rc = current_device_ok();
    if (rc) return rc;
    c.P.slots = slots;
    c.P.n_tokens = n_tokens;
    c.P.H = p->H;
    c.P.group = p->group;
    c.P.lg_group = ilog2(p->group);
    c.P.lg_page = ilog2(p->page_size);
    c.P.n_slots = (long long)p->n_pages * p->page_size;
    sign_masks(p->d, seed, c.P.sign_mask);
    c.d = p->d;
    c.dtype = dtype;
    c.stream = static_cast<cudaStream_t>(stream);
    return quantize ? paged_quantize(c) : paged_dequantize(c);
}

// The checks of a batch and its query heads that need no pointers
static int check_batch(const char* fn, const srftkv_pages* k, int Hq, const srftkv_paged_batch* b) {
    if (Hq <= 0 || Hq % k->H || Hq / k->H > 128) return bad(fn, "Hq must be a multiple of H, at most 128 times it");
    if (b->B < 0 || b->total_q < 0 || b->max_q < 0) return bad(fn, "B, total_q and max_q must be >= 0");
    if (b->max_pages <= 0) return bad(fn, "max_pages must be > 0");
    if ((long long)b->max_pages * k->page_size > (1 << 30)) return bad(fn, "max_pages * page_size must be at most 2^30");
    if (b->max_seq_len < 0 || b->max_seq_len > b->max_pages * k->page_size)
        return bad(fn, "max_seq_len must be between 0 and max_pages * page_size");
    if ((long long)b->total_q * Hq > INT_MAX) return bad(fn, "total_q * Hq must be below 2^31");
    if (b->max_q > b->total_q) return bad(fn, "max_q must not exceed total_q");
    if (b->B && b->total_q && b->max_q < 1) return bad(fn, "max_q must be at least 1");
    if ((long long)b->max_q * (Hq / k->H) > (1 << 22)) return bad(fn, "max_q * Hq / H must be at most 2^22");
    if ((long long)b->B * k->H > 65535) return bad(fn, "B * H must be at most 65535");
    return SRFTKV_OK;
}
// A window of all positions is none
static int window_of(int window, int max_len) { return window < max_len ? window : 0; }
static int batch_len(const srftkv_pages* k, const srftkv_paged_batch* b) {
    return b->max_seq_len ? b->max_seq_len : b->max_pages * k->page_size;
}

}  // namespace srftkv

using namespace srftkv;

extern "C" {

int srft_kv_quantize_paged(const srftkv_pages* k, const void* xk, int64_t xk_stride, const srftkv_pages* v,
                           const void* xv, int64_t xv_stride, const int64_t* slots, int n_tokens, int dtype,
                           uint64_t sign_seed, void* stream) {
    return paged_codec("srft_kv_quantize_paged", k, const_cast<void*>(xk), xk_stride, v, const_cast<void*>(xv), xv_stride,
                       slots, n_tokens, dtype, sign_seed, stream, true);
}

int srft_kv_dequantize_paged(const srftkv_pages* k, void* xk, int64_t xk_stride, const srftkv_pages* v, void* xv,
                             int64_t xv_stride, const int64_t* slots, int n_tokens, int dtype, uint64_t sign_seed,
                             void* stream) {
    return paged_codec("srft_kv_dequantize_paged", k, xk, xk_stride, v, xv, xv_stride, slots, n_tokens, dtype, sign_seed,
                       stream, false);
}

size_t q4kv_paged_attention_workspace_size(const srftkv_pages* k, int Hq, const srftkv_paged_batch* b, int window) {
    const char* fn = "q4kv_paged_attention_workspace_size";
    if (!k || !b) return 0;
    if (check_pages(fn, k) || check_batch(fn, k, Hq, b) || window < 0) return 0;
    const int len = batch_len(k, b);
    return paged_attention_workspace(k->d, Hq, k->H, b->B, b->total_q, b->max_q, len, window_of(window, len));
}

int q4kv_paged_attention(const void* q, int64_t q_stride, void* out, int64_t out_stride, int dtype, int Hq,
                         const srftkv_pages* k, const srftkv_pages* v, const srftkv_paged_batch* b, float sm_scale,
                         int window, uint64_t sign_seed, void* workspace, size_t workspace_bytes, void* stream) {
    const char* fn = "q4kv_paged_attention";
    if (!k || !v || !b) return bad(fn, "k, v and batch must not be NULL");
    int rc = check_pages(fn, k);
    if (!rc) rc = check_pages(fn, v);
    if (!rc) rc = check_pair(fn, k, v);
    if (!rc) rc = check_batch(fn, k, Hq, b);
    if (rc) return rc;
    if (k->scale_format != v->scale_format) return bad(fn, "k and v must share the scale format");
    if (dtype != SRFTKV_DTYPE_FP16 && dtype != SRFTKV_DTYPE_BF16)
        return bad(fn, "dtype must be SRFTKV_DTYPE_FP16 or SRFTKV_DTYPE_BF16");
    if (window < 0) return bad(fn, "window must be >= 0");
    if (!std::isfinite(sm_scale)) return bad(fn, "sm_scale must be finite");
    const int64_t row = (int64_t)Hq * k->d;
    if (!stride_ok(q_stride, row) || !stride_ok(out_stride, row))
        return bad(fn, "a token stride must be 0 or a multiple of 8 of at least Hq * d");
    if (b->B == 0 || b->total_q == 0) return SRFTKV_OK;
    if (!q || !out || !aligned16(q) || !aligned16(out)) return bad(fn, "q and out must be 16-byte aligned device pointers");
    if (!b->block_table || !b->seq_lens) return bad(fn, "block_table and seq_lens must not be NULL");
    if ((reinterpret_cast<uintptr_t>(b->block_table) | reinterpret_cast<uintptr_t>(b->seq_lens) |
         reinterpret_cast<uintptr_t>(b->cu_q)) & 3)
        return bad(fn, "block_table, seq_lens and cu_q must be 4-byte aligned");
    if (!b->cu_q && b->total_q < b->B) return bad(fn, "without cu_q, total_q must be at least B");
    rc = current_device_ok();
    if (rc) return rc;
    PagedAttnCall c;
    std::memset(&c, 0, sizeof(c));
    PagedAttnParams& P = c.P;
    P.q = q;
    P.out = out;
    P.q_stride = q_stride ? q_stride : row;
    P.out_stride = out_stride ? out_stride : row;
    P.kc = static_cast<const uint8_t*>(k->codes);
    P.ks = static_cast<const uint8_t*>(k->scales);
    P.vc = static_cast<const uint8_t*>(v->codes);
    P.vs = static_cast<const uint8_t*>(v->scales);
    P.lam_k = k->lambda;
    P.lam_v = v->lambda;
    P.table = b->block_table;
    P.seq_lens = b->seq_lens;
    P.cu_q = b->cu_q;
    P.B = b->B;
    P.max_pages = b->max_pages;
    P.total_q = b->total_q;
    P.max_q = b->max_q;
    P.max_len = batch_len(k, b);
    P.Hq = Hq;
    P.Hkv = k->H;
    P.rep = Hq / k->H;
    P.n_pages = k->n_pages;
    P.lg_page = ilog2(k->page_size);
    P.group = k->group;
    P.lg_group = ilog2(k->group);
    P.sfmt = k->scale_format;
    P.tr_k = k->transform;
    P.tr_v = v->transform;
    P.window = window_of(window, P.max_len);
    const float sc = sm_scale > 0.f ? sm_scale : 1.0f / std::sqrt((float)k->d);
    P.qscale = sc * 1.4426950408889634f;
    sign_masks(k->d, sign_seed, P.sign_mask);
    c.d = k->d;
    c.dtype = dtype;
    c.bits_k = k->bits;
    c.bits_v = v->bits;
    c.workspace = workspace;
    c.workspace_bytes = workspace_bytes;
    c.stream = static_cast<cudaStream_t>(stream);
    const size_t need = paged_attention_workspace(k->d, Hq, k->H, P.B, P.total_q, P.max_q, P.max_len, P.window);
    if (need && (!workspace || !aligned16(workspace) || workspace_bytes < need)) {
        set_error("%s: workspace must be 16-byte aligned and hold %zu bytes (got %zu)", fn, need, workspace_bytes);
        return SRFTKV_ERR_INVALID;
    }
    return paged_attention(c);
}

}  // extern "C"
