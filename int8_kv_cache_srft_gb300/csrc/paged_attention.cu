// paged_attention.cu -- q4kv_paged_attention: causal attention of ragged query
// rows over a paged packed cache.
//
// In the rotated coordinates of the cache (R orthogonal): q~ = R q / lambda_K *
// sm_scale * log2 e, s_t = q~ . (codes_K scale_K)_t, an online softmax over the
// visible tokens, o = sum_t p_t (codes_V scale_V)_t / sum_t p_t, and
// out = R^T (o / lambda_V).
//
// One warp a (query token, head): it walks the sequence's tokens, each lane
// holding d/32 coordinates.
#include "codec_impl.cuh"
#include "paged.h"
#include "paged_rotate.cuh"

namespace srftkv {

static __device__ unsigned int g_paged_attn_fault;

template <int D, typename T>
__global__ void __launch_bounds__(128) paged_attn_warp_kernel(const __grid_constant__ PagedAttnParams P, int bits_k,
                                                              int bits_v) {
    constexpr int E = D / 32;
    __shared__ float2 sm[4][D / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const long long u = (long long)blockIdx.x * 4 + warp;
    const int i = (int)(u / P.Hq), hq = (int)(u - (long long)i * P.Hq), h = hq / P.rep;
    const int q0 = P.cu_q ? P.cu_q[b] : b;
    const int m = min(P.cu_q ? P.cu_q[b + 1] - q0 : 1, P.max_q);
    if (i >= m || q0 < 0 || q0 + i >= P.total_q) return;
    const int len = min(max(P.seq_lens[b], 0), P.max_len);
    const int pos = len - m + i;
    float v[E], l[E];
    rot::load_row<D, T>(static_cast<const T*>(P.q) + (q0 + i) * P.q_stride + (long long)hq * D, lane, v);
    rot::forward<D>(v, lane, P.tr_k, P.sign_mask, sm[warp]);
    if (P.lam_k) {
        rot::load_lambda<D>(P.lam_k + (long long)h * D, lane, l);
#pragma unroll
        for (int j = 0; j < E; ++j) v[j] = __fdiv_rn(v[j], l[j]);
    }
    float o[E] = {}, mx = -INFINITY, den = 0.f;
    const int ng = D >> P.lg_group, gi = (E * lane) >> P.lg_group;
    const int sb = P.sfmt == SRFTKV_SCALE_FP32 ? 4 : P.sfmt == SRFTKV_SCALE_FP16 ? 2 : 1;
    for (int t = P.window ? max(0, pos - P.window + 1) : 0; t <= pos; ++t) {
        const int pg = P.table[(long long)b * P.max_pages + (t >> P.lg_page)];
        const bool ok = (unsigned)pg < (unsigned)P.n_pages;
        if (!ok && lane == 0) atomicOr(P.fault, kFaultPage);
        const long long row = (((long long)pg * P.Hkv + h) << P.lg_page) | (t & ((1 << P.lg_page) - 1));
        float c[E], s = 0.f;
        if (ok) {
            if (bits_k == 4) rot::load_codes<D, 4>(P.kc + row * (D / 2), lane, c);
            else rot::load_codes<D, 8>(P.kc + row * D, lane, c);
            const float sc = load_scale(P.ks + row * ng * sb, gi, P.sfmt);
#pragma unroll
            for (int j = 0; j < E; ++j) s = fmaf(c[j] * sc, v[j], s);
        }
#pragma unroll
        for (int k = 16; k; k >>= 1) s += rot::sx(s, k);
        s *= P.qscale;
        const float mn = fmaxf(mx, s), f = exp2f(mx - mn), p = exp2f(s - mn);
        mx = mn;
        den = den * f + p;
        float sc = 0.f;
        if (ok) {
            if (bits_v == 4) rot::load_codes<D, 4>(P.vc + row * (D / 2), lane, c);
            else rot::load_codes<D, 8>(P.vc + row * D, lane, c);
            sc = load_scale(P.vs + row * ng * sb, gi, P.sfmt);
        }
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] = ok ? fmaf(p * sc, c[j], o[j] * f) : o[j] * f;
    }
    const float inv = den > 0.f ? 1.f / den : 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) o[j] *= inv;
    if (P.lam_v) {
        rot::load_lambda<D>(P.lam_v + (long long)h * D, lane, l);
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] = __fdiv_rn(o[j], l[j]);
    }
    rot::inverse<D>(o, lane, P.tr_v, P.sign_mask, sm[warp]);
    rot::store_row<D, T>(static_cast<T*>(P.out) + (q0 + i) * P.out_stride + (long long)hq * D, lane, o);
}

size_t paged_attention_workspace(int d, int Hq, int Hkv, int B, int total_q, int max_q, int max_len, int window) {
    return 16;
}

template <int D>
static void launch(const PagedAttnCall& c, const PagedAttnParams& P) {
    const dim3 grid((unsigned)(((long long)P.max_q * P.Hq + 3) / 4), P.B);
    if (c.dtype == SRFTKV_DTYPE_BF16)
        paged_attn_warp_kernel<D, __nv_bfloat16><<<grid, 128, 0, c.stream>>>(P, c.bits_k, c.bits_v);
    else
        paged_attn_warp_kernel<D, __half><<<grid, 128, 0, c.stream>>>(P, c.bits_k, c.bits_v);
}

int paged_attention(const PagedAttnCall& c) {
    PagedAttnParams P = c.P;
    static SymbolCache cache;
    void* f = nullptr;
    if (symbol_address(cache, &g_paged_attn_fault, &f, "the paged attention's fault word")) return SRFTKV_ERR_CUDA;
    P.fault = static_cast<unsigned int*>(f);
    if (c.d == 64) launch<64>(c, P);
    else if (c.d == 128) launch<128>(c, P);
    else launch<256>(c, P);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("paged attention launch failed: %s", cudaGetErrorString(e));
        return SRFTKV_ERR_CUDA;
    }
    return SRFTKV_OK;
}

unsigned int paged_attn_take_fault() {
    unsigned int v = 0, z = 0;
    cudaMemcpyFromSymbol(&v, g_paged_attn_fault, sizeof(v));
    if (v) cudaMemcpyToSymbol(g_paged_attn_fault, &z, sizeof(z));
    return v;
}

}  // namespace srftkv
