// paged_attention.cu -- q4kv_paged_attention: causal attention of ragged query
// rows over a paged packed cache: how a call's work is divided, and the kernel
// that joins partial results.
//
// In the rotated coordinates of the cache (R orthogonal): q~ = R q / lambda_K *
// sm_scale * log2 e, s_t = q~ . (codes_K scale_K)_t, an online softmax over the
// visible tokens, o = sum_t p_t (codes_V scale_V)_t / sum_t p_t, and
// out = R^T (o / lambda_V).
#include <algorithm>

#include "attn_frag.cuh"
#include "paged.h"
#include "paged_rotate.cuh"

namespace srftkv {

static __device__ unsigned int g_paged_attn_fault;

// Join the partial results of one (query token, head), one warp a row:
// o = sum_p 2^(m_p - M) acc_p / sum_p 2^(m_p - M) l_p, then / lambda_V and R^T.
// Partials with m = -inf are empty and their acc counts for nothing.
template <int D, typename T>
__global__ void __launch_bounds__(128) paged_attn_combine_kernel(const __grid_constant__ PagedAttnParams P, int n_parts,
                                                                 const float* __restrict__ part_ml,
                                                                 const float* __restrict__ part_acc) {
    constexpr int E = D / 32;
    __shared__ float2 sm[4][D / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const long long u = (long long)blockIdx.x * 4 + warp;
    const int i = (int)(u / P.Hq), hq = (int)(u - (long long)i * P.Hq), h = hq / P.rep;
    const int q0 = P.cu_q ? P.cu_q[b] : b;
    const int m = min(P.cu_q ? P.cu_q[b + 1] - q0 : 1, P.max_q);
    griddep_wait();  // the partial results
    if (i >= m || q0 < 0 || q0 + i >= P.total_q) return;
    const long long at = ((long long)(q0 + i) * P.Hq + hq) * n_parts;
    // four partials at a time, their loads all at once; an empty one's acc holds anything and is not used
    float M = -INFINITY, o[E] = {}, l = 0.f;
    for (int p0 = 0; p0 < n_parts; p0 += 4) {
        float2 ml[4];
        float a[4][E];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int p = min(p0 + k, n_parts - 1);
            ml[k] = __ldg(reinterpret_cast<const float2*>(part_ml) + at + p);
            rot::load_lambda<D>(part_acc + (at + p) * D, lane, a[k]);
            if (p0 + k >= n_parts) ml[k].x = -INFINITY;
        }
        const float mn = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);
        if (mn == -INFINITY) continue;
        const float f = exp2f(M - mn);
        M = mn;
        l *= f;
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] *= f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (ml[k].x == -INFINITY) continue;
            const float w = exp2f(ml[k].x - mn);
            l = fmaf(w, ml[k].y, l);
#pragma unroll
            for (int j = 0; j < E; ++j) o[j] = fmaf(w, a[k][j], o[j]);
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int j = 0; j < E; ++j) o[j] *= inv;
    if (P.lam_v) {
        float lam[E];
        rot::load_lambda<D>(P.lam_v + (long long)h * D, lane, lam);
#pragma unroll
        for (int j = 0; j < E; ++j) o[j] = __fdiv_rn(o[j], lam[j]);
    }
    rot::inverse<D>(o, lane, P.tr_v, P.sign_mask, sm[warp]);
    rot::store_row<D, T>(static_cast<T*>(P.out) + (q0 + i) * P.out_stride + (long long)hq * D, lane, o);
}

// How a call is divided: a pure function of its sizes (the workspace size and the launch both ask for it).
struct Plan {
    bool few;        // the split kernel; else the tile kernel
    SplitWork S;
    TileWork W;
    int blocks;      // tile kernel: row blocks a (sequence, kv head)
    int n_parts;     // partial results a row; 1: written as the answer at once
    bool expand;     // tile kernel: the tiles are laid down as fp16 first
    size_t img_off;  // part_ml at 0, part_acc at acc_off, images here
    size_t acc_off;
    size_t bytes;
};
// The most workspace that laying tiles down may take (an eighth of it is what one layer of 128 k tokens and 2 kv heads
// takes); past it they are turned where they are used.
constexpr size_t kMaxImages = 1ull << 30;
static Plan work_out_plan(int d, int Hq, int Hkv, int B, int total_q, int max_q, int max_len, int window, int sm_count) {
    Plan p = {};
    const int rep = Hq / Hkv;
    const long long rows = (long long)max_q * rep, sms = sm_count;
    // 8 ragged sequences of 9 k to 32 k tokens, 8 kv heads, int4: the split kernel reads the cache once for every 8 rows
    // (d = 256: 4), the tile kernel once for 128; d = 64: 197 us against 225 at 40 rows, 233 against 226 at 48; d = 128:
    // 223 against 277 at 20 rows, 288 against 270 at 32; d = 256: 501 against 617 at 24, 663 against 619 at 32
    p.few = rows <= (d == 64 ? 40 : 28);
    if (p.few) {
        p.S.nr = rows > 4 && d <= 128 ? 2 : 1;
        p.S.groups = (int)((rows + 4 * p.S.nr - 1) / (4 * p.S.nr));
        // tokens any row group sees, with the chunk its window starts inside
        long long see = max_len;
        if (window) see = std::min<long long>(see, (long long)window + max_q - 1 + 31);
        const long long base = (long long)B * Hkv * p.S.groups;
        // Two or three CTAs run on an SM.  Lengths are ragged in earnest and max_seq_len is only their bound, so from
        // four sequences on a split is a quarter of what one CTA would get if all were the longest (the scheduler evens the
        // rest out; with one sequence there is nothing to even out: 49 us in one wave, 74 in four, at 20 rows), but
        // no less than 512 tokens (the rotation, fragments and join are worth about 256), unless one wave holds
        // all of them anyway (24 sequences of 1 to 9215 tokens: 66 us with a quarter, 68 with a half, 81 with all of it).
        const long long at_once = (d == 256 ? 2 : 3) * sms;
        const long long even = (see * base + at_once - 1) / at_once;  // tokens of a CTA in one wave
        long long tokens = std::max(even / std::min(B, 4), std::min<long long>(even, 512));
        tokens = (std::min(tokens, see) + 127) / 128 * 128;
        p.S.tokens = (int)tokens;
        p.S.n_splits = (int)((see + tokens - 1) / tokens);
        p.n_parts = p.S.n_parts = p.S.n_splits;
    } else {
        const int bn = d == 256 ? 64 : 128;
        p.W.dual = d != 256 && rows <= 128;
        p.W.rows_per_block = d == 256 || p.W.dual ? 128 : 256;
        p.blocks = (int)((rows + p.W.rows_per_block - 1) / p.W.rows_per_block);
        // the most tiles any block sees
        long long see = max_len;
        if (window) see = std::min<long long>(see, (long long)window + (p.W.rows_per_block - 1) / rep + 1);
        long long tiles = (see + bn - 1) / bn;
        if (window) tiles = std::min<long long>((max_len + bn - 1) / bn, tiles + 1);
        // one CTA runs on an SM: split the cache where that shortens waves * (tiles a split + the fixed part)
        const long long base = (long long)B * Hkv * p.blocks, fixed = 6;
        long long best = 1, best_cost = -1;
        for (long long s = 1; s <= std::min<long long>(tiles, 64); ++s) {
            const long long tps = (tiles + s - 1) / s;
            if (s > 1 && (tiles + tps - 1) / tps != s) continue;
            const long long cost = (base * s + sms - 1) / sms * (tps + fixed);
            if (best_cost < 0 || cost < best_cost) best = s, best_cost = cost;
        }
        p.W.n_splits = (int)best;
        p.W.tps = (int)((tiles + best - 1) / best);
        p.n_parts = p.W.n_parts = p.W.n_splits * (p.W.dual ? 2 : 1);
    }
    if (p.n_parts > 1) {
        const size_t n = (size_t)total_q * Hq * p.n_parts;
        p.acc_off = (n * 8 + 255) / 256 * 256;
        p.bytes = p.acc_off + n * d * 4;
    }
    if (!p.few && p.blocks >= 3) {
        const int bn = d == 256 ? 64 : 128;
        p.W.tiles = (max_len + bn - 1) / bn;
        const size_t img = (size_t)B * Hkv * p.W.tiles * (4 * bn * d);
        if (img <= kMaxImages) {
            p.expand = true;
            p.img_off = (p.bytes + 255) / 256 * 256;
            p.bytes = p.img_off + img;
        }
    }
    return p;
}

// (the last one of this host thread is kept: a decode loop asks for the same one every call, twice)
static const Plan& make_plan(int d, int Hq, int Hkv, int B, int total_q, int max_q, int max_len, int window) {
    struct Key {
        int v[9];
    };
    thread_local Key last = {};
    thread_local Plan plan = {};
    const Key k = {{d, Hq, Hkv, B, total_q, max_q, max_len, window, device_sm_count()}};
    if (!std::equal(k.v, k.v + 9, last.v)) {
        plan = work_out_plan(d, Hq, Hkv, B, total_q, max_q, max_len, window, k.v[8]);
        last = k;
    }
    return plan;
}

size_t paged_attention_workspace(int d, int Hq, int Hkv, int B, int total_q, int max_q, int max_len, int window) {
    if (B == 0 || total_q == 0) return 0;
    return make_plan(d, Hq, Hkv, B, total_q, max_q, max_len, window).bytes;
}

template <int D>
static cudaError_t launch_combine(const PagedAttnCall& c, const PagedAttnParams& P, int n_parts, const float* ml,
                                  const float* acc) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long long)P.max_q * P.Hq + 3) / 4), P.B);
    cfg.blockDim = dim3(128);
    cfg.stream = c.stream;
    cudaLaunchAttribute attr[1];  // it may start while the kernel before it ends, and waits for it on the device
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto* k = c.dtype == SRFTKV_DTYPE_BF16 ? paged_attn_combine_kernel<D, __nv_bfloat16> : paged_attn_combine_kernel<D, __half>;
    return cudaLaunchKernelEx(&cfg, k, P, n_parts, ml, acc);
}

int paged_attention(const PagedAttnCall& c) {
    PagedAttnParams P = c.P;
    static SymbolCache cache;
    void* f = nullptr;
    if (symbol_address(cache, &g_paged_attn_fault, &f, "the paged attention's fault word")) return SRFTKV_ERR_CUDA;
    P.fault = static_cast<unsigned int*>(f);
    Plan plan = make_plan(c.d, P.Hq, P.Hkv, P.B, P.total_q, P.max_q, P.max_len, P.window);
    float* ml = static_cast<float*>(c.workspace);
    float* acc = reinterpret_cast<float*>(static_cast<char*>(c.workspace) + plan.acc_off);
    int rc;
    if (plan.few) {
        SplitWork& S = plan.S;
        S.bits_k = c.bits_k;
        S.bits_v = c.bits_v;
        S.dtype = c.dtype;
        S.part_ml = ml;
        S.part_acc = acc;
        using Fn = int (*)(const PagedAttnParams&, const SplitWork&, cudaStream_t);
        static const Fn fn[3][3] = {{launch_split64_fp32, launch_split64_fp16, launch_split64_e8m0},
                                    {launch_split128_fp32, launch_split128_fp16, launch_split128_e8m0},
                                    {launch_split256_fp32, launch_split256_fp16, launch_split256_e8m0}};
        rc = fn[c.d == 64 ? 0 : c.d == 128 ? 1 : 2][P.sfmt](P, S, c.stream);
    } else {
        TileWork& W = plan.W;
        W.bits_k = c.bits_k;
        W.bits_v = c.bits_v;
        W.dtype = c.dtype;
        W.part_ml = ml;
        W.part_acc = acc;
        W.images = plan.expand ? static_cast<uint8_t*>(c.workspace) + plan.img_off : nullptr;
        rc = c.d == 64    ? launch_tile64(P, W, plan.blocks, c.stream)
             : c.d == 128 ? launch_tile128(P, W, plan.blocks, c.stream)
                          : launch_tile256(P, W, plan.blocks, c.stream);
    }
    if (rc || plan.n_parts == 1) return rc;
    const cudaError_t e = c.d == 64    ? launch_combine<64>(c, P, plan.n_parts, ml, acc)
                          : c.d == 128 ? launch_combine<128>(c, P, plan.n_parts, ml, acc)
                                       : launch_combine<256>(c, P, plan.n_parts, ml, acc);
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
