// paged_codec.cu -- srft_kv_quantize_paged and srft_kv_dequantize_paged: rows
// of K and V encoded into, and decoded from, the slots of a page pool.
//
// Per row x of head h and token t with slot s: p = R diag(sign) x, z = lambda p,
// per group scale = max|z| / Q in the side's format, codes = rint(z / scale),
// stored in row s % page_size of page s / page_size; and back,
// x = diag(sign) R^T ((codes * scale) / lambda).  Scales and rounding are
// group_scale's and the magic-number FMA's of the contiguous codec, so a page
// holds the bytes the contiguous call would store for the same z.
//
// One warp a row (paged_rotate.cuh) here; many rows on the tensor cores (paged_codec_tc.cuh).
#include "codec_impl.cuh"
#include "paged.h"
#include "paged_rotate.cuh"

namespace srftkv {

static __device__ unsigned int g_paged_codec_fault;

namespace {
constexpr int PW = 4;  // rows (warps) a block
}

// The packed row of (token, head): page (s >> lg_page), row s & (page_size - 1); -1: no row
__device__ __forceinline__ long long paged_row(const PagedCodecParams& P, long long slot, int h) {
    return ((slot >> P.lg_page) * P.H + h) << P.lg_page | (slot & ((1ll << P.lg_page) - 1));
}

// Work item r of a launch: (side, token, head), head fastest.  False: nothing to do (padding, a bad slot).
struct PagedItem {
    int side, t, h;
    long long row;
};
__device__ __forceinline__ bool paged_item(const PagedCodecParams& P, long long r, int lane, PagedItem& it) {
    const long long per = (long long)P.n_tokens * P.H;
    if (r >= per * P.n_sides) return false;
    it.side = r >= per;
    const long long u = r - (it.side ? per : 0);
    it.t = (int)(u / P.H);
    it.h = (int)(u - (long long)it.t * P.H);
    const long long slot = __ldg(P.slots + it.t);
    if (slot < 0) return false;
    if (slot >= P.n_slots) {
        if (lane == 0) atomicOr(P.fault, kFaultSlot);
        return false;
    }
    it.row = paged_row(P, slot, it.h);
    return true;
}

// Codes and scales of one rotated row held E coordinates a lane
template <int D, int BITS, int SF>
__device__ __forceinline__ void store_packed(const float (&z)[D / 32], int lane, int group, int lg_group,
                                             uint8_t* crow, uint8_t* srow) {
    constexpr int E = D / 32;
    constexpr float Q = BITS == 4 ? 7.f : 127.f, MAG = kMagic + (BITS == 4 ? 8.f : 128.f);
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) a = fmaxf(a, fabsf(z[i]));
    const int gl = group / E;  // lanes a group
    for (int m = 1; m < gl; m <<= 1) a = fmaxf(a, rot::sx(a, m));
    float sc, inv;
    uint32_t raw;
    group_scale<BITS, SF>(a, sc, raw, inv);
    uint32_t w[E * BITS > 32 ? 2 : 1] = {};
#pragma unroll
    for (int i = 0; i < E; ++i) {
        float m = fmaf(z[i], inv, MAG);
        if (SF == SRFTKV_SCALE_FP16 && a > 65504.f * Q) m = fminf(fmaxf(m, MAG - Q), MAG + Q);  // a saturated scale
        const uint32_t c = (__float_as_uint(m) ^ (BITS == 4 ? 8u : 128u)) & ((1u << BITS) - 1u);
        w[i * BITS / 32] |= c << ((i * BITS) & 31);
    }
    uint8_t* p = crow + E * BITS / 8 * lane;
    if constexpr (E * BITS == 64) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (E * BITS == 32) *reinterpret_cast<uint32_t*>(p) = w[0];
    else if constexpr (E * BITS == 16) *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    else *p = (uint8_t)w[0];
    if ((lane & (gl - 1)) == 0) {
        const int j = (E * lane) >> lg_group;
        if constexpr (SF == SRFTKV_SCALE_FP32) reinterpret_cast<float*>(srow)[j] = sc;
        else if constexpr (SF == SRFTKV_SCALE_FP16) reinterpret_cast<uint16_t*>(srow)[j] = (uint16_t)raw;
        else srow[j] = (uint8_t)raw;
    }
}

template <int D, typename T>
__global__ void __launch_bounds__(PW * 32) paged_quantize_warp_kernel(const __grid_constant__ PagedCodecParams P) {
    constexpr int E = D / 32;
    __shared__ float2 sm[PW][D / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    PagedItem it;
    if (!paged_item(P, (long long)blockIdx.x * PW + warp, lane, it)) return;
    const PagedSideK& S = P.side[it.side];
    float v[E];
    rot::load_row<D, T>(static_cast<const T*>(S.x) + it.t * S.x_stride + (long long)it.h * D, lane, v);
    rot::forward<D>(v, lane, S.transform, P.sign_mask, sm[warp]);
    if (S.lambda != nullptr) {
        float l[E];
        rot::load_lambda<D>(S.lambda + (long long)it.h * D, lane, l);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] *= l[i];
    }
    uint8_t* crow = S.codes + it.row * (D * S.bits / 8);
    const int ng = D >> P.lg_group;
    uint8_t* srow = S.scales + it.row * ng * (S.sfmt == SRFTKV_SCALE_FP32 ? 4 : S.sfmt == SRFTKV_SCALE_FP16 ? 2 : 1);
    auto put = [&](auto sf) {
        constexpr int SF = decltype(sf)::value;
        if (S.bits == 4) store_packed<D, 4, SF>(v, lane, P.group, P.lg_group, crow, srow);
        else store_packed<D, 8, SF>(v, lane, P.group, P.lg_group, crow, srow);
    };
    if (S.sfmt == SRFTKV_SCALE_FP32) put(std::integral_constant<int, SRFTKV_SCALE_FP32>{});
    else if (S.sfmt == SRFTKV_SCALE_FP16) put(std::integral_constant<int, SRFTKV_SCALE_FP16>{});
    else put(std::integral_constant<int, SRFTKV_SCALE_E8M0>{});
}

template <int D, typename T>
__global__ void __launch_bounds__(PW * 32) paged_dequantize_warp_kernel(const __grid_constant__ PagedCodecParams P) {
    constexpr int E = D / 32;
    __shared__ float2 sm[PW][D / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    PagedItem it;
    if (!paged_item(P, (long long)blockIdx.x * PW + warp, lane, it)) return;
    const PagedSideK& S = P.side[it.side];
    const int ng = D >> P.lg_group;
    const uint8_t* crow = S.codes + it.row * (D * S.bits / 8);
    const uint8_t* srow = S.scales + it.row * ng * (S.sfmt == SRFTKV_SCALE_FP32 ? 4 : S.sfmt == SRFTKV_SCALE_FP16 ? 2 : 1);
    float v[E];
    const float sc = load_scale(srow, (E * lane) >> P.lg_group, S.sfmt);
    if (S.bits == 4) rot::load_codes<D, 4>(crow, lane, v);
    else rot::load_codes<D, 8>(crow, lane, v);
    if (S.lambda != nullptr) {
        float l[E];
        rot::load_lambda<D>(S.lambda + (long long)it.h * D, lane, l);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = __fdiv_rn(v[i] * sc, l[i]);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] *= sc;
    }
    rot::inverse<D>(v, lane, S.transform, P.sign_mask, sm[warp]);
    rot::store_row<D, T>(static_cast<T*>(S.x) + it.t * S.x_stride + (long long)it.h * D, lane, v);
}

template <int D, typename T>
static int launch_warp(const PagedCodecParams& P, cudaStream_t stream, bool quantize) {
    const long long rows = (long long)P.n_tokens * P.H * P.n_sides;
    const unsigned blocks = (unsigned)((rows + PW - 1) / PW);
    if (quantize) paged_quantize_warp_kernel<D, T><<<blocks, PW * 32, 0, stream>>>(P);
    else paged_dequantize_warp_kernel<D, T><<<blocks, PW * 32, 0, stream>>>(P);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) {
        set_error("paged codec launch failed: %s", cudaGetErrorString(e));
        return SRFTKV_ERR_CUDA;
    }
    return SRFTKV_OK;
}
template <int D>
static int launch_d(const PagedCodecParams& P, int dtype, cudaStream_t stream, bool quantize) {
    return dtype == SRFTKV_DTYPE_BF16 ? launch_warp<D, __nv_bfloat16>(P, stream, quantize)
                                      : launch_warp<D, __half>(P, stream, quantize);
}

static int launch(const PagedCodecCall& c, bool quantize) {
    PagedCodecParams P = c.P;
    static SymbolCache cache;
    void* f = nullptr;
    if (symbol_address(cache, &g_paged_codec_fault, &f, "the paged codec's fault word")) return SRFTKV_ERR_CUDA;
    P.fault = static_cast<unsigned int*>(f);
    const FastDiv div = make_fastdiv((uint32_t)P.H);
    P.div_mul = div.mul;
    P.div_shift = div.shift;
    // Many rows: the tensor cores, which every CTA first builds R_s for (10 us a call at d = 128, 6 at 64, 19 to 30 at
    // 256); few: one warp a row (d = 128: 8.8 us at 8192 rows, 14.3 at 16384 against 10 here; d = 64: 5.9 and 9.4 against
    // 5.6; d = 256: 20 and 36 at 16384 and 32768, against 25 at both written and 34 read back).  The write's epilogue
    // holds 32 columns a thread, so its groups end there; both sides rotate with one R_s.
    const long long rows = (long long)P.n_tokens * P.H * P.n_sides;
    const bool one_r = P.n_sides == 1 || P.side[0].transform == P.side[1].transform;
    if (rows >= (c.d < 256 ? 10240 : quantize ? 20480 : 28672) && one_r && (!quantize || P.group <= 32)) {
        if (c.d == 64) return launch_paged_codec_tc64(P, c.dtype, quantize, c.stream);
        if (c.d == 128) return launch_paged_codec_tc128(P, c.dtype, quantize, c.stream);
        return launch_paged_codec_tc256(P, c.dtype, quantize, c.stream);
    }
    if (c.d == 64) return launch_d<64>(P, c.dtype, c.stream, quantize);
    if (c.d == 128) return launch_d<128>(P, c.dtype, c.stream, quantize);
    return launch_d<256>(P, c.dtype, c.stream, quantize);
}
int paged_quantize(const PagedCodecCall& c) { return launch(c, true); }
int paged_dequantize(const PagedCodecCall& c) { return launch(c, false); }

unsigned int paged_codec_take_fault() {
    unsigned int v = 0, z = 0;
    cudaMemcpyFromSymbol(&v, g_paged_codec_fault, sizeof(v));
    if (v) cudaMemcpyToSymbol(g_paged_codec_fault, &z, sizeof(z));
    return v;
}

}  // namespace srftkv
