// paged_rotate.cuh -- the rotation of one head vector by one warp, for
// d = 64, 128 and 256, and 16-bit rows as a warp loads and stores them.
//
// Lane l holds the E = d/32 consecutive coordinates E l .. E l + E - 1.
// SRFT: with z_n = u_2n + i u_2n+1 (u = s x, N = d/2 points, E/2 of them a
// lane) a decimation-in-frequency FFT, stages of half-size h >= E/2 across
// lanes (shuffles), the rest inside a lane; it leaves Z in bit-reversed order,
// which one pass through shared memory undoes and which also brings Z_{N-k}
// beside Z_k for the real split
//   y_k = (Z_k + conj Z_{N-k})/2 + W_d^k (Z_k - conj Z_{N-k})/2i,
// p_0 = y_0, p_1 = y_N, p_2k = sqrt2 Re y_k, p_2k+1 = sqrt2 Im y_k, all over
// sqrt d.  The inverse runs the same steps backwards.  SRHT: Walsh-Hadamard
// butterflies on the same layout.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "srft_math.cuh"

namespace srftkv {
namespace rot {

template <int D>
struct Dim {
    static_assert(D == 64 || D == 128 || D == 256, "head dimension");
    static constexpr int E = D / 32;  // coordinates a lane
    static constexpr int N = D / 2;   // complex points
    static constexpr int C = E / 2;   // complex points a lane
    static constexpr int LG = D == 64 ? 5 : D == 128 ? 6 : 7;  // log2 N
};

// e^{-2 pi i m / 256}, per-lane indices through the L1-served table
__device__ __forceinline__ float2 twid(int m) { return make_float2(tw_re_lane(m), tw_im_lane(m)); }
// Bring the twiddle table (2 KB) to L1 while something else is waited for: a warp that turns one row meets it cold
__device__ __forceinline__ void prefetch_twiddles(int lane) {
    if (lane < 16) asm volatile("prefetch.global.L1 [%0];" ::"l"(reinterpret_cast<const char*>(&g_tw) + 128 * lane));
}
__device__ __forceinline__ float sx(float v, int m) { return __shfl_xor_sync(0xffffffffu, v, m); }

// Unnormalised DFT of the warp's N complex points (v[2j], v[2j+1] = point C l + j); INV: conjugate
// twiddles.  The result sits in bit-reversed order.
template <int D, bool INV>
__device__ __forceinline__ void fft_dif(float (&v)[Dim<D>::E], int lane) {
    constexpr int N = Dim<D>::N, C = Dim<D>::C;
#pragma unroll
    for (int h = N / 2; h >= 1; h >>= 1) {
        if (h >= C) {
            const int m = h / C;
            const bool up = (lane & m) == 0;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const float pr = sx(v[2 * j], m), pi = sx(v[2 * j + 1], m);
                float2 w = twid(((C * lane + j) & (h - 1)) * (128 / h));
                if (INV) w.y = -w.y;
                const float dr = pr - v[2 * j], di = pi - v[2 * j + 1];
                v[2 * j] = up ? v[2 * j] + pr : dr * w.x - di * w.y;
                v[2 * j + 1] = up ? v[2 * j + 1] + pi : dr * w.y + di * w.x;
            }
        } else {
#pragma unroll
            for (int j = 0; j < C; ++j) {
                if (j & h) continue;
                float2 w = twid((j & (h - 1)) * (128 / h));
                if (INV) w.y = -w.y;
                const float ar = v[2 * j], ai = v[2 * j + 1], br = v[2 * (j + h)], bi = v[2 * (j + h) + 1];
                const float dr = ar - br, di = ai - bi;
                v[2 * j] = ar + br;
                v[2 * j + 1] = ai + bi;
                v[2 * (j + h)] = dr * w.x - di * w.y;
                v[2 * (j + h) + 1] = dr * w.y + di * w.x;
            }
        }
    }
}
// position C l + j of a bit-reversed result -> its index
template <int D>
__device__ __forceinline__ int unreversed(int e) {
    return (int)(__brev((unsigned)e) >> (32 - Dim<D>::LG));
}

// p = R u for the signed row u; sm: N float2 of this warp's shared memory
template <int D>
__device__ __forceinline__ void srft_forward(float (&v)[Dim<D>::E], int lane, float2* sm) {
    constexpr int N = Dim<D>::N, C = Dim<D>::C;
    const float isd = rsqrtf((float)D), c2 = 1.41421356237309505f * isd;
    fft_dif<D, false>(v, lane);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < C; ++j) sm[unreversed<D>(C * lane + j)] = make_float2(v[2 * j], v[2 * j + 1]);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int k = C * lane + j;
        const float2 a = sm[k], b = sm[(N - k) & (N - 1)];
        const float er = 0.5f * (a.x + b.x), ei = 0.5f * (a.y - b.y);
        const float orr = 0.5f * (a.y + b.y), oi = -0.5f * (a.x - b.x);
        const float2 w = twid(k * (256 / D));
        if (k == 0) {
            v[2 * j] = isd * (er + orr);
            v[2 * j + 1] = isd * (er - orr);
        } else {
            v[2 * j] = c2 * (er + (w.x * orr - w.y * oi));
            v[2 * j + 1] = c2 * (ei + (w.x * oi + w.y * orr));
        }
    }
}
// u = R^T p
template <int D>
__device__ __forceinline__ void srft_inverse(float (&v)[Dim<D>::E], int lane, float2* sm) {
    constexpr int N = Dim<D>::N, C = Dim<D>::C;
    const float isd = rsqrtf((float)D), c2 = 1.41421356237309505f * isd;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < C; ++j) sm[C * lane + j] = make_float2(v[2 * j], v[2 * j + 1]);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const int k = C * lane + j;
        const float2 a = sm[k], b = sm[(N - k) & (N - 1)];
        if (k == 0) {  // a = (y_0, y_N): Z_0 = (y_0 + y_N)/2 + i (y_0 - y_N)/2, times 2/sqrt(d)
            v[2 * j] = isd * (a.x + a.y);
            v[2 * j + 1] = isd * (a.x - a.y);
        } else {  // y_k = p / sqrt2: E = (y_k + conj y_{N-k})/2, O = (y_k - conj y_{N-k})/2 conj(W), Z = E + iO
            const float er = 0.5f * (a.x + b.x), ei = 0.5f * (a.y - b.y);
            const float fr = 0.5f * (a.x - b.x), fi = 0.5f * (a.y + b.y);
            const float2 w = twid(k * (256 / D));
            const float orr = fr * w.x + fi * w.y, oi = fi * w.x - fr * w.y;
            v[2 * j] = c2 * (er - oi);
            v[2 * j + 1] = c2 * (ei + orr);
        }
    }
    fft_dif<D, true>(v, lane);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < C; ++j) sm[unreversed<D>(C * lane + j)] = make_float2(v[2 * j], v[2 * j + 1]);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < C; ++j) {
        const float2 a = sm[C * lane + j];
        v[2 * j] = a.x;
        v[2 * j + 1] = a.y;
    }
}
// H u / sqrt(d) (its own inverse)
template <int D>
__device__ __forceinline__ void wht(float (&v)[Dim<D>::E], int lane) {
    constexpr int E = Dim<D>::E;
    const float isd = rsqrtf((float)D);
#pragma unroll
    for (int h = 1; h < E; h <<= 1)
#pragma unroll
        for (int j = 0; j < E; ++j)
            if (!(j & h)) {
                const float x = v[j], y = v[j + h];
                v[j] = x + y;
                v[j + h] = x - y;
            }
#pragma unroll
    for (int m = 1; m < 32; m <<= 1)
#pragma unroll
        for (int j = 0; j < E; ++j) {
            const float o = sx(v[j], m);
            v[j] = (lane & m) ? o - v[j] : v[j] + o;
        }
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] *= isd;
}
// the signs of this lane's coordinates (mask word i: bit 15 for coordinate 2i, bit 31 for 2i + 1)
template <int D>
__device__ __forceinline__ void flip_signs(float (&v)[Dim<D>::E], int lane, const uint32_t* mask) {
#pragma unroll
    for (int j = 0; j < Dim<D>::C; ++j) {
        const uint32_t w = mask[Dim<D>::C * lane + j];
        v[2 * j] = __uint_as_float(__float_as_uint(v[2 * j]) ^ ((w & 0x8000u) << 16));
        v[2 * j + 1] = __uint_as_float(__float_as_uint(v[2 * j + 1]) ^ (w & 0x80000000u));
    }
}
template <int D>
__device__ __forceinline__ void forward(float (&v)[Dim<D>::E], int lane, int transform, const uint32_t* mask, float2* sm) {
    flip_signs<D>(v, lane, mask);
    if (transform == SRFTKV_TRANSFORM_SRHT) wht<D>(v, lane);
    else srft_forward<D>(v, lane, sm);
}
template <int D>
__device__ __forceinline__ void inverse(float (&v)[Dim<D>::E], int lane, int transform, const uint32_t* mask, float2* sm) {
    if (transform == SRFTKV_TRANSFORM_SRHT) wht<D>(v, lane);
    else srft_inverse<D>(v, lane, sm);
    flip_signs<D>(v, lane, mask);
}

// ---- 16-bit rows (T = __half or __nv_bfloat16), 2 E bytes a lane ----
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}
template <int W>
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[W]) {
    if constexpr (W == 4) {
        const uint4 t = __ldg(reinterpret_cast<const uint4*>(p));
        w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
    } else if constexpr (W == 2) {
        const uint2 t = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = t.x, w[1] = t.y;
    } else {
        w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
}
template <int W>
__device__ __forceinline__ void store_words(void* p, const uint32_t (&w)[W]) {
    if constexpr (W == 4) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (W == 2) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
}
template <int D, typename T>
__device__ __forceinline__ void load_row(const T* row, int lane, float (&v)[Dim<D>::E]) {
    uint32_t w[Dim<D>::C];
    load_words<Dim<D>::C>(row + Dim<D>::E * lane, w);
#pragma unroll
    for (int j = 0; j < Dim<D>::C; ++j) {
        const float2 f = unpack2<T>(w[j]);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
    }
}
template <int D, typename T>
__device__ __forceinline__ void store_row(T* row, int lane, const float (&v)[Dim<D>::E]) {
    uint32_t w[Dim<D>::C];
#pragma unroll
    for (int j = 0; j < Dim<D>::C; ++j) w[j] = pack2<T>(v[2 * j], v[2 * j + 1]);
    store_words<Dim<D>::C>(row + Dim<D>::E * lane, w);
}
template <int D>
__device__ __forceinline__ void load_lambda(const float* lam, int lane, float (&l)[Dim<D>::E]) {
    if constexpr (Dim<D>::E == 2) {
        const float2 a = __ldg(reinterpret_cast<const float2*>(lam) + lane);
        l[0] = a.x, l[1] = a.y;
    } else {
#pragma unroll
        for (int j = 0; j < Dim<D>::E / 4; ++j) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(lam) + (Dim<D>::E / 4) * lane + j);
            l[4 * j] = a.x, l[4 * j + 1] = a.y, l[4 * j + 2] = a.z, l[4 * j + 3] = a.w;
        }
    }
}

// This lane's E codes of a packed row, as floats (bits 4 or 8; E codes are E*bits/8 bytes: 1 to 8)
template <int D, int BITS>
__device__ __forceinline__ void load_codes(const uint8_t* crow, int lane, float (&v)[Dim<D>::E]) {
    constexpr int E = Dim<D>::E, BY = E * BITS / 8;
    uint32_t w[BY > 4 ? 2 : 1];
    const uint8_t* p = crow + BY * lane;
    if constexpr (BY == 8) load_words<2>(p, w);
    else if constexpr (BY == 4) load_words<1>(p, w);
    else if constexpr (BY == 2) w[0] = __ldg(reinterpret_cast<const unsigned short*>(p));
    else w[0] = __ldg(p);
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const int sh = (i * BITS) & 31;
        v[i] = (float)((int)(w[i * BITS / 32] << (32 - BITS - sh)) >> (32 - BITS));
    }
}

}  // namespace rot
}  // namespace srftkv
