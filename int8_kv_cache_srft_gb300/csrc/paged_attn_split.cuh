// paged_attn_split.cuh -- attention of a few query rows over the paged cache:
// one token (or a few) a sequence, where the bytes of the cache are the cost.
// (Two row groups a CTA at d <= 128: three CTAs an SM with a few spills took 223 us
// where two without took 264, at 20 rows over 8 sequences of 9 k to 32 k tokens.)
//
// Grid (splits, sequence and kv head, row groups).  A CTA's 4 NR query rows
// (query tokens times the heads of its kv head) share every byte it reads.
// Each of its four warps streams every fourth chunk of CH tokens of the split
// into its own ring of NS shared-memory stages and keeps its own online softmax;
// the warps meet in shared memory at the end.  The copies are 16 bytes a lane
// (cp.async): every lane finds its own page, rows past the end and pages that do
// not exist arrive as zeros, and a chunk costs about 30 instructions.  TMA boxes
// of 16 to 32 rows cost twice that in address and barrier work of one lane while
// the others waited (515 against 447 us at 16 x 131072 tokens, d = 128, int4, fp16
// scales), and one producer lane for four warps could not keep up (680 us).
// Measured there: 6.0 TB/s with fp16 scales, 6.4 with fp32 (88 and 95 % of the
// copy rate), 273 warp instructions a 16-token tile, issue slots 56 % busy; two
// stages and four CTAs an SM 469 us, two and three 456, four and two 508.
//
//   S = codes_K . q~  with mma.sync m16n8k16: codes as exact fp16 (offset-binary
//       subnormals, attn_frag.cuh), 16 tokens a tile; columns 2c, 2c+1 carry
//       row c's two 16-dim groups of a 32-dim chunk (8-bit keys: column 2c
//       alone), so the group scale multiplies the fp32 partial, K rounded
//       nowhere.
//   acc += codes_V^T . (p scale_V), the offset taken out by a second
//       contraction of the same operand with the constant -8 (-128), so the
//       accumulators never hold more than a tile's worth of it.
//
// The cache is read as it is and never turned back: q is rotated here (one warp
// a row, while the first chunks are on their way), the sum on the way out.
// What bounds it: the bytes of the cache at 4-bit codes; the logic ops that
// turn codes into operands are next.
//
// Roundings: q~ to fp16 (with one row group at d <= 128 as hi + lo, about 22
// bits); p scale_V to fp16 (with fp16 scales p is rounded before the product
// too).  p is at most 2^2 beside 4-bit and 2^6 beside 8-bit codes: code * scale
// below 65504 keeps p scale_V finite, and small scales above fp16's subnormals.
#pragma once

#include <type_traits>

#include "attn_frag.cuh"
#include "paged.h"
#include "paged_rotate.cuh"
#include "ptx.cuh"

namespace srftkv {

namespace split {

constexpr int WARPS = 4;

template <int SF>
constexpr int sbytes() { return SF == SRFTKV_SCALE_FP32 ? 4 : SF == SRFTKV_SCALE_FP16 ? 2 : 1; }
constexpr int up(int v, int a) { return (v + a - 1) / a * a; }

// A plane of code rows in shared memory: rows of up to 128 bytes whose 16-byte pieces are XORed with their 128-byte
// line (ldmatrix then reads without bank conflicts); 256-byte rows as two 128-byte halves one after the other
template <int RB, int CH>
struct Plane {
    static constexpr int R = RB < 128 ? RB : 128, HALVES = RB / R, BYTES = CH * RB;
    static __device__ __forceinline__ int swz(int r) { return ((r * R) >> 7) & (R / 16 - 1); }
};
template <int D, int BK, int BV, int SF>
struct Cfg {
    static constexpr int RK = D * BK / 8, RV = D * BV / 8, SR = D / 16 * sbytes<SF>();  // row bytes (scales: at most)
    static constexpr int CH = 32 * (RK + RV + 2 * SR) <= 9216 ? 32 : 16;                // tokens a chunk
    static constexpr int OFF_V = up(CH * RK, 1024), OFF_KS = OFF_V + up(CH * RV, 1024);
    static constexpr int OFF_VS = OFF_KS + up(CH * SR, 128);
    static constexpr int STAGE = up(OFF_VS + CH * SR, 1024);
    static constexpr int NS = WARPS * 3 * STAGE <= 70 * 1024 ? 3 : 2;                       // stages a warp
};
template <int D, int BK, int BV, int SF, int NR, bool LO>
struct Smem {
    using C = Cfg<D, BK, BV, SF>;
    static constexpr int ROWS = 4 * NR;
    static constexpr int RING = WARPS * C::NS * C::STAGE;
    static constexpr int MERGE = WARPS * ROWS * (D + 2) * 4;      // over the ring, at the end
    static constexpr int BODY = up(RING > MERGE ? RING : MERGE, 16);
    static constexpr int OFF_Q = BODY;                            // q~ rows
    static constexpr int OFF_QL = OFF_Q + ROWS * D * 4;           // the low halves of q~'s fragments (LO)
    static constexpr int OFF_ROT = OFF_QL + (LO ? D / 32 * 512 : 0);  // a warp's rotation scratch
    static constexpr int OFF_END = OFF_ROT + WARPS * D * 4;
    static constexpr int BYTES = OFF_END + 1024;
};

// scale f (16-dim unit) of staged row r, rows of D/16 scales
template <int D, int SF>
__device__ __forceinline__ float scale_at(const uint8_t* s, int r, int f) {
    const int i = r * (D / 16) + f;
    if constexpr (SF == SRFTKV_SCALE_FP32) return reinterpret_cast<const float*>(s)[i];
    else if constexpr (SF == SRFTKV_SCALE_FP16) return __half2float(reinterpret_cast<const __half*>(s)[i]);
    else return __uint_as_float((uint32_t)s[i] << 23);
}
// scales of units 4p .. 4p+3 of staged row r
template <int D, int SF>
__device__ __forceinline__ void scales4(const uint8_t* s, int r, int p, float (&v)[4]) {
    const int i = r * (D / 16) + 4 * p;
    if constexpr (SF == SRFTKV_SCALE_FP32) {
        const float4 f = *reinterpret_cast<const float4*>(s + i * 4);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else if constexpr (SF == SRFTKV_SCALE_FP16) {
        const uint2 w = *reinterpret_cast<const uint2*>(s + i * 2);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&w.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&w.y));
        v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(s + i);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = __uint_as_float(((w >> (8 * k)) & 0xFFu) << 23);
    }
}
// Groups wider than 16: spread the staged rows of D >> lg scales to rows of D/16 in place (lane r takes row r), so
// the tiles are read with constant offsets whatever the group
template <int D, int SF>
__device__ __forceinline__ void spread_scales(uint8_t* s, int rows, int lg, int lane) {
    using U = typename std::conditional<SF == SRFTKV_SCALE_FP32, uint32_t,
                                        typename std::conditional<SF == SRFTKV_SCALE_FP16, uint16_t, uint8_t>::type>::type;
    U* v = reinterpret_cast<U*>(s);
    U t[D / 16];
    if (lane < rows) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) t[i] = v[lane * (D >> lg) + ((16 * i) >> lg)];
    }
    __syncwarp();
    if (lane < rows) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) v[lane * (D / 16) + i] = t[i];
    }
}
// (w & mask) ^ flip as one logic op: the mask comes in a register the compiler cannot see through (two immediates
// would take two)
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
    uint32_t r;
    asm volatile("mov.u32 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float opaque(float v) {
    float r;
    asm volatile("mov.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
template <uint32_t FLIP>
__device__ __forceinline__ uint32_t pick(uint32_t w, uint32_t mask) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(w), "r"(mask), "n"(FLIP));  // (a & b) ^ c
    return r;
}
__device__ __forceinline__ uint32_t h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// 16 bytes to shared memory, the first n of them from global memory and zeros behind them
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// D = A . B, m16n8k16
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// D = A . B + (c[0] .. c[3]), m16n8k16
__device__ __forceinline__ void mma16816_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1, const float* c) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

}  // namespace split

template <int D, int BK, int BV, int SF, int NR, bool LO>
__global__ void __launch_bounds__(128, D == 256 ? 2 : 3)
    paged_attn_split_kernel(const __grid_constant__ PagedAttnParams P, const __grid_constant__ SplitWork W) {
    using C = split::Cfg<D, BK, BV, SF>;
    using M = split::Smem<D, BK, BV, SF, NR, LO>;
    using PK = split::Plane<C::RK, C::CH>;
    using PV = split::Plane<C::RV, C::CH>;
    constexpr int CH = C::CH, NT = CH / 16, NS = C::NS, NP = D / 64, E = D / 32;
    constexpr float PBITS = BV == 4 ? 2.f : 6.f;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;

    // ---- rows and chunks of this CTA ----
    const int b = blockIdx.y / P.Hkv, h = blockIdx.y - b * P.Hkv, spl = blockIdx.x;
    const int q0 = P.cu_q ? P.cu_q[b] : b;
    int m_tok = min(P.cu_q ? P.cu_q[b + 1] - q0 : 1, P.max_q);
    if (q0 < 0) m_tok = 0;
    m_tok = min(m_tok, P.total_q - q0);
    const int row0 = blockIdx.z * M::ROWS, n_rows = min(m_tok * P.rep - row0, M::ROWS);
    if (n_rows <= 0) return;
    const int len = min(max(P.seq_lens[b], 0), P.max_len);
    const int pos_lo = len - m_tok + row0 / P.rep, pos_hi = len - m_tok + (row0 + n_rows - 1) / P.rep;
    auto row_at = [&](int r) -> long long {  // row r of the group in [total_q * Hq]
        const int i = (row0 + r) / P.rep;
        return (long long)(q0 + i) * P.Hq + h * P.rep + (row0 + r - i * P.rep);
    };
    auto row_ptr = [&](const void* base, long long stride, int r) -> long long {  // element offset of row r of q / out
        const int i = (row0 + r) / P.rep;
        return (q0 + i) * stride + (long long)(h * P.rep + (row0 + r - i * P.rep)) * D;
    };
    const int low_all = P.window ? max(0, pos_lo - P.window + 1) : 0;  // the first token any row sees
    const int first_chunk = low_all / CH;
    const int c_begin = first_chunk + spl * W.chunks;
    const int c_end = min(pos_hi >= 0 ? pos_hi / CH + 1 : 0, c_begin + W.chunks);
    if (c_begin >= c_end) {  // nothing visible here: zeros, or empty partials
        for (int r = threadIdx.x; r < n_rows; r += blockDim.x) {
            if (W.n_parts == 1) {
                uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.out) + row_ptr(P.out, P.out_stride, r));
                for (int k = 0; k < D / 8; ++k) o[k] = make_uint4(0, 0, 0, 0);
            } else {
                float* ml = W.part_ml + (row_at(r) * W.n_parts + spl) * 2;
                ml[0] = -INFINITY;
                ml[1] = 0.f;
            }
        }
        griddep_launch_dependents();
        return;
    }

    // ---- copies of a chunk into a stage of this warp's ring, 16 bytes a lane and step ----
    uint8_t* ring = smem + warp * NS * C::STAGE;
    const int srb = (D >> P.lg_group) * split::sbytes<SF>();  // staged scale row as it lies in the page
    const int* table = P.table + (long long)b * P.max_pages;
    int pages[NT];  // of the next chunk to load, looked up a chunk ahead
    auto look_up = [&](int chunk) {
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            const int t = chunk * CH + 16 * x;
            pages[x] = chunk < c_end && t < len ? __ldg(table + (t >> P.lg_page)) : 0;
        }
    };
    auto load = [&](int chunk, int s) {
        if (chunk < c_end) {
            const uint32_t st = ptx::smem_u32(ring + s * C::STAGE);
            const int t0 = chunk * CH;
            long long row[NT];  // packed row of token 16 x of the chunk
            int have[NT];       // tokens of the 16 that are there
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                const bool seen = t0 + 16 * x + 15 >= low_all;  // (pages before every window may be gone)
                const bool ok = seen && (unsigned)pages[x] < (unsigned)P.n_pages;
                have[x] = ok ? len - t0 - 16 * x : 0;
                if (seen && !ok) atomicOr(P.fault, kFaultPage);
                row[x] = ok ? (long long)(pages[x] * P.Hkv + h) << P.lg_page | ((t0 + 16 * x) & ((1 << P.lg_page) - 1)) : 0;
            }
            auto codes = [&](const uint8_t* plane, uint32_t dst, auto pl, auto rbc) {
                using PL = decltype(pl);
                constexpr int RB = decltype(rbc)::value, LPR = RB / 16, RPI = 32 / LPR, PER = PL::R / 16;
                const int lr = lane / LPR, col = lane % LPR;
#pragma unroll
                for (int i = 0; i < CH / RPI; ++i) {
                    const int x = i * RPI / 16, r = i * RPI + lr;
                    split::copy16(dst + (col / PER) * (CH * 128) + r * PL::R + (((col % PER) ^ PL::swz(r)) << 4),
                                  plane + (row[x] + (r & 15)) * RB + col * 16, (r & 15) < have[x] ? 16 : 0);
                }
            };
            codes(P.kc, st, PK{}, std::integral_constant<int, C::RK>{});
            codes(P.vc, st + C::OFF_V, PV{}, std::integral_constant<int, C::RV>{});
            // scales: the 16 rows of a half lie one after the other, 16 srb bytes
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int j = 0; j < (C::SR + 31) / 32; ++j) {
                    const int at = (32 * j + lane) * 16;  // byte of the half's scales
                    if (at < 16 * srb) {
                        const int n = min(max(have[x] * srb - at, 0), 16);
                        split::copy16(st + C::OFF_KS + 16 * x * srb + at, P.ks + row[x] * srb + (n ? at : 0), n);
                        split::copy16(st + C::OFF_VS + 16 * x * srb + at, P.vs + row[x] * srb + (n ? at : 0), n);
                    }
                }
            look_up(chunk + split::WARPS);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if (warp == 0) rot::prefetch_twiddles(lane);
    look_up(c_begin + warp);
#pragma unroll
    for (int j = 0; j < NS - 1; ++j) load(c_begin + warp + j * split::WARPS, j);

    // ---- q~ = R q sm_scale log2 e / lambda_K, one warp a row ----
    float* qs = reinterpret_cast<float*>(smem + M::OFF_Q);
    float2* scratch = reinterpret_cast<float2*>(smem + M::OFF_ROT) + warp * (D / 2);
#pragma unroll 1
    for (int r = warp; r < M::ROWS; r += split::WARPS) {
        float v[E] = {};
        if (r < n_rows) {
            const uint16_t* src = static_cast<const uint16_t*>(P.q) + row_ptr(P.q, P.q_stride, r);
            if (W.dtype == SRFTKV_DTYPE_BF16) rot::load_row<D>(reinterpret_cast<const __nv_bfloat16*>(src), lane, v);
            else rot::load_row<D>(reinterpret_cast<const __half*>(src), lane, v);
            rot::forward<D>(v, lane, P.tr_k, P.sign_mask, scratch);
#pragma unroll
            for (int j = 0; j < E; ++j) v[j] *= P.qscale;
            if (P.lam_k) {
                float l[E];
                rot::load_lambda<D>(P.lam_k + (long long)h * D, lane, l);
#pragma unroll
                for (int j = 0; j < E; ++j) v[j] = __fdiv_rn(v[j], l[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < E; ++j) qs[r * D + E * lane + j] = v[j];
    }
    __syncthreads();

    // ---- K-side B fragments: column g = (row g/2, half g%2); nb: minus the code offset times the column sum, for
    // this thread's columns 2c, 2c+1: the accumulators' start where registers allow to keep whole ones (QUAD; built
    // anew they cost four moves a tile and chunk), else added times the scale ----
    constexpr bool QUAD = BK == 4 && NR == 1 && !LO && D <= 128;  // nb kept as whole accumulator starts
    constexpr int NB = QUAD ? D / 8 : D / 16;
    uint32_t qh[NR][D / 8];
    uint4* qlo = reinterpret_cast<uint4*>(smem + M::OFF_QL);  // [D/32][lane]: every warp's are the same
    float nb[NR][NB];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
        const float* q = qs + (4 * nr + (g >> 1)) * D;
        if constexpr (BK == 4) {
            const float on = (c >> 1) == (g & 1) ? 1.f : 0.f;
#pragma unroll
            for (int mm = 0; mm < D / 32; ++mm) {
                // thread c: dims 8c .. 8c+7 of the chunk; pairs (j, j+4), the high-nibble rows with q / 16
                const float4 a = *reinterpret_cast<const float4*>(q + 32 * mm + 8 * c);
                const float4 e = *reinterpret_cast<const float4*>(q + 32 * mm + 8 * c + 4);
                const float x[4] = {a.x * on, a.y * on, a.z * on, a.w * on}, y[4] = {e.x * on, e.y * on, e.z * on, e.w * on};
                float part = 0.f;
                uint32_t ql[4] = {};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float u = (j & 1) ? 0.0625f : 1.f;
                    if constexpr (LO) {
                        split_h2(x[j] * u, y[j] * u, qh[nr][4 * mm + j], ql[j]);
                        part += (h2_sum(qh[nr][4 * mm + j]) + h2_sum(ql[j])) * ((j & 1) ? 16.f : 1.f);
                    } else {
                        qh[nr][4 * mm + j] = split::h2(x[j] * u, y[j] * u);
                        part += h2_sum(qh[nr][4 * mm + j]) * ((j & 1) ? 16.f : 1.f);
                    }
                }
                if (LO && warp == 0) qlo[mm * 32 + lane] = make_uint4(ql[0], ql[1], ql[2], ql[3]);
                part += __shfl_xor_sync(0xffffffffu, part, 1);
                part += __shfl_xor_sync(0xffffffffu, part, 2);
                const float n0 = (-8.f / kSub) * __shfl_sync(0xffffffffu, part, 8 * c);
                const float n1 = (-8.f / kSub) * __shfl_sync(0xffffffffu, part, 8 * c + 4);
                if constexpr (QUAD) {
                    nb[nr][4 * mm] = split::opaque(n0), nb[nr][4 * mm + 1] = split::opaque(n1);
                    nb[nr][4 * mm + 2] = split::opaque(n0), nb[nr][4 * mm + 3] = split::opaque(n1);
                } else {
                    nb[nr][2 * mm] = n0, nb[nr][2 * mm + 1] = n1;
                }
            }
        } else {
            const float on = (g & 1) ? 0.f : 1.f;
#pragma unroll
            for (int mm = 0; mm < D / 16; ++mm) {  // thread c: dims 4c .. 4c+3; pairs (j, j+2)
                const float4 a = *reinterpret_cast<const float4*>(q + 16 * mm + 4 * c);
                float part;
                if constexpr (LO) {
                    uint32_t l0, l1;
                    split_h2(a.x * on, a.z * on, qh[nr][2 * mm], l0);
                    split_h2(a.y * on, a.w * on, qh[nr][2 * mm + 1], l1);
                    if (warp == 0) reinterpret_cast<uint2*>(qlo + (mm >> 1) * 32 + lane)[mm & 1] = make_uint2(l0, l1);
                    part = h2_sum(qh[nr][2 * mm]) + h2_sum(l0) + h2_sum(qh[nr][2 * mm + 1]) + h2_sum(l1);
                } else {
                    qh[nr][2 * mm] = split::h2(a.x * on, a.z * on);
                    qh[nr][2 * mm + 1] = split::h2(a.y * on, a.w * on);
                    part = h2_sum(qh[nr][2 * mm]) + h2_sum(qh[nr][2 * mm + 1]);
                }
                part += __shfl_xor_sync(0xffffffffu, part, 1);
                part += __shfl_xor_sync(0xffffffffu, part, 2);
                nb[nr][mm] = (-128.f / kSub) * __shfl_sync(0xffffffffu, part, 8 * c);
            }
        }
    }

    if constexpr (LO) __syncthreads();  // qlo

    float acc[NR][D / 4], mx[NR], l[NR];
    int pos[NR], low[NR];  // row c of each group: the last and first position it sees
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
        for (int i = 0; i < D / 4; ++i) acc[nr][i] = 0.f;
        mx[nr] = -INFINITY;
        l[nr] = 0.f;
        const int r = 4 * nr + c;
        pos[nr] = r < n_rows ? len - m_tok + (row0 + r) / P.rep : -1;  // rows past the last see nothing
        low[nr] = P.window ? pos[nr] - P.window + 1 : 0;
    }
    // per-lane ldmatrix rows: 8-row groups (0-7 | 8-15) x (chunk | chunk + 1)
    const int rl = (lane & 7) + ((lane >> 3) & 1) * 8, dl = lane >> 4;
    const uint32_t ko = rl * PK::R, kx = (uint32_t)(dl ^ PK::swz(rl)) << 4;
    const uint32_t vo = rl * PV::R, vx = (uint32_t)(dl ^ PV::swz(rl)) << 4;
    auto plane_at = [](uint32_t base, uint32_t off, uint32_t x16, int R, int tr, int seg) -> uint32_t {
        const int per = R / 16;  // 16-byte chunks a (half) row
        return base + (seg / per) * (CH * 128) + off + tr * R + (((uint32_t)(seg % per) << 4) ^ x16);
    };

    // codes -> offset-binary fp16 subnormals (attn_frag.cuh)
    const uint32_t m_lo = split::opaque(0x000F000Fu), m_hi = split::opaque(0x00F000F0u), m_by = split::opaque(0x00FF00FFu);
    // the V side's offset as an A operand: -8 in the units of low (2^-24) and high (2^-20) nibbles, or -128 of bytes;
    // four registers kept as they are (as immediates they were moved into place before every use)
    const uint32_t off0 = split::opaque(BV == 4 ? 0x80088008u : 0x80808080u), off1 = split::opaque(0x80808080u);
    const uint32_t off2 = split::opaque(BV == 4 ? 0x80088008u : 0x80808080u), off3 = split::opaque(0x80808080u);
    auto lo4 = [&](uint32_t w) { return split::pick<0x00080008u>(w, m_lo); };
    auto hi4 = [&](uint32_t w) { return split::pick<0x00800080u>(w, m_hi); };
    auto by8 = [&](uint32_t w) { return split::pick<0x00800080u>(w, m_by); };

    int it = 0;
    for (int chunk = c_begin + warp; chunk < c_end; chunk += split::WARPS, ++it) {
        const int s = it % NS;
        asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
        __syncwarp();  // the chunk is there for every lane, and the stage before it is free
        load(chunk + (NS - 1) * split::WARPS, (it + NS - 1) % NS);
        uint8_t* st = ring + s * C::STAGE;
        const uint32_t kb = ptx::smem_u32(st), vb = ptx::smem_u32(st + C::OFF_V);
        uint8_t *ks = st + C::OFF_KS, *vs = st + C::OFF_VS;
        const int t0 = chunk * CH;
        if (P.lg_group != 4) {
            split::spread_scales<D, SF>(ks, CH, P.lg_group, lane);
            split::spread_scales<D, SF>(vs, CH, P.lg_group, lane);
            __syncwarp();
        }
        // ---- scores: sc[nr][st][r] of row c, token 16 st + g + 8 r, in units of 2^-24 ----
        float sc[NR][NT][2];
#pragma unroll
        for (int tt = 0; tt < NT; ++tt) {
            const int tr = 16 * tt;
            float2 a0[NR], a1[NR];
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) a0[nr] = a1[nr] = make_float2(0.f, 0.f);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                float s0[4], s1[4];
                split::scales4<D, SF>(ks, tr + g, p, s0);
                split::scales4<D, SF>(ks, tr + g + 8, p, s1);
                if constexpr (BK == 4) {
                    uint32_t r[4];
                    ldsm_x4(plane_at(kb, ko, kx, PK::R, tr, 2 * p), r);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int mm = 2 * p + e;
                        const uint32_t rg = r[2 * e], r8 = r[2 * e + 1], rs = rg >> 8, rs8 = r8 >> 8;
                        const uint32_t x0 = lo4(rg), x1 = lo4(r8), x2 = hi4(rg), x3 = hi4(r8);
                        const uint32_t y0 = lo4(rs), y1 = lo4(rs8), y2 = hi4(rs), y3 = hi4(rs8);
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr) {
                            float d[4];
                            if constexpr (QUAD)
                                split::mma16816_from(d, x0, x1, x2, x3, qh[nr][4 * mm], qh[nr][4 * mm + 1], &nb[nr][4 * mm]);
                            else
                                split::mma16816_zero(d, x0, x1, x2, x3, qh[nr][4 * mm], qh[nr][4 * mm + 1]);
                            mma16816(d, y0, y1, y2, y3, qh[nr][4 * mm + 2], qh[nr][4 * mm + 3]);
                            if constexpr (LO) {
                                const uint4 q4 = qlo[mm * 32 + lane];
                                mma16816(d, x0, x1, x2, x3, q4.x, q4.y);
                                mma16816(d, y0, y1, y2, y3, q4.z, q4.w);
                            }
                            a0[nr] = fma2(s0[2 * e], s0[2 * e + 1], d[0], d[1], a0[nr]);
                            a1[nr] = fma2(s1[2 * e], s1[2 * e + 1], d[2], d[3], a1[nr]);
                            if constexpr (!QUAD) {
                                a0[nr] = fma2(s0[2 * e], s0[2 * e + 1], nb[nr][2 * mm], nb[nr][2 * mm + 1], a0[nr]);
                                a1[nr] = fma2(s1[2 * e], s1[2 * e + 1], nb[nr][2 * mm], nb[nr][2 * mm + 1], a1[nr]);
                            }
                        }
                    }
                } else {
#pragma unroll
                    for (int e2 = 0; e2 < 2; ++e2) {
                        uint32_t r[4];
                        ldsm_x4(plane_at(kb, ko, kx, PK::R, tr, 4 * p + 2 * e2), r);
                        uint4 q4;
                        if constexpr (LO) q4 = qlo[(2 * p + e2) * 32 + lane];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int mm = 4 * p + 2 * e2 + e;
                            const uint32_t rg = r[2 * e], r8 = r[2 * e + 1];
                            const uint32_t x0 = by8(rg), x1 = by8(r8), x2 = by8(rg >> 8), x3 = by8(r8 >> 8);
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr) {
                                float d[4];
                                split::mma16816_zero(d, x0, x1, x2, x3, qh[nr][2 * mm], qh[nr][2 * mm + 1]);
                                if constexpr (LO) mma16816(d, x0, x1, x2, x3, e ? q4.z : q4.x, e ? q4.w : q4.y);
                                a0[nr].x = fmaf(s0[2 * e2 + e], d[0] + nb[nr][mm], a0[nr].x);
                                a1[nr].x = fmaf(s1[2 * e2 + e], d[2] + nb[nr][mm], a1[nr].x);
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                sc[nr][tt][0] = a0[nr].x + a0[nr].y;
                sc[nr][tt][1] = a1[nr].x + a1[nr].y;
            }
        }
        // ---- mask, online softmax ----
        // (rows past the last have q~ = 0 and no output: they need no mask)
        const bool edge = t0 + CH - 1 > pos_lo || (P.window && t0 < pos_hi - P.window + 1);
        uint32_t pb[NR][NT][2];  // fp16 scales: (p of token g, p of token g + 8)
        float pf[NR][NT][2];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            if (edge) {
#pragma unroll
                for (int tt = 0; tt < NT; ++tt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int t = t0 + 16 * tt + g + 8 * r;
                        if (t > pos[nr] || t < low[nr]) sc[nr][tt][r] = -INFINITY;
                    }
            }
            float mt = -INFINITY;
#pragma unroll
            for (int tt = 0; tt < NT; ++tt) mt = fmaxf(mt, fmaxf(sc[nr][tt][0], sc[nr][tt][1]));
            mt *= kSub;
            if (__any_sync(0xffffffffu, mt > mx[nr])) {
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
                const float mn = fmaxf(mx[nr], mt);
                const float f = mn == -INFINITY ? 1.f : ex2(mx[nr] - mn);
                l[nr] *= f;
#pragma unroll
                for (int i = 0; i < D / 4; ++i) acc[nr][i] *= f;
                mx[nr] = mn;
            }
            const float bias = mx[nr] == -INFINITY ? 0.f : mx[nr] - PBITS;
#pragma unroll
            for (int tt = 0; tt < NT; ++tt) {
                pf[nr][tt][0] = ex2(fmaf(sc[nr][tt][0], kSub, -bias));
                pf[nr][tt][1] = ex2(fmaf(sc[nr][tt][1], kSub, -bias));
                l[nr] += pf[nr][tt][0] + pf[nr][tt][1];
                if constexpr (SF == SRFTKV_SCALE_FP16) pb[nr][tt][0] = split::h2(pf[nr][tt][0], pf[nr][tt][1]);
            }
        }
        // ---- acc += codes_V^T . (p scale) ----
        const int hd = g >> 1, side = g & 1;
#pragma unroll
        for (int tt = 0; tt < NT; ++tt) {
            const int tr = 16 * tt;
            uint32_t q2[NR][2];  // fp16 scales: p of tokens (2c, 2c+1), (2c+8, 2c+9) of row hd
            float p4[NR][4];     // otherwise: of tokens 2c, 2c+1, 2c+8, 2c+9
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
                if constexpr (SF == SRFTKV_SCALE_FP16) {
                    const uint32_t u = __shfl_sync(0xffffffffu, pb[nr][tt][0], 8 * c + hd);
                    const uint32_t w = __shfl_sync(0xffffffffu, pb[nr][tt][0], 8 * c + 4 + hd);
                    q2[nr][0] = __byte_perm(u, w, 0x5410);
                    q2[nr][1] = __byte_perm(u, w, 0x7632);
                    if (BV == 8 && side) q2[nr][0] = q2[nr][1] = 0u;
                } else {
                    p4[nr][0] = __shfl_sync(0xffffffffu, pf[nr][tt][0], 8 * c + hd);
                    p4[nr][1] = __shfl_sync(0xffffffffu, pf[nr][tt][0], 8 * c + 4 + hd);
                    p4[nr][2] = __shfl_sync(0xffffffffu, pf[nr][tt][1], 8 * c + hd);
                    p4[nr][3] = __shfl_sync(0xffffffffu, pf[nr][tt][1], 8 * c + 4 + hd);
                    if (BV == 8 && side) p4[nr][0] = p4[nr][1] = p4[nr][2] = p4[nr][3] = 0.f;
                }
            }
            const int t4[4] = {tr + 2 * c, tr + 2 * c + 1, tr + 2 * c + 8, tr + 2 * c + 9};
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                // units of this thread's column in the piece: 4-bit 2e + side (e = 0, 1), 8-bit all four
                constexpr int NU = BV == 4 ? 2 : 4;
                uint32_t s2[NU][2];
                float sf[NU][4];
                if constexpr (SF == SRFTKV_SCALE_FP16) {
                    uint2 w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) w[k] = *reinterpret_cast<const uint2*>(vs + (t4[k] * (D / 16) + 4 * p) * 2);
#pragma unroll
                    for (int u = 0; u < NU; ++u) {
                        const bool second = BV == 4 ? u == 1 : u >= 2;
                        const uint32_t sel = (BV == 4 ? side : (u & 1)) ? 0x7632u : 0x5410u;
                        s2[u][0] = __byte_perm(second ? w[0].y : w[0].x, second ? w[1].y : w[1].x, sel);
                        s2[u][1] = __byte_perm(second ? w[2].y : w[2].x, second ? w[3].y : w[3].x, sel);
                    }
                } else {
#pragma unroll
                    for (int u = 0; u < NU; ++u)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            sf[u][k] = split::scale_at<D, SF>(vs, t4[k], 4 * p + (BV == 4 ? 2 * u + side : u));
                }
                auto operand = [&](int nr, int u, uint32_t& b0, uint32_t& b1) {
                    if constexpr (SF == SRFTKV_SCALE_FP16) {
                        b0 = split::hmul2(q2[nr][0], s2[u][0]);
                        b1 = split::hmul2(q2[nr][1], s2[u][1]);
                    } else {
                        const float2 f0 = mul2(p4[nr][0], p4[nr][1], sf[u][0], sf[u][1]);
                        const float2 f1 = mul2(p4[nr][2], p4[nr][3], sf[u][2], sf[u][3]);
                        b0 = split::h2(f0.x, f0.y);
                        b1 = split::h2(f1.x, f1.y);
                    }
                };
                if constexpr (BV == 4) {
                    uint32_t r[4];
                    ldsm_x4_t(plane_at(vb, vo, vx, PV::R, tr, 2 * p), r);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t R0 = r[2 * e], R1 = r[2 * e + 1], S0 = R0 >> 8, S1 = R1 >> 8;
                        const uint32_t x0 = lo4(R0), x1 = hi4(R0), x2 = lo4(R1), x3 = hi4(R1);
                        const uint32_t y0 = lo4(S0), y1 = hi4(S0), y2 = lo4(S1), y3 = hi4(S1);
#pragma unroll
                        for (int nr = 0; nr < NR; ++nr) {
                            uint32_t b0, b1;
                            operand(nr, e, b0, b1);
                            float(&f0)[4] = *reinterpret_cast<float(*)[4]>(&acc[nr][8 * (2 * p + e)]);
                            float(&f1)[4] = *reinterpret_cast<float(*)[4]>(&acc[nr][8 * (2 * p + e) + 4]);
                            mma16816(f0, x0, x1, x2, x3, b0, b1);
                            mma16816(f1, y0, y1, y2, y3, b0, b1);
                            mma16816(f0, off0, off1, off2, off3, b0, b1);
                            mma16816(f1, off0, off1, off2, off3, b0, b1);
                        }
                    }
                } else {
#pragma unroll
                    for (int e2 = 0; e2 < 2; ++e2) {
                        uint32_t r[4];
                        ldsm_x4_t(plane_at(vb, vo, vx, PV::R, tr, 4 * p + 2 * e2), r);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t R0 = r[2 * e], R1 = r[2 * e + 1];
                            const uint32_t x0 = by8(R0), x1 = by8(R0 >> 8), x2 = by8(R1), x3 = by8(R1 >> 8);
#pragma unroll
                            for (int nr = 0; nr < NR; ++nr) {
                                uint32_t b0, b1;
                                operand(nr, 2 * e2 + e, b0, b1);
                                float(&f0)[4] = *reinterpret_cast<float(*)[4]>(&acc[nr][4 * (4 * p + 2 * e2 + e)]);
                                mma16816(f0, x0, x1, x2, x3, b0, b1);
                                mma16816(f0, off0, off1, off2, off3, b0, b1);
                            }
                        }
                    }
                }
            }
        }
    }
    griddep_launch_dependents();

    // ---- the four warps meet, over the ring (its copies have all been waited for: the last groups are empty) ----
    __syncthreads();
    float* mw = reinterpret_cast<float*>(smem);        // [warps][rows][2]
    float* aw = mw + split::WARPS * M::ROWS * 2;       // [warps][rows][D]
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[nr] += __shfl_xor_sync(0xffffffffu, l[nr], off);
        if (g == 0) {
            mw[(warp * M::ROWS + 4 * nr + c) * 2] = mx[nr];
            mw[(warp * M::ROWS + 4 * nr + c) * 2 + 1] = l[nr];
        }
        float* a = aw + (warp * M::ROWS + 4 * nr + c) * D;
#pragma unroll
        for (int i = 0; i < D / 4; ++i) {
            const int e = i & 3;
            if constexpr (BV == 4) {  // rows g: dim 4g + 2j of the chunk (low nibbles), rows g + 8: the next one
                const int cb = i >> 3, j = (i >> 2) & 1;
                if ((e & 1) == (g >= 4 ? 1 : 0)) a[32 * cb + 4 * g + 2 * j + (e >> 1)] = acc[nr][i] * ((e >> 1) ? 1048576.f : kSub);
            } else {
                if ((e & 1) == 0) a[16 * (i >> 2) + 2 * g + (e >> 1)] = acc[nr][i] * kSub;
            }
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int r = warp; r < n_rows; r += split::WARPS) {
        float Mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < split::WARPS; ++w) Mx = fmaxf(Mx, mw[(w * M::ROWS + r) * 2]);
        float L = 0.f, o[E] = {};
        if (Mx != -INFINITY) {
#pragma unroll
            for (int w = 0; w < split::WARPS; ++w) {
                const float f = ex2(mw[(w * M::ROWS + r) * 2] - Mx);
                L = fmaf(f, mw[(w * M::ROWS + r) * 2 + 1], L);
#pragma unroll
                for (int j = 0; j < E; ++j) o[j] = fmaf(f, aw[(w * M::ROWS + r) * D + E * lane + j], o[j]);
            }
        }
        if (W.n_parts > 1) {
            const long long at = row_at(r) * W.n_parts + spl;
            if (lane == 0) *reinterpret_cast<float2*>(W.part_ml + 2 * at) = make_float2(Mx, L);
            float* a = W.part_acc + at * D + E * lane;
            if constexpr (E == 2) *reinterpret_cast<float2*>(a) = make_float2(o[0], o[1]);
            else {
#pragma unroll
                for (int j = 0; j < E / 4; ++j)
                    reinterpret_cast<float4*>(a)[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
        } else {
            const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
            for (int j = 0; j < E; ++j) o[j] *= inv;
            if (P.lam_v) {
                float lam[E];
                rot::load_lambda<D>(P.lam_v + (long long)h * D, lane, lam);
#pragma unroll
                for (int j = 0; j < E; ++j) o[j] = __fdiv_rn(o[j], lam[j]);
            }
            rot::inverse<D>(o, lane, P.tr_v, P.sign_mask, scratch);
            uint16_t* dst = static_cast<uint16_t*>(P.out) + row_ptr(P.out, P.out_stride, r);
            if (W.dtype == SRFTKV_DTYPE_BF16) rot::store_row<D>(reinterpret_cast<__nv_bfloat16*>(dst), lane, o);
            else rot::store_row<D>(reinterpret_cast<__half*>(dst), lane, o);
        }
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
template <int D, int BK, int BV, int SF, int NR, bool LO>
static int launch_split_one(const PagedAttnParams& P, const SplitWork& W, cudaStream_t stream) {
    using C = split::Cfg<D, BK, BV, SF>;
    using M = split::Smem<D, BK, BV, SF, NR, LO>;
    static_assert(M::BYTES <= 232448, "shared memory");
    SplitWork w = W;
    w.chunks = W.tokens / C::CH;
    auto* kernel = paged_attn_split_kernel<D, BK, BV, SF, NR, LO>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(done, reinterpret_cast<const void*>(kernel), M::BYTES);
    if (e == cudaSuccess) {
        kernel<<<dim3(W.n_splits, P.B * P.Hkv, W.groups), 128, M::BYTES, stream>>>(P, w);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) {
        set_error("paged attention launch failed: %s", cudaGetErrorString(e));
        return SRFTKV_ERR_CUDA;
    }
    return SRFTKV_OK;
}

template <int D, int SF, int NR, bool LO>
static int launch_split_bits(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s) {
    if (W.bits_k == 4)
        return W.bits_v == 4 ? launch_split_one<D, 4, 4, SF, NR, LO>(P, W, s) : launch_split_one<D, 4, 8, SF, NR, LO>(P, W, s);
    return W.bits_v == 4 ? launch_split_one<D, 8, 4, SF, NR, LO>(P, W, s) : launch_split_one<D, 8, 8, SF, NR, LO>(P, W, s);
}
// LO: bf16 rows carry 8 bits and their answer is rounded to 8, so q~ in fp16 alone (11) is not what limits it; fp16
// rows get hi + lo where registers allow (6 % of the time at 16 x 131072 tokens)
template <int D, int SF>
static int launch_split(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s) {
    if constexpr (D <= 128) {
        if (W.nr == 2) return launch_split_bits<D, SF, 2, false>(P, W, s);
        if (W.dtype == SRFTKV_DTYPE_FP16) return launch_split_bits<D, SF, 1, true>(P, W, s);
    }
    return launch_split_bits<D, SF, 1, false>(P, W, s);
}

}  // namespace srftkv
