// paged_attn_tile.cuh -- attention of blocks of query rows over the paged
// cache on the 5th-generation tensor cores (each d in its own translation
// unit).  The query rows of one sequence and kv head are its query tokens
// times the Hq / H heads that read that kv head, token-major; a CTA takes 256
// (d = 64, 128) or 128 (d = 256) of them and a range of the cache in tiles of
// BN tokens.
//
//   q~ = R_s q * sm_scale log2(e) / lambda_K      (one contraction, R_s as fp16 hi + lo)
//   S  = q~ . K^T,  K = code * scale in fp16       (M = 128 rows, N = BN tokens)
//   P  = 2^(S - m), online maximum m and sum l in fp32, one thread a row
//   O += P . V, V = code * scale in fp16           (P from tensor memory)
//   out = R_s^T (O / l / lambda_V)                 (one contraction more)
//
// The cache is never rotated back token by token: R_s is orthogonal, so the
// scores and the sum are the same in its coordinates.
//
// Warps: 0-7 softmax (a group of four a q tile; warp w reads tensor-memory
// lanes 32(w%4)..+31), 8-15 dequantise tiles from the pages into shared memory
// (128-byte-swizzled rows, two stages of K and of V), 16 issues the MMAs.  The
// two q tiles alternate on the tensor cores: while one is in its softmax the
// other's P.V and next S run.  At d = 256 O takes half of tensor memory, so
// one q tile alternates between two S buffers instead.
//
// Many blocks of rows read the same tiles, and turning codes into fp16 costs as
// many instructions as the softmax: with three blocks or more a kernel before
// this one lays every tile down once, as the image it has in shared memory
// (paged_expand_kernel, into the workspace), and the tiles arrive by one bulk
// copy each.
//
// What bounds it: the chain of one stream, softmax pass (1300 cycles a tile at
// d = 128: 128 exponentials a thread at 4 cycles a warp instruction, and their
// conversions), store of P (250), P.V and the next S (1024 with the other stream's
// between), which comes to about 2900 cycles for the 2048 that the products of
// both streams take.  Hence one barrier wait of the issuing warp a step (a wait
// between two MMAs costs 105 to 176 idle cycles though its phase is complete),
// one pass over S with the maximum in use so far (kLazy), and P kept in registers
// until the vote.  Measured: 2048 queries at 32768 tokens, 12 heads over 2, fp32
// scales: 347 us, 1150 TFLOP/s (59 % of cuBLAS's best; 502 us in the first form);
// 8191 queries at d = 64, 16 heads over 4: 277 us, 490 TFLOP/s, the exponentials.
//
// Few rows (at most 128 a sequence and kv head, "dual"): both streams hold the
// same rows and take every other tile, each with its own m, l and O, joined by
// the combine kernel like splits of the cache.
//
// Roundings: q~, K, V, P to fp16 (2^-11 each; K and V are exact code * scale
// products rounded once; with fp32 scales the scale enters as hi + lo), and
// O / l and R_s to fp16 on the way out.  m, l, S and O are fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "attn_frag.cuh"
#include "codec_tc_common.cuh"
#include "paged.h"
#include "ptx.cuh"
#include "srft_math.cuh"
#include "tcgen05.cuh"

namespace srftkv {

namespace tile {

constexpr int SM_WARPS = 8, DQ_WARPS = 8;
constexpr int THREADS = (SM_WARPS + DQ_WARPS + 1) * 32;
constexpr float kLazy = 8.f;  // O is rescaled when the maximum grew by more than this (P stays below 2^8)

template <int D>
struct Cfg {
    static constexpr int NQ = D == 256 ? 1 : 2;    // q tiles of 128 rows
    static constexpr int BN = D == 256 ? 64 : 128; // tokens a tile
    static constexpr int QB = 128 * D * 2;         // bytes of a q tile
    static constexpr int TB = BN * D * 2;          // bytes of a K or V tile
    static constexpr int OFF_K = NQ * QB;
    static constexpr int OFF_V = OFF_K + 2 * TB;
    static constexpr int OFF_TW = OFF_V + 2 * TB;       // cos, -sin of 2 pi m / d
    static constexpr int OFF_SG = OFF_TW + D * 8;       // sign words
    static constexpr int OFF_BAR = OFF_SG + D * 2;
    static constexpr int USED = OFF_BAR + 256;
    // one CTA an SM: it owns all of tensor memory
    static constexpr int SMEM = (USED > 120 * 1024 ? USED : 120 * 1024) + 1024;
    static constexpr int O_COL = 256;
    static constexpr int S_STEP = NQ == 2 ? 128 : BN;   // columns between S buffers
    static constexpr int R_COL = NQ == 2 ? 0 : O_COL;   // rotated q (fp32) before the loop
    // P.  At d = 128 tensor memory is full and P takes the columns its S was read from: the next S into them is
    // issued after the P.V that reads them and has its shape, so the two run in order.  At the other d the two
    // shapes differ (their order is not given) and there are columns to spare; a P is then only overwritten after
    // the next S of its buffer was seen complete, whose commit covers the P.V before it.
    static constexpr int P_COL = D == 128 ? 0 : D == 64 ? 384 : 128;
    static constexpr int P_STEP = D == 128 ? S_STEP : BN / 2;
    static_assert(SMEM <= 232448, "shared memory");
};

// Descriptors as two words, so that a loop steps through an operand by adding to the low one.  K-major, 128-byte
// swizzle (tc::sw128_desc); and MN-major (rows of the contraction index, 64 of N a 128-byte row): 8-row groups 1024
// bytes apart, 64-column blocks `lbo` bytes apart.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return ((addr >> 4) & 0x3FFFu) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr, uint32_t lbo) { return ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16); }
__device__ __forceinline__ uint64_t desc(uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; }
// One thread of a converged warp.  The MMA warp runs its loop as a whole and only the issue is one thread's: with the
// loop itself in one thread every operand was moved to a uniform register at its use, and eight MMAs took 900 cycles to
// issue that take 512 to run.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool b_mn) {
    return tc::idesc_f16_f32(M, N) | (b_mn ? 1u << 16 : 0u);
}

// A softmax thread holds a row of P (64 registers) beside two loads of S (32); a dequantising one needs half of that.
// The kernel is compiled for kRegs a thread (launch_tile checks it): 8 warps give back 16, 8 take them (at 64 the others spilled).
constexpr int kRegs = 96;
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 112;"); }
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 80;"); }

// Entries x0 .. x0 + 7 of row n of R_s times 2^UP
template <int D, int UP>
__device__ __forceinline__ void r_entries(int n, int x0, bool srht, const float2* tw, const uint32_t* sg, float (&v)[8]) {
    const float isd = rsqrtf((float)D) * (float)(1 << UP), c2 = 1.41421356237309505f * isd;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int x = x0 + e;
        if (srht) v[e] = (__popc(n & x) & 1) ? -isd : isd;
        else if (n == 0) v[e] = isd;
        else if (n == 1) v[e] = (x & 1) ? -isd : isd;
        else {
            const float2 w = tw[((n >> 1) * x) & (D - 1)];
            v[e] = c2 * ((n & 1) ? w.y : w.x);
        }
        if (sg[x >> 1] & ((e & 1) ? 0x80000000u : 0x8000u)) v[e] = -v[e];
    }
}
// the 16-byte chunk of them as fp16 hi (and lo)
template <int D, bool LO, int UP = 0>
__device__ __forceinline__ void r_chunk(int n, int x0, bool srht, const float2* tw, const uint32_t* sg, uint4& hi,
                                        uint4& lo) {
    float v[8];
    r_entries<D, UP>(n, x0, srht, tw, sg, v);
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (LO) split_pair_h2(v[2 * j], v[2 * j + 1], h[j], l[j]);
        else h[j] = pack_half2(v[2 * j], v[2 * j + 1]);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    if constexpr (LO) lo = make_uint4(l[0], l[1], l[2], l[3]);
}

// eight 4-bit codes of word w (or eight 8-bit codes of words w, w2) times the scale, as fp16 pairs in the
// order of dq_kperm; LO: the scale is sh + sl
template <int BITS, bool LO>
__device__ __forceinline__ uint4 dequant8(uint32_t w, uint32_t w2, uint32_t sh, uint32_t sl) {
    uint32_t c[4];
    if constexpr (BITS == 4) {
        const uint32_t ws = w >> 8;
        c[0] = codes_lo4(w);
        c[1] = codes_hi4(w);
        c[2] = codes_lo4(ws);
        c[3] = codes_hi4(ws);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c[j] = codes_b8(__byte_perm(w, w2, j | (j << 4) | ((4 + j) << 8) | ((4 + j) << 12)));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = LO ? h2fma(c[j], sh, h2mul(c[j], sl)) : h2mul(c[j], sh);
    return make_uint4(c[0], c[1], c[2], c[3]);
}

// The raw bytes of one dequantising thread's piece of a tile row: DP coordinates (32 or 64)
template <int DP>
struct Piece {
    uint32_t w[DP / 4];   // 8-bit: DP/4 words, 4-bit: the first DP/8
    float sc[DP / 16];    // scale of each 16-coordinate unit, or (packed) its bits as loaded
    bool packed;          // sc[0 .. 1] hold the units' fp16 scales two a word, sc[0] their e8m0 bytes: a conversion
                          // beside the load would wait for it
};
template <int DP>
__device__ __forceinline__ void unpack_scales(Piece<DP>& p, int sfmt) {
    constexpr int U = DP / 16;
    if (!p.packed) return;
    const uint32_t a = __float_as_uint(p.sc[0]), b = U > 2 ? __float_as_uint(p.sc[U > 2 ? 1 : 0]) : 0u;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const uint32_t w = i < 2 ? a : b;
        if (sfmt == SRFTKV_SCALE_FP16) p.sc[i] = __half2float(__ushort_as_half((unsigned short)(w >> (16 * (i & 1)))));
        else p.sc[i] = __uint_as_float(((a >> (8 * i)) & 0xFFu) << 23);
    }
}

// Load the piece of row `row` (packed row index, -1: zeros) that starts at coordinate x0
template <int D, int DP>
__device__ __forceinline__ void load_piece(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                           long long row, int x0, int bits, int sfmt, int lg_group, Piece<DP>& p) {
    constexpr int U = DP / 16;
    p.packed = lg_group == 4 && sfmt != SRFTKV_SCALE_FP32;
    if (row < 0) {
#pragma unroll
        for (int i = 0; i < DP / 4; ++i) p.w[i] = 0u;
#pragma unroll
        for (int i = 0; i < U; ++i) p.sc[i] = 0.f;
        return;
    }
    if (bits == 4) {
        const uint4* c = reinterpret_cast<const uint4*>(codes + row * (D / 2) + x0 / 2);
#pragma unroll
        for (int i = 0; i < DP / 32; ++i) {
            const uint4 v = __ldg(c + i);
            p.w[4 * i] = v.x, p.w[4 * i + 1] = v.y, p.w[4 * i + 2] = v.z, p.w[4 * i + 3] = v.w;
        }
    } else {
        const uint4* c = reinterpret_cast<const uint4*>(codes + row * D + x0);
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
            const uint4 v = __ldg(c + i);
            p.w[4 * i] = v.x, p.w[4 * i + 1] = v.y, p.w[4 * i + 2] = v.z, p.w[4 * i + 3] = v.w;
        }
    }
    const int ng = D >> lg_group;
    if (lg_group == 4) {  // one scale a unit: a vector of them
        if (sfmt == SRFTKV_SCALE_FP32) {
            const float* s = reinterpret_cast<const float*>(scales) + row * ng + x0 / 16;
            if constexpr (U == 4) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(s));
                p.sc[0] = v.x, p.sc[1] = v.y, p.sc[2] = v.z, p.sc[3] = v.w;
            } else {
                const float2 v = __ldg(reinterpret_cast<const float2*>(s));
                p.sc[0] = v.x, p.sc[1] = v.y;
            }
        } else if (sfmt == SRFTKV_SCALE_FP16) {
            const __half* s = reinterpret_cast<const __half*>(scales) + row * ng + x0 / 16;
            if constexpr (U == 4) {
                const uint2 t = __ldg(reinterpret_cast<const uint2*>(s));
                p.sc[0] = __uint_as_float(t.x), p.sc[1] = __uint_as_float(t.y);
            } else {
                p.sc[0] = __uint_as_float(__ldg(reinterpret_cast<const uint32_t*>(s)));
            }
        } else {
            uint32_t v;
            if constexpr (U == 4) v = __ldg(reinterpret_cast<const uint32_t*>(scales + row * ng + x0 / 16));
            else v = __ldg(reinterpret_cast<const unsigned short*>(scales + row * ng + x0 / 16));
            p.sc[0] = __uint_as_float(v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const long long at = row * ng + ((x0 + 16 * i) >> lg_group);
            if (sfmt == SRFTKV_SCALE_FP32) p.sc[i] = __ldg(reinterpret_cast<const float*>(scales) + at);
            else if (sfmt == SRFTKV_SCALE_FP16) p.sc[i] = __half2float(__ldg(reinterpret_cast<const __half*>(scales) + at));
            else p.sc[i] = __uint_as_float((uint32_t)__ldg(scales + at) << 23);
        }
    }
}

// Write a piece as fp16 into row r of a swizzled tile of BN rows
template <int D, int BN, int DP, int BITS, bool LO>
__device__ __forceinline__ void store_piece(uint8_t* tile, int r, int x0, const Piece<DP>& p) {
#pragma unroll
    for (int u = 0; u < DP / 16; ++u) {
        const __half h = __float2half_rn(p.sc[u]);
        const uint32_t sh = half2_bcast(h);
        const uint32_t sl = LO ? half2_bcast(__float2half_rn(p.sc[u] - __half2float(h))) : 0u;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int k = 2 * u + e;  // 8-coordinate chunk of the piece
            const uint4 v = BITS == 4 ? dequant8<4, LO>(p.w[k], 0u, sh, sl)
                                      : dequant8<8, LO>(p.w[(2 * k) % (DP / 4)], p.w[(2 * k + 1) % (DP / 4)], sh, sl);
            const int x = x0 + 8 * k;
            *reinterpret_cast<uint4*>(tile + (x >> 6) * (BN * 128) + r * 128 + ((((x & 63) >> 3) ^ (r & 7)) << 4)) = v;
        }
    }
}
template <int D, int BN, int DP>
__device__ __forceinline__ void store_piece_any(uint8_t* tile, int r, int x0, int bits, bool lo, const Piece<DP>& p) {
    if (bits == 4) {
        if (lo) store_piece<D, BN, DP, 4, true>(tile, r, x0, p);
        else store_piece<D, BN, DP, 4, false>(tile, r, x0, p);
    } else {
        if (lo) store_piece<D, BN, DP, 8, true>(tile, r, x0, p);
        else store_piece<D, BN, DP, 8, false>(tile, r, x0, p);
    }
}

}  // namespace tile

// The tiles of one (sequence, kv head) as fp16 images: K then V, each TB bytes as the tile kernel wants it in shared
// memory.  Tiles that no query sees are left out.
template <int D>
__global__ void __launch_bounds__(256) paged_expand_kernel(const __grid_constant__ PagedAttnParams P,
                                                           const __grid_constant__ TileWork W) {
    using C = tile::Cfg<D>;
    constexpr int BN = C::BN, DP = BN * D / 256, PER = D / DP;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const int t = blockIdx.x, b = blockIdx.y / P.Hkv, h = blockIdx.y - b * P.Hkv;
    const int len = min(max(P.seq_lens[b], 0), P.max_len);
    const int m_tok = P.cu_q ? min(max(P.cu_q[b + 1] - P.cu_q[b], 0), P.max_q) : 1;
    const int low = P.window ? max(0, len - m_tok - P.window + 1) : 0;  // the first token the first query sees
    if (m_tok > 0 && t * BN < len && (t + 1) * BN > low) {
        const int r = threadIdx.x / PER, x0 = (threadIdx.x % PER) * DP, tok = t * BN + r;
        long long row = -1;
        if (tok < len && tok >= low) {  // (pages before every window may be gone: not looked at)
            const int pg = __ldg(P.table + (long long)b * P.max_pages + (tok >> P.lg_page));
            if ((unsigned)pg < (unsigned)P.n_pages)
                row = (((long long)pg * P.Hkv + h) << P.lg_page) | (tok & ((1 << P.lg_page) - 1));
            else
                atomicOr(P.fault, kFaultPage);
        }
        tile::Piece<DP> pk, pv;
        tile::load_piece<D, DP>(P.kc, P.ks, row, x0, W.bits_k, P.sfmt, P.lg_group, pk);
        tile::load_piece<D, DP>(P.vc, P.vs, row, x0, W.bits_v, P.sfmt, P.lg_group, pv);
        const bool lo = P.sfmt == SRFTKV_SCALE_FP32;
        tile::unpack_scales(pk, P.sfmt);
        tile::unpack_scales(pv, P.sfmt);
        tile::store_piece_any<D, BN, DP>(smem, r, x0, W.bits_k, lo, pk);
        tile::store_piece_any<D, BN, DP>(smem + C::TB, r, x0, W.bits_v, lo, pv);
        ptx::fence_proxy_async_smem();
        __syncthreads();
        if (threadIdx.x == 0) {
            uint8_t* to = W.images + ((long long)blockIdx.y * W.tiles + t) * (2 * C::TB);
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(ptx::smem_u32(smem)),
                         "r"(2 * C::TB)
                         : "memory");
            ptx::bulk_commit();
            ptx::bulk_wait<0>();
        }
    }
    griddep_launch_dependents();
}

template <int D>
__global__ void __launch_bounds__(tile::THREADS, 1)
    paged_attn_tile_kernel(const __grid_constant__ PagedAttnParams P, const __grid_constant__ TileWork W) {
    using C = tile::Cfg<D>;
    constexpr int NQ = C::NQ, BN = C::BN;
    constexpr int SMW = 4 * NQ;  // softmax warps at work
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

    // ---- this CTA's rows and tiles ----
    const int b = blockIdx.x / P.Hkv, h = blockIdx.x - b * P.Hkv;
    const int blk = gridDim.y - 1 - blockIdx.y;  // the longest rows (causal) first
    const int split = blockIdx.z;
    const int q0 = P.cu_q ? P.cu_q[b] : b;
    int m_tok = min(P.cu_q ? P.cu_q[b + 1] - q0 : 1, P.max_q);
    if (q0 < 0) m_tok = 0;
    m_tok = min(m_tok, P.total_q - q0);
    const int n_rows = m_tok * P.rep;
    const int row0 = blk * W.rows_per_block;
    if (row0 >= n_rows) {
        griddep_wait();  // (a kernel after this one may start only once the expanding kernel is over too)
        return;
    }
    const int len = min(max(P.seq_lens[b], 0), P.max_len);
    const int rows_here = min(W.rows_per_block, n_rows - row0);
    const int pos_lo = len - m_tok + row0 / P.rep, pos_hi = len - m_tok + (row0 + rows_here - 1) / P.rep;
    const int low = P.window ? max(0, pos_lo - P.window + 1) : 0;  // the first token any row sees
    int ta = low / BN;
    int tb = pos_hi >= 0 ? pos_hi / BN + 1 : 0;
    ta = ta + split * W.tps;
    tb = min(tb, W.n_splits > 1 ? ta + W.tps : tb);
    const int n = max(0, tb - ta);  // tiles
    const bool dual = NQ == 2 && W.dual;

    // row r of the block -> its row of q / out
    auto out_row = [&](int r, int& i, int& hq) {
        i = (row0 + r) / P.rep;
        hq = h * P.rep + (row0 + r - i * P.rep);
        i += q0;
    };
    if (n == 0) {  // nothing visible: zeros, or empty partials
        griddep_wait();
        for (int r = threadIdx.x; r < rows_here; r += blockDim.x) {
            int i, hq;
            out_row(r, i, hq);
            if (W.n_parts == 1) {
                uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.out) + i * P.out_stride + (long long)hq * D);
                for (int c = 0; c < D / 8; ++c) o[c] = make_uint4(0, 0, 0, 0);
            } else {
                const int per = W.n_parts / W.n_splits;
                for (int e = 0; e < per; ++e) {
                    float* ml = W.part_ml + (((long long)i * P.Hq + hq) * W.n_parts + split * per + e) * 2;
                    ml[0] = -INFINITY;
                    ml[1] = 0.f;
                }
            }
        }
        return;
    }

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    auto bar = [&](int i) { return ptx::smem_u32(&bars[i]); };
    // READY + 2 i + (j & 1): all that stream i's MMAs of step j need: its P, the V tile of the step and the K tile of
    // the S that follows.  One barrier, and so one wait of the MMA warp: a wait costs the tensor cores 105 idle cycles
    // even when it finds the phase complete.  Two of them in turn, so that an arrival for step j cannot land in the
    // phase of step j - 1; what frees the K and V stages of step j also completes step j - 2.
    // S_DONE, PV_DONE + 2 i + (j & 1): the S and the P.V of step j of stream i, which also free the K and V tile (with
    // two streams on a tile: stream 1's, the later one).
    constexpr int K_FIRST = 0, S_DONE = 2, PV_DONE = 6, READY = 10, ROT = 14, R_FULL = 15, EP_FULL = 16, OUT_FULL = 17,
                  N_BARS = 18;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(&bars[N_BARS]);
    float2* tw = reinterpret_cast<float2*>(smem + C::OFF_TW);
    uint32_t* sg = reinterpret_cast<uint32_t*>(smem + C::OFF_SG);
    if (threadIdx.x == 0) {
        for (int s = 0; s < 2; ++s) {
            const int tile_arrivals = W.images ? 1 : tile::DQ_WARPS;
            ptx::mbar_init(bar(K_FIRST + s), tile_arrivals);
            for (int i = 0; i < 2; ++i) ptx::mbar_init(bar(READY + 2 * i + s), 4 + (i == 0 || dual ? 2 * tile_arrivals : 0));
            for (int i = 0; i < 2; ++i) {
                ptx::mbar_init(bar(S_DONE + 2 * i + s), 1);
                ptx::mbar_init(bar(PV_DONE + 2 * i + s), 1);
            }
        }
        ptx::mbar_init(bar(ROT), 1);
        ptx::mbar_init(bar(R_FULL), tile::DQ_WARPS);
        ptx::mbar_init(bar(EP_FULL), SMW);
        ptx::mbar_init(bar(OUT_FULL), 1);
        ptx::fence_barrier_init();
    }
    if (warp == 16) {
        tc::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
        tc::tmem_relinquish();
    }
    for (int m = threadIdx.x; m < D; m += blockDim.x) tw[m] = make_float2(tw_re_lane(m * (256 / D)), tw_im_lane(m * (256 / D)));
    for (int i = threadIdx.x; i < D / 2; i += blockDim.x) sg[i] = P.sign_mask[i];

    // ---- q rows as fp16 into the q tiles (zeros past the last row) ----
    const int q_rows = dual || NQ == 1 ? 128 : 256;
    for (int c = threadIdx.x; c < q_rows * (D / 8); c += blockDim.x) {
        const int r = c / (D / 8), ch = c % (D / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < rows_here) {
            int i, hq;
            out_row(r, i, hq);
            v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.q) + i * P.q_stride + (long long)hq * D) + ch);
            if (W.dtype == SRFTKV_DTYPE_BF16) {  // 8 significant bits: exact in fp16 within its range
                uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xFFFF0000u);
                    w[j] = pack_half2(lo, hi);
                }
            }
        }
        *reinterpret_cast<uint4*>(smem + (r >> 7) * C::QB + (ch >> 3) * 16384 + (r & 127) * 128 +
                                  (((ch & 7) ^ (r & 7)) << 4)) = v;
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    bool failed = false;

    // ---- rotate them: R_s rows in steps of 128 outputs, hi and lo, in the K and V stages ----
    const int n_qt = q_rows / 128;
    constexpr int NB = D < 128 ? D : 128;
    for (int nh = 0; nh < D / NB; ++nh) {
        for (int c = threadIdx.x; c < NB * (D / 8); c += blockDim.x) {
            const int nr = c / (D / 8), ch = c % (D / 8);
            uint4 hi, lo;
            tile::r_chunk<D, true>(nh * NB + nr, 8 * ch, P.tr_k == SRFTKV_TRANSFORM_SRHT, tw, sg, hi, lo);
            uint8_t* at = smem + C::OFF_K + (ch >> 3) * (NB * 128) + nr * 128 + (((ch & 7) ^ (nr & 7)) << 4);
            *reinterpret_cast<uint4*>(at) = hi;
            *reinterpret_cast<uint4*>(at + NB * D * 2) = lo;
        }
        ptx::fence_proxy_async_smem();
        __syncthreads();
        if (warp == 0 && tile::elect()) {
            const uint32_t bo = tile::desc_k(sbase + C::OFF_K);
            for (int i = 0; i < n_qt; ++i) {
                const uint32_t ao = tile::desc_k(sbase + i * C::QB), dst = tmem + C::R_COL + i * 128 + nh * NB;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t as = (ks >> 2) * 1024 + (ks & 3) * 2, bs = (ks >> 2) * (NB * 8) + (ks & 3) * 2;
                    tc::mma_f16(dst, tile::desc(ao + as), tile::desc(bo + bs), tile::idesc(128, NB, false), ks > 0);
                    tc::mma_f16(dst, tile::desc(ao + as), tile::desc(bo + bs + NB * D / 8), tile::idesc(128, NB, false), 1);
                }
            }
            tc::commit(bar(ROT));
        }
        __syncwarp();
        if (!__all_sync(0xffffffffu, ptx::mbar_spin_bounded(bar(ROT), nh & 1))) failed = true;  // (a warp's lanes alike)
        tc::fence_after_sync();
        __syncthreads();
    }
    // each softmax thread scales its row and writes it back as the A operand, in the order of dq_kperm
    if (warp < 4 * n_qt && !failed) {
        const int i = warp >> 2, r = 32 * (warp & 3) + lane;
        uint8_t* qrow = smem + i * C::QB + r * 128;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
            uint32_t v[32];
            tc::ld_32x32b_x32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + C::R_COL + i * 128 + 32 * c, v);
            tc::wait_ld(v);
            float f[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]) * P.qscale;
            if (P.lam_k) {
#pragma unroll
                for (int j = 0; j < 32; ++j) f[j] = __fdiv_rn(f[j], __ldg(P.lam_k + (long long)h * D + 32 * c + j));
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const int ch = 4 * c + w;
                *reinterpret_cast<uint4*>(qrow + (ch >> 3) * 16384 + (((ch & 7) ^ (r & 7)) << 4)) =
                    make_uint4(pack_half2(f[8 * w], f[8 * w + 4]), pack_half2(f[8 * w + 1], f[8 * w + 5]),
                               pack_half2(f[8 * w + 2], f[8 * w + 6]), pack_half2(f[8 * w + 3], f[8 * w + 7]));
            }
        }
        ptx::fence_proxy_async_smem();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();

    auto steps_of = [&](int i) { return dual ? (n + 1 - i) / 2 : n; };
    // the barrier that tile t's K and V arrive on, and whether the step of its V is its stream's last but `ahead`
    constexpr int AHEAD = NQ == 2 ? 1 : 2;  // steps between a P.V and the S issued after it
    auto v_bar = [&](int t) { return dual ? READY + 2 * (t & 1) + ((t >> 1) & 1) : READY + (t & 1); };
    auto k_bar = [&](int t) {
        if (dual) return t < 2 ? K_FIRST + t : READY + 2 * (t & 1) + (((t >> 1) - 1) & 1);
        return t < AHEAD ? K_FIRST + t : READY + ((t - AHEAD) & 1);
    };
    // tile t's K (V) was read: the barrier, and its phase's parity
    const int last = NQ == 2 ? 1 : 0;
    auto freed = [&](int which, int t) { return dual ? which + 2 * (t & 1) + ((t >> 1) & 1) : which + 2 * last + (t & 1); };
    auto freed_parity = [&](int t) -> uint32_t { return dual ? (t >> 2) & 1 : (t >> 1) & 1; };
    auto no_next_k = [&](int t) { return t + (dual ? 2 : AHEAD) >= n; };  // the barrier of V t gets its K arrivals bare
    auto wait = [&](int which, uint32_t parity) -> bool {  // a whole warp, converged afterwards
        if (__all_sync(0xffffffffu, ptx::mbar_spin_bounded(bar(which), parity))) return true;
        failed = true;
        return false;
    };

    // (d = 256: warps 4-7 have nothing to do)
    if (warp < SMW) {
        // =========================== softmax ===========================
        if (NQ == 2) tile::more_registers();
        if (!failed) {
        const int i = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int r = (dual ? 0 : i * 128) + 32 * (warp & 3) + lane;
        const bool live = r < rows_here;
        const bool any_live = __any_sync(0xffffffffu, live);
        int oi = 0, hq = 0;
        if (live) out_row(r, oi, hq);
        const int pos = live ? len - m_tok + (row0 + r) / P.rep : -1;
        const int first = P.window ? pos - P.window + 1 : 0;
        const uint32_t o_col = tmem + lanes + C::O_COL + (NQ == 2 ? i * D : 0);
        float mx = -INFINITY, l = 0.f;
        const int steps = steps_of(i);
        for (int j = 0; j < steps; ++j) {
            const int sb = NQ == 2 ? i : (j & 1);
            if (!wait(S_DONE + 2 * i + (j & 1), (j >> 1) & 1)) break;
            if (any_live) {
                tc::fence_after_sync();
                const int t0 = (ta + (dual ? 2 * j + i : j)) * BN;
                const uint32_t s_col = tmem + lanes + sb * C::S_STEP, p_col = tmem + lanes + C::P_COL + sb * C::P_STEP;
                const int hi = pos - t0, lo = first - t0;  // visible columns lo .. hi
                const bool full = __all_sync(0xffffffffu, hi >= BN - 1 && lo <= 0);
                // One pass: P with the maximum in use so far, and the tile's own maximum beside it.  The former may lag
                // by kLazy (P stays below 2^8); where a row of the warp outgrew that, O is rescaled and the pass
                // is taken again, from S, which is still there: P stays in registers until the vote.
                uint32_t p[BN / 2];
                float sum = 0.f;
                auto pass = [&](float mu) -> float {
                    float2 s2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    float mt[2] = {-INFINITY, -INFINITY};
                    uint32_t v[2][16];
                    tc::ld_32x32b_x16(s_col, v[0]);
#pragma unroll
                    for (int c = 0; c < BN / 16; ++c) {
                        uint32_t(&w)[16] = v[c & 1];
                        tc::wait_ld(w);
                        if (c + 1 < BN / 16) tc::ld_32x32b_x16(s_col + 16 * (c + 1), v[(c + 1) & 1]);
                        if (!full) {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (16 * c + e > hi || 16 * c + e < lo) w[e] = 0xFF800000u;
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float a = __uint_as_float(w[2 * e]), d = __uint_as_float(w[2 * e + 1]);
                            mt[e & 1] = fmaxf(mt[e & 1], fmaxf(a, d));
                            const float2 x = __fadd2_rn(make_float2(a, d), make_float2(-mu, -mu));
                            const float2 y = make_float2(ex2(x.x), ex2(x.y));
                            s2[e & 1] = __fadd2_rn(s2[e & 1], y);
                            p[8 * c + e] = pack_half2(y.x, y.y);
                        }
                    }
                    sum = (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
                    return fmaxf(mt[0], mt[1]);
                };
                const float mt = pass(mx == -INFINITY ? 0.f : mx);
                const bool grow = mt > mx + tile::kLazy || (mx == -INFINITY && mt > -INFINITY);
                if (__any_sync(0xffffffffu, grow)) {
                    const float mn = fmaxf(mx, mt);
                    const float f = mx == -INFINITY ? 0.f : ex2(mx - mn);  // (O is 0 or unset while mx is -inf)
                    l *= f;
                    mx = mn;
                    if (j > 0) {
                        if (!wait(PV_DONE + 2 * i + ((j - 1) & 1), ((j - 1) >> 1) & 1)) break;
                        tc::fence_after_sync();
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t v[32];
                            tc::ld_32x32b_x32(o_col + 32 * c, v);
                            tc::wait_ld(v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
                            tc::st_32x32b_x32(o_col + 32 * c, v);
                        }
                    }
                    pass(mx == -INFINITY ? 0.f : mx);
                }
                l += sum;
#pragma unroll
                for (int c = 0; c < BN / 64; ++c) tc::st_32x32b_x32(p_col + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(p + 32 * c));
                tc::wait_st();
                tc::fence_before_sync();
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(READY + 2 * i + (j & 1)));
        }
        // ---- the end: O / l rotated back, or a partial result ----
        if (!failed && steps > 0) {
            if (wait(PV_DONE + 2 * i + ((steps - 1) & 1), ((steps - 1) >> 1) & 1)) tc::fence_after_sync();
        }
        if (W.n_parts > 1) {
            if (!failed && live) {
                const int part = dual ? 2 * split + i : split;
                const long long at = ((long long)oi * P.Hq + hq) * W.n_parts + part;
                W.part_ml[2 * at] = steps ? mx : -INFINITY;
                W.part_ml[2 * at + 1] = l;
            }
            if (!failed && steps > 0 && any_live) {
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t v[32];
                    tc::ld_32x32b_x32(o_col + 32 * c, v);
                    tc::wait_ld(v);
                    if (live) {
                        const int part = dual ? 2 * split + i : split;
                        uint4* o = reinterpret_cast<uint4*>(W.part_acc + (((long long)oi * P.Hq + hq) * W.n_parts + part) * D + 32 * c);
#pragma unroll
                        for (int w = 0; w < 4; ++w) {  // column 8w + 2k + e holds coordinate 8w + k + 4e
                            o[2 * w] = make_uint4(v[8 * w], v[8 * w + 2], v[8 * w + 4], v[8 * w + 6]);
                            o[2 * w + 1] = make_uint4(v[8 * w + 1], v[8 * w + 3], v[8 * w + 5], v[8 * w + 7]);
                        }
                    }
                }
            }
        } else if (!failed) {
            const float inv = l > 0.f ? 1.f / l : 0.f;
            uint8_t* arow = smem + i * C::QB + (32 * (warp & 3) + lane) * 128;
            const int rr = 32 * (warp & 3) + lane;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tc::ld_32x32b_x32(o_col + 32 * c, v);
                tc::wait_ld(v);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    float f[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)  // natural coordinate k from column 2 (k % 4) + k / 4
                        f[k] = l > 0.f ? __uint_as_float(v[8 * w + 2 * (k & 3) + (k >> 2)]) * inv : 0.f;
                    if (P.lam_v) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            f[k] = __fdiv_rn(f[k], __ldg(P.lam_v + (long long)h * D + 32 * c + 8 * w + k));
                    }
                    const int ch = 4 * c + w;
                    *reinterpret_cast<uint4*>(arow + (ch >> 3) * 16384 + (((ch & 7) ^ (rr & 7)) << 4)) =
                        make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]), pack_half2(f[4], f[5]),
                                   pack_half2(f[6], f[7]));
                }
            }
            ptx::fence_proxy_async_smem();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(EP_FULL));
            if (wait(OUT_FULL, 0) && any_live) {
                tc::fence_after_sync();
                uint16_t* o = static_cast<uint16_t*>(P.out) + oi * P.out_stride + (long long)hq * D;
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t v[32];
                    tc::ld_32x32b_x32(tmem + lanes + i * 128 + 32 * c, v);
                    tc::wait_ld(v);
                    uint32_t w[16];
                    if (W.dtype == SRFTKV_DTYPE_BF16) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const __nv_bfloat162 t = __floats2bfloat162_rn(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                            w[e] = *reinterpret_cast<const uint32_t*>(&t);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = pack_half2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                    }
                    if (live) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            reinterpret_cast<uint4*>(o + 32 * c)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                    }
                }
            }
        }
        }
    } else if (warp >= 8 && warp < 16) {
        // =========================== dequantise ===========================
        if (NQ == 2) tile::fewer_registers();
        if (!failed) {
        constexpr int DP = BN * D / 256;        // coordinates a thread
        constexpr int PER = D / DP;             // threads a row
        const int dt = threadIdx.x - 256, r = dt / PER, x0 = (dt % PER) * DP;
        const int* table = P.table + (long long)b * P.max_pages;
        const bool lo = P.sfmt == SRFTKV_SCALE_FP32;
        // the page of this thread's token in tile t (looked up two tiles ahead, and not looked at until its row is wanted),
        // and its packed row, -1: none
        auto page_of = [&](int t) -> int {
            const int tok = (ta + t) * BN + r;
            return t < n && tok < len ? __ldg(table + (tok >> P.lg_page)) : 0;
        };
        auto row_of = [&](int t, int pg) -> long long {
            const int tok = (ta + t) * BN + r;
            if (t >= n || tok >= len || tok < low) return -1;  // (pages before every window may be gone)
            if ((unsigned)pg >= (unsigned)P.n_pages) {
                atomicOr(P.fault, kFaultPage);
                return -1;
            }
            return ((((long long)pg * P.Hkv + h) << P.lg_page) | (tok & ((1 << P.lg_page) - 1)));
        };
        if (W.images) {
            // one thread fetches the images; the other warps wait for it at the barrier below
            if (warp == 8) {
                griddep_wait();  // (the expanding kernel)
                const bool one = tile::elect();
                const uint8_t* img = W.images + ((long long)blockIdx.x * W.tiles + ta) * (2 * C::TB);
                for (int t = 0; t < n; ++t) {
                    const int st = t & 1;
                    if (t >= 2 && !wait(freed(S_DONE, t - 2), freed_parity(t - 2))) break;
                    if (one) {
                        ptx::mbar_arrive_expect_tx(bar(k_bar(t)), C::TB);
                        ptx::bulk_load(sbase + C::OFF_K + st * C::TB, img + (long long)t * (2 * C::TB), C::TB, bar(k_bar(t)));
                    }
                    if (t >= 2 && !wait(freed(PV_DONE, t - 2), freed_parity(t - 2))) break;
                    if (one) {
                        ptx::mbar_arrive_expect_tx(bar(v_bar(t)), C::TB);
                        ptx::bulk_load(sbase + C::OFF_V + st * C::TB, img + (long long)t * (2 * C::TB) + C::TB, C::TB, bar(v_bar(t)));
                        if (no_next_k(t)) ptx::mbar_arrive(bar(v_bar(t)));
                    }
                    __syncwarp();
                }
                // a wait that ran out: the copies it leaves land before the CTA ends
                // (their barriers may miss other arrivals, so time stands in for them: about 30 ms)
                if (failed)
                    for (int k = 0; k < 30000; ++k) __nanosleep(1000);
            }
        } else {
        tile::Piece<DP> pk, pv;
        long long row = row_of(0, page_of(0));
        tile::load_piece<D, DP>(P.kc, P.ks, row, x0, W.bits_k, P.sfmt, P.lg_group, pk);
        tile::load_piece<D, DP>(P.vc, P.vs, row, x0, W.bits_v, P.sfmt, P.lg_group, pv);
        int next = page_of(1);
        for (int t = 0; t < n; ++t) {
            row = row_of(t + 1, next);
            next = page_of(t + 2);
            const int st = t & 1;
            if (t >= 2 && !wait(freed(S_DONE, t - 2), freed_parity(t - 2))) break;
            tile::unpack_scales(pk, P.sfmt);
            tile::store_piece_any<D, BN, DP>(smem + C::OFF_K + st * C::TB, r, x0, W.bits_k, lo, pk);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(k_bar(t)));
            tile::load_piece<D, DP>(P.kc, P.ks, row, x0, W.bits_k, P.sfmt, P.lg_group, pk);
            if (t >= 2 && !wait(freed(PV_DONE, t - 2), freed_parity(t - 2))) break;
            tile::unpack_scales(pv, P.sfmt);
            tile::store_piece_any<D, BN, DP>(smem + C::OFF_V + st * C::TB, r, x0, W.bits_v, lo, pv);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(bar(v_bar(t)));
                if (no_next_k(t)) ptx::mbar_arrive(bar(v_bar(t)));
            }
            tile::load_piece<D, DP>(P.vc, P.vs, row, x0, W.bits_v, P.sfmt, P.lg_group, pv);
        }
        }
        if (W.n_parts == 1 && !failed) {
            // R_s for the way back, where the K tiles were (d = 256: and the V tiles), once their last MMAs are done:
            // rows n of 64 inputs, the MN-major B operand
            // (with images only the fetching warp has followed the stages' phases)
            if (!W.images || warp == 8)
                for (int t = max(0, n - 2); t < n; ++t) {
                    wait(freed(S_DONE, t), freed_parity(t));
                    if (NQ == 1) wait(freed(PV_DONE, t), freed_parity(t));
                }
            if (W.images) ptx::named_bar_sync(1, 256);
            if (!failed) {
                for (int c = dt; c < D * (D / 8); c += 256) {
                    const int nr = c / (D / 8), ch = c % (D / 8);
                    uint4 hi, unused;
                    tile::r_chunk<D, false>(nr, 8 * ch, P.tr_v == SRFTKV_TRANSFORM_SRHT, tw, sg, hi, unused);
                    *reinterpret_cast<uint4*>(smem + C::OFF_K + (ch >> 3) * (D * 128) + nr * 128 +
                                              (((ch & 7) ^ (nr & 7)) << 4)) = hi;
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(R_FULL));
            }
        } else if (W.n_parts == 1 && W.images) {
            ptx::named_bar_sync(1, 256);  // (a warp whose wait ran out meets the others there all the same)
        }
        } else if (W.n_parts == 1 && W.images) {
            ptx::named_bar_sync(1, 256);
        }
    } else if (!failed && warp == 16) {
        // =========================== MMA ===========================
        const bool one = tile::elect();
        const uint32_t qd = tile::desc_k(sbase), kd = tile::desc_k(sbase + C::OFF_K),
                       vd = tile::desc_mn(sbase + C::OFF_V, BN * 128);
        auto issue_s = [&](int sb, int qt, int t) {
            const uint32_t ao = qd + qt * (C::QB / 16), bo = kd + (t & 1) * (C::TB / 16), dst = tmem + sb * C::S_STEP;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
                tc::mma_f16(dst, tile::desc(ao + (ks >> 2) * 1024 + (ks & 3) * 2), tile::desc(bo + (ks >> 2) * (BN * 8) + (ks & 3) * 2),
                            tile::idesc(128, BN, false), ks > 0);
        };
        auto issue_pv = [&](int sb, int oc, int t, bool first) {
            const uint32_t bo = vd + (t & 1) * (C::TB / 16), dst = tmem + C::O_COL + oc, pa = tmem + C::P_COL + sb * C::P_STEP;
#pragma unroll
            for (int ks = 0; ks < BN / 16; ++ks)
                tc::mma_f16_ta(dst, pa + 8 * ks, tile::desc(bo + ks * 128), tile::idesc(128, D, true), !(first && ks == 0));
        };
        auto ready = [&](int which, uint32_t parity) -> bool {
            if (__all_sync(0xffffffffu, ptx::mbar_test_bounded(bar(which), parity))) return true;
            failed = true;
            return false;
        };
        // S of stream i, step j (its K tile is there)
        auto start_s = [&](int i, int j) {
            const int t = dual ? 2 * j + i : j;
            if (t >= n) return;
            if (one) {
                issue_s(NQ == 2 ? i : (j & 1), dual ? 0 : i, t);
                tc::commit(bar(S_DONE + 2 * i + (j & 1)));
            }
            __syncwarp();
        };
        bool ok = ready(K_FIRST, 0) && (!(dual || NQ == 1) || n < 2 || ready(K_FIRST + 1, 0));
        if (ok) {
            tc::fence_after_sync();
            start_s(0, 0);
            if (NQ == 2) start_s(1, 0);
            else start_s(0, 1);
        }
        for (int j = 0; ok && j < steps_of(0); ++j)
            for (int i = 0; ok && i < NQ; ++i) {
                const int t = dual ? 2 * j + i : j;
                if (t >= n) continue;
                ok = ready(READY + 2 * i + (j & 1), (j >> 1) & 1);
                if (!ok) break;
                tc::fence_after_sync();
                if (one) {
                    issue_pv(NQ == 2 ? i : (j & 1), NQ == 2 ? i * D : 0, t, j == 0);
                    tc::commit(bar(PV_DONE + 2 * i + (j & 1)));
                }
                __syncwarp();
                start_s(i, j + AHEAD);
            }
        if (W.n_parts == 1 && !failed && wait(R_FULL, 0) && wait(EP_FULL, 0)) {
            tc::fence_after_sync();
            if (one) {
                const uint32_t bo = tile::desc_mn(sbase + C::OFF_K, D * 128);
                for (int i = 0; i < NQ; ++i)
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        tc::mma_f16(tmem + i * 128, tile::desc(qd + i * (C::QB / 16) + (ks >> 2) * 1024 + (ks & 3) * 2),
                                    tile::desc(bo + ks * 128), tile::idesc(128, D, true), ks > 0);
                tc::commit(bar(OUT_FULL));
            }
            __syncwarp();
        }
    }
    if (failed) atomicOr(P.fault, kFaultWait);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 16) tc::tmem_dealloc(tmem, 512);
}

template <int D>
static int launch_tile(const PagedAttnParams& P, const TileWork& W, int blocks, cudaStream_t stream) {
    using C = tile::Cfg<D>;
    // the registers the warps pass to each other are counted on kRegs at launch: another count would leave some waiting
    static std::atomic<int> regs{0};
    static std::atomic<unsigned long long> done{0}, done_expand{0};
    cudaError_t e = cudaSuccess;
    if (regs.load() == 0) {
        cudaFuncAttributes at;
        e = cudaFuncGetAttributes(&at, paged_attn_tile_kernel<D>);
        if (e == cudaSuccess) regs.store(at.numRegs);
    }
    if (e == cudaSuccess && C::NQ == 2 && (regs.load() + 7) / 8 * 8 != tile::kRegs) {
        set_error("paged attention: the tile kernel was built for %d registers a thread, not %d", regs.load(), tile::kRegs);
        return SRFTKV_ERR_CUDA;
    }
    if (e == cudaSuccess)
        e = allow_smem(done, reinterpret_cast<const void*>(paged_attn_tile_kernel<D>), C::SMEM);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        cfg.stream = stream;
        if (W.images) {
            cfg.gridDim = dim3(W.tiles, P.B * P.Hkv);
            cfg.blockDim = dim3(256);
            cfg.dynamicSmemBytes = 2 * C::TB + 1024;
            e = allow_smem(done_expand, reinterpret_cast<const void*>(paged_expand_kernel<D>), 2 * C::TB + 1024);
            if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, paged_expand_kernel<D>, P, W);
            // the tile kernel turns its q rows while the last tiles are laid down
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
        }
        cfg.gridDim = dim3(P.B * P.Hkv, blocks, W.n_splits);
        cfg.blockDim = dim3(tile::THREADS);
        cfg.dynamicSmemBytes = C::SMEM;
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, paged_attn_tile_kernel<D>, P, W);
    }
    if (e != cudaSuccess) {
        set_error("paged attention launch failed: %s", cudaGetErrorString(e));
        return SRFTKV_ERR_CUDA;
    }
    return SRFTKV_OK;
}

}  // namespace srftkv
