// paged_codec_tc.cuh -- writing and reading back many rows of the paged cache
// with the rotation as a contraction on the tensor cores (each d in its own
// translation unit).  One persistent CTA an SM walks tiles of 128 consecutive
// tokens of one (side, head); the heads of a token block are neighbouring
// tiles, so the SMs read and write whole tokens of x together.
//
//   write:  P = X . R_s^T (X exact; R_s as fp16 hi + lo beside fp16 rows, as three
//           bf16 parts beside bf16 rows), then lambda, group scales, rounding and
//           packing, one thread a row and 32 columns
//   read:   X = P . R_s, P = code * scale / lambda rounded to fp16 once
//
// Warps (8 and 16, or 16 and 8): some bring a tile in (write: 16-bit rows,
// coalesced; read: codes and scales turned into P) and lay it down as the swizzled
// A operand; the last issues the MMAs into a ring of accumulators; the others take
// them out.
//
// At d = 256 three parts of R_s do not fit: there bf16 rows go over to fp16, as
// they are where their largest value lies in [2^-6, 2^15), else multiplied by the
// power of two that brings it to [1, 2); the epilogue multiplies it back in.
//
// What bounds it: the bytes of x (2 d a vector) and of the rows (d b / 8 + scales),
// and near it the instructions of both ends (issue 58 % busy writing, 43 % reading).
// 2 M rows at d = 128, 4-bit codes: written in 130 us from fp16 (5.7 TB/s, 84 % of the
// copy rate), 138 from bf16, read back in 180 (4.0 TB/s); d = 64: 75, 74 and 115.
// 1 M rows at d = 256: 293, 372 (converted rows) and 230.
#pragma once

#include "codec_impl.cuh"
#include "paged_attn_tile.cuh"

namespace srftkv {

namespace ctc {

// The write holds R_s times 2^8: its residual lo (2^-12 of entries near sqrt(2/d)) is then a normal fp16 number, and
// P is good to about 2^-23 of the row; codes of 8 bits turn on 2^-20 of a group's largest value.
constexpr int kUp = 8;

template <int D, bool WRITE, int DT>
struct Cfg {
    // rows of bf16 against three bf16 parts of R_s (24 bits), nothing to convert (d = 128, 2 M rows: 197 us converted)
    static constexpr bool BF = WRITE && DT == SRFTKV_DTYPE_BF16 && D <= 128;
    static constexpr int PARTS = !WRITE ? 1 : BF ? 3 : 2, UP = WRITE && !BF ? kUp : 0;
    // Warps that bring tiles in, and that take them out: the heavier end of each direction gets sixteen (with eight at
    // both ends a tile took 2 us of dependent instructions, whatever the memory did); but for the write at d = 256,
    // where a tile waits in the loaders' registers and 25 warps leave too few
    static constexpr int NL = WRITE || D < 256 ? 8 : 16, NE = D < 256 ? 16 : 8, THREADS = (NL + NE + 1) * 32, MMA = NL + NE;
    static constexpr int NB = WRITE && D == 256 ? 128 : D;  // output columns a CTA (d = 256: half of them)
    static constexpr int NSPLIT = D / NB;
    static constexpr int B_BYTES = NB * D * 2 * PARTS;
    static constexpr int A_BYTES = 128 * D * 2;
    // A stages.  d <= 128: the write's copies land in them PD tiles ahead; the read's raw bytes wait in a ring of
    // their own, PD tiles ahead, 16 bytes a thread and step.  d = 256 has room for one stage, and a tile waits in
    // registers.
    static constexpr bool AHEAD = D <= 128;
    static constexpr int ST = !AHEAD ? 1 : WRITE && !(BF && D == 128) ? 4 : 3, PD = 2;
    static constexpr int NACC = WRITE || D < 256 ? 4 : 2;       // accumulators of NB columns
    static constexpr int TPR = NL / 4;                          // read: threads a row
    static constexpr int RAW16 = D / (16 * TPR) + 1;            // 16-byte pieces a thread (8-bit codes; scales last)
    static constexpr int RAW = AHEAD && !WRITE ? RAW16 * NL * 512 : 0;
    static constexpr int OFF_A = B_BYTES;
    static constexpr int OFF_RAW = OFF_A + ST * A_BYTES;
    static constexpr int OFF_TW = OFF_RAW + PD * RAW;
    static constexpr int OFF_SG = OFF_TW + D * 8;
    static constexpr int OFF_RF = OFF_SG + D * 2;      // write of converted bf16 rows: 2^e of the rows of eight tiles
    static constexpr int OFF_OUT = OFF_RF + (WRITE && !BF ? 8 * 128 * 4 : 0);  // read: 32 rows of 64 bytes for each epilogue warp
    static constexpr int OFF_BAR = OFF_OUT + (WRITE ? 0 : NE * 2048);
    static constexpr int USED = OFF_BAR + 256;
    static constexpr int SMEM = (USED > 120 * 1024 ? USED : 120 * 1024) + 1024;
    static_assert(SMEM <= 232448, "shared memory");
};

// n (at most B) bytes from global memory to shared memory and zeros behind them
template <int B>
__device__ __forceinline__ void copy(uint32_t dst, const void* src, int n) {
    if constexpr (B == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else if constexpr (B == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

struct Tile {
    int side, h, t0;
};
__device__ __forceinline__ Tile tile_at(const PagedCodecParams& P, int u, int per_side) {
    Tile t;
    t.side = u >= per_side;
    const int r = u - (t.side ? per_side : 0);
    const int tb = (int)((__umulhi((uint32_t)r, P.div_mul) + (uint32_t)r) >> P.div_shift);  // r / H
    t.h = r - tb * P.H;
    t.t0 = tb * 128;
    return t;
}
// Token t's slot as it stands in the list (-1 past the call's tokens).  Looked up a tile ahead and not looked at until
// then: a check beside the load holds the warp for the load's latency, once a tile.
__device__ __forceinline__ long long slot_of(const PagedCodecParams& P, int t) {
    return t < P.n_tokens ? __ldg(P.slots + t) : -1;
}
// its packed row in head h, or -1 (padding, outside the pool)
__device__ __forceinline__ long long row_of(const PagedCodecParams& P, long long slot, int h) {
    if (slot < 0) return -1;
    if (slot >= P.n_slots) {
        atomicOr(P.fault, kFaultSlot);
        return -1;
    }
    return ((slot >> P.lg_page) * P.H + h) << P.lg_page | (slot & ((1ll << P.lg_page) - 1));
}

}  // namespace ctc

// The parts both directions share: barriers, tensor memory, R_s.  BODY: see the two kernels.
template <int D, bool WRITE, int DT>
struct CtcCommon {
    using C = ctc::Cfg<D, WRITE, DT>;
    static constexpr int A_FULL = 0, A_EMPTY = C::ST, ACC_FULL = 2 * C::ST, ACC_EMPTY = 2 * C::ST + C::NACC,
                         N_BARS = 2 * C::ST + 2 * C::NACC;

    // R_s rows: write [n][x] in its parts (K-major B: rows are the outputs n0 .. n0 + NB - 1); read [n][x] with the
    // rows in the order of dq_kperm (MN-major B: rows are the contraction index)
    static __device__ void setup(uint8_t* smem, uint64_t* bars, uint32_t* slot, int warp, const uint32_t* sign, bool srht,
                                 int n0) {
        float2* tw = reinterpret_cast<float2*>(smem + C::OFF_TW);
        uint32_t* sg = reinterpret_cast<uint32_t*>(smem + C::OFF_SG);
        if (threadIdx.x == 0) {
            for (int i = 0; i < C::ST; ++i) {
                ptx::mbar_init(ptx::smem_u32(&bars[A_FULL + i]), C::NL);
                ptx::mbar_init(ptx::smem_u32(&bars[A_EMPTY + i]), 1);
            }
            for (int i = 0; i < C::NACC; ++i) {
                ptx::mbar_init(ptx::smem_u32(&bars[ACC_FULL + i]), 1);
                ptx::mbar_init(ptx::smem_u32(&bars[ACC_EMPTY + i]), WRITE ? 4 * (C::NB / 32) : 8);
            }
            ptx::fence_barrier_init();
        }
        if (warp == C::MMA) {
            tc::tmem_alloc(ptx::smem_u32(slot), 512);
            tc::tmem_relinquish();
        }
        for (int m = threadIdx.x; m < D; m += blockDim.x)
            tw[m] = make_float2(tw_re_lane(m * (256 / D)), tw_im_lane(m * (256 / D)));
        for (int i = threadIdx.x; i < D / 2; i += blockDim.x) sg[i] = sign[i];
        tc::fence_before_sync();
        __syncthreads();
        tc::fence_after_sync();
        constexpr int ROWS = WRITE ? C::NB : D;
        for (int c = threadIdx.x; c < ROWS * (D / 8); c += blockDim.x) {
            const int r = c / (D / 8), ch = c % (D / 8);
            uint8_t* at = smem + (ch >> 3) * (ROWS * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
            if constexpr (C::BF) {
                float f[8];
                tile::r_entries<D, 0>(n0 + r, 8 * ch, srht, tw, sg, f);
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
                        w[j] = *reinterpret_cast<const uint32_t*>(&b);
                        f[2 * j] -= __uint_as_float(w[j] << 16);
                        f[2 * j + 1] -= __uint_as_float(w[j] & 0xFFFF0000u);
                    }
                    *reinterpret_cast<uint4*>(at + k * ROWS * D * 2) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else {
                uint4 hi, lo;
                tile::r_chunk<D, WRITE, C::UP>(WRITE ? n0 + r : dq_kperm(r), 8 * ch, srht, tw, sg, hi, lo);
                *reinterpret_cast<uint4*>(at) = hi;
                if constexpr (WRITE) *reinterpret_cast<uint4*>(at + ROWS * D * 2) = lo;
            }
        }
        ptx::fence_proxy_async_smem();
        __syncthreads();
    }
};

// DT: SRFTKV_DTYPE_*
template <int D, int DT>
__global__ void __launch_bounds__(ctc::Cfg<D, true, DT>::THREADS, 1) paged_quantize_tc_kernel(const __grid_constant__ PagedCodecParams P) {
    using S = CtcCommon<D, true, DT>;
    constexpr bool CONVERT = DT == SRFTKV_DTYPE_BF16 && !S::C::BF;  // bf16 rows go over to fp16
    using C = typename S::C;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    auto bar = [&](int i) { return ptx::smem_u32(&bars[i]); };
    uint32_t* slot = reinterpret_cast<uint32_t*>(&bars[S::N_BARS]);
    float* rf = reinterpret_cast<float*>(smem + C::OFF_RF);
    const int half = blockIdx.x % C::NSPLIT, first = blockIdx.x / C::NSPLIT, step = gridDim.x / C::NSPLIT;
    const int per_side = (P.n_tokens + 127) / 128 * P.H, total = per_side * P.n_sides;
    S::setup(smem, bars, slot, warp, P.sign_mask, P.side[0].transform == SRFTKV_TRANSFORM_SRHT, half * C::NB);
    const uint32_t tmem = *slot;
    bool failed = false;

    if (warp < C::NL) {
        // 16 rows a warp; a step covers 32 / (D / 8) rows, 16 bytes a lane; each lane lays down, and in the bf16 case
        // later converts in place, its own pieces
        constexpr int LPR = D / 8, RPS = LPR >= 32 ? 1 : 32 / LPR, NI = 16 * LPR / 32, PD = C::PD;
        const int ch = lane % LPR;
        uint4 v[C::AHEAD ? 1 : NI];
        auto piece = [&](int s, int r) -> uint32_t {
            return C::OFF_A + s * C::A_BYTES + (ch >> 3) * 16384 + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
        };
        auto load = [&](int u, int s) {
            if (u < total) {
                const ctc::Tile t = ctc::tile_at(P, u, per_side);
                const PagedSideK& sd = P.side[t.side];
                const uint16_t* x = static_cast<const uint16_t*>(sd.x) + (long long)t.h * D + ch * 8;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int r = 16 * warp + i * RPS + lane / LPR, tok = t.t0 + r;
                    const bool in = tok < P.n_tokens;
                    if constexpr (C::AHEAD)
                        ctc::copy<16>(sbase + piece(s, r), x + (in ? tok : 0) * sd.x_stride, in ? 16 : 0);
                    else
                        v[i] = in ? __ldg(reinterpret_cast<const uint4*>(x + tok * sd.x_stride)) : make_uint4(0, 0, 0, 0);
                }
            }
            if constexpr (C::AHEAD) ctc::commit_copies();
        };
#pragma unroll
        for (int j = 0; j < (C::AHEAD ? PD : 1); ++j) load(first + j * step, j);
        auto empty = [&](int tile) -> bool {  // the stage of this CTA's tile number `tile` has been read
            if (tile < C::ST) return true;
            return __all_sync(0xffffffffu, ptx::mbar_spin_bounded(bar(S::A_EMPTY + tile % C::ST), (tile / C::ST - 1) & 1));
        };
        int i_tile = 0;
        for (int u = first; u < total; u += step, ++i_tile) {
            const int s = i_tile % C::ST;
            if constexpr (C::AHEAD) ctc::wait_copies<PD - 1>();
            else if (!empty(i_tile)) {
                failed = true;
                break;
            }
            if constexpr (!C::AHEAD || CONVERT) {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int r = 16 * warp + i * RPS + lane / LPR;
                    uint4* at = reinterpret_cast<uint4*>(smem + piece(s, r));
                    const uint4 q = C::AHEAD ? *at : v[C::AHEAD ? 0 : i];
                    uint32_t w[4] = {q.x, q.y, q.z, q.w};
                    if constexpr (CONVERT) {
                        // exponents of this lane's values, two a word; rows whose largest lies in [2^-6, 2^15) go over as
                        // they are (an error of 2^-25 at most), others by the power of two that brings it to [1, 2)
                        uint32_t m2 = 0;
#pragma unroll
                        for (int j = 0; j < 4; ++j) m2 = __vmaxu2(m2, w[j] & 0x7F807F80u);
                        const uint32_t me = max(m2 & 0xFFFFu, m2 >> 16) >> 7;
                        const uint32_t big = __ballot_sync(0xffffffffu, me >= 127 - 6), huge = __ballot_sync(0xffffffffu, me >= 127 + 15);
                        bool fine = huge == 0;
#pragma unroll
                        for (int k = 0; k < 32 / LPR; ++k) fine &= (big & ((uint32_t)((1ull << LPR) - 1) << (k * LPR))) != 0;
                        float up = 1.f, down = 1.f;
                        if (!fine) {
                            uint32_t m = me;
#pragma unroll
                            for (int k = 1; k < LPR; k <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, k));
                            const int e = min(max((int)m, 1), 253);  // (rows of zeros; the last binade lands in [2, 4))
                            up = __uint_as_float((uint32_t)(254 - e) << 23);  // 2^(127 - e)
                            down = __uint_as_float((uint32_t)e << 23);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = pack_half2(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xFFFF0000u) * up);
                        if (ch == 0) rf[(i_tile & 7) * 128 + r] = down;
                    }
                    *at = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(S::A_FULL + s));
            if constexpr (C::AHEAD) {
                if (u + PD * step < total && !empty(i_tile + PD)) {
                    failed = true;
                    break;
                }
                load(u + PD * step, (i_tile + PD) % C::ST);
            } else {
                load(u + step, 0);
            }
        }
        if constexpr (C::AHEAD) ctc::wait_copies<0>();  // (after a wait that ran out some are under way)
    } else if (warp < C::MMA) {
        // a warp: lanes 32 quarter .., a unit of 32 columns or more of them in turn; where a tile has fewer units than
        // there are warps, those left over take every other tile
        constexpr int UNITS = C::NB / 32, PER = C::NE / 4, GROUPS = PER > UNITS ? PER / UNITS : 1;
        const int quarter = warp & 3, unit = ((warp - C::NL) >> 2) % UNITS, group = ((warp - C::NL) >> 2) / UNITS;
        auto slot_at = [&](int u) { return u < total ? ctc::slot_of(P, ctc::tile_at(P, u, per_side).t0 + 32 * quarter + lane) : -1ll; };
        int i_tile = group;
        long long next = slot_at(first + group * step);
        for (int u = first + group * step; u < total; u += GROUPS * step, i_tile += GROUPS) {
            const int a = i_tile % C::NACC;
            const ctc::Tile t = ctc::tile_at(P, u, per_side);
            const PagedSideK& sd = P.side[t.side];
            const int r = 32 * quarter + lane;
            const long long row = ctc::row_of(P, next, t.h);
            next = slot_at(u + GROUPS * step);
            if (!__all_sync(0xffffffffu, ptx::mbar_spin_bounded(bar(S::ACC_FULL + a), (i_tile / C::NACC) & 1))) {
                failed = true;
                break;
            }
            tc::fence_after_sync();
            const float up = CONVERT ? rf[(i_tile & 7) * 128 + r] : 1.f;
#pragma unroll 1
            for (int c0 = 32 * unit; c0 < C::NB; c0 += 32 * (PER < UNITS ? PER : UNITS)) {
                uint32_t raw[32];
                tc::ld_32x32b_x32(tmem + ((uint32_t)(32 * quarter) << 16) + a * C::NB + c0, raw);
                tc::wait_ld(raw);
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(S::ACC_EMPTY + a));
                if (row >= 0) {
                    const int col = half * C::NB + c0;
                    float z[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(raw[j]);
                    if (CONVERT && up != 1.f) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) z[j] *= up;
                    }
                    if (sd.lambda != nullptr) {
                        const float4* l = reinterpret_cast<const float4*>(sd.lambda + (long long)t.h * D + col);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 f = __ldg(l + j);
                            z[4 * j] *= f.x, z[4 * j + 1] *= f.y, z[4 * j + 2] *= f.z, z[4 * j + 3] *= f.w;
                        }
                    }
                    const int ng = D >> P.lg_group, sb = sd.sfmt == SRFTKV_SCALE_FP32 ? 4 : sd.sfmt == SRFTKV_SCALE_FP16 ? 2 : 1;
                    uint8_t* srow = sd.scales + (row * ng + (col >> P.lg_group)) * sb;
                    uint8_t* crow = sd.codes + row * (D * sd.bits / 8) + col * sd.bits / 8;
                    auto put = [&](auto bits) {
                        constexpr int B = decltype(bits)::value;
                        if (sd.sfmt == SRFTKV_SCALE_FP32) quant_store_row<32, B, SRFTKV_SCALE_FP32, C::UP>(z, P.group, crow, srow);
                        else if (sd.sfmt == SRFTKV_SCALE_FP16) quant_store_row<32, B, SRFTKV_SCALE_FP16, C::UP>(z, P.group, crow, srow);
                        else quant_store_row<32, B, SRFTKV_SCALE_E8M0, C::UP>(z, P.group, crow, srow);
                    };
                    if (sd.bits == 4) put(std::integral_constant<int, 4>{});
                    else put(std::integral_constant<int, 8>{});
                }
                __syncwarp();
            }
        }
    } else {
        const bool one = tile::elect();
        int i_tile = 0;
        for (int u = first; u < total; u += step, ++i_tile) {
            const int s = i_tile % C::ST, a = i_tile % C::NACC;
            if (!__all_sync(0xffffffffu, ptx::mbar_spin_bounded(bar(S::A_FULL + s), (i_tile / C::ST) & 1)) ||
                (i_tile >= C::NACC &&
                 !__all_sync(0xffffffffu, ptx::mbar_spin_bounded(bar(S::ACC_EMPTY + a), (i_tile / C::NACC - 1) & 1)))) {
                failed = true;
                break;
            }
            tc::fence_after_sync();
            if (one) {
                const uint32_t ao = tile::desc_k(sbase + C::OFF_A + s * C::A_BYTES), bo = tile::desc_k(sbase), dst = tmem + a * C::NB;
                // the smallest part first: an accumulation rounds to the size of the sum so far, which that leaves small,
                // so only the D/16 steps of the largest count
                constexpr uint32_t idesc = tile::idesc(128, C::NB, false) | (C::BF ? 1u << 7 | 1u << 10 : 0u);  // (A, B bf16)
#pragma unroll
                for (int ks = 0; ks < C::PARTS * (D / 16); ++ks) {
                    const int k = ks % (D / 16), part = C::PARTS - 1 - ks / (D / 16);
                    const uint32_t as = (k >> 2) * 1024 + (k & 3) * 2, bs = (k >> 2) * (C::NB * 8) + (k & 3) * 2;
                    tc::mma_f16(dst, tile::desc(ao + as), tile::desc(bo + bs + part * (C::NB * D / 8)), idesc, ks > 0);
                }
                tc::commit(bar(S::A_EMPTY + s));
                tc::commit(bar(S::ACC_FULL + a));
            }
            __syncwarp();
        }
    }
    if (failed) atomicOr(P.fault, kFaultWait);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == C::MMA) tc::tmem_dealloc(tmem, 512);
}

template <int D, int DT>
__global__ void __launch_bounds__(ctc::Cfg<D, false, DT>::THREADS, 1) paged_dequantize_tc_kernel(const __grid_constant__ PagedCodecParams P) {
    using S = CtcCommon<D, false, DT>;
    using C = typename S::C;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sbase = ptx::smem_u32(smem);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    auto bar = [&](int i) { return ptx::smem_u32(&bars[i]); };
    uint32_t* slot = reinterpret_cast<uint32_t*>(&bars[S::N_BARS]);
    const int first = blockIdx.x, step = gridDim.x;
    const int per_side = (P.n_tokens + 127) / 128 * P.H, total = per_side * P.n_sides;
    S::setup(smem, bars, slot, warp, P.sign_mask, P.side[0].transform == SRFTKV_TRANSFORM_SRHT, 0);
    const uint32_t tmem = *slot;
    bool failed = false;

    if (warp < C::NL) {
        // TPR threads a row, DP coordinates each
        constexpr int DP = D / C::TPR, PD = C::PD, U = DP / 16;
        const int r = threadIdx.x / C::TPR, x0 = (threadIdx.x % C::TPR) * DP;
        tile::Piece<DP> p;
        auto slot_at = [&](int u) { return u < total ? ctc::slot_of(P, ctc::tile_at(P, u, per_side).t0 + r) : -1ll; };
        const int ng = D >> P.lg_group;
        auto raw = [&](int q, int i) { return (uint32_t)(C::OFF_RAW + q * C::RAW + (i * C::NL * 32 + (int)threadIdx.x) * 16); };
        auto load = [&](int u, int q, long long slot) {  // into the raw ring (or registers)
            if (u < total) {
                const long long row = ctc::row_of(P, slot, ctc::tile_at(P, u, per_side).h);
                const PagedSideK& sd = P.side[u >= per_side];
                if constexpr (C::AHEAD) {
                    const int n = row < 0 ? 0 : 16;
                    const long long at = row < 0 ? 0 : row;
                    const uint8_t* c = sd.codes + (at * D + x0) * sd.bits / 8;
#pragma unroll
                    for (int i = 0; i < C::RAW16 - 1; ++i)
                        if (i < (C::RAW16 - 1) * sd.bits / 8) ctc::copy<16>(sbase + raw(q, i), c + 16 * i, n);
                    const int sb = sd.sfmt == SRFTKV_SCALE_FP32 ? 4 : sd.sfmt == SRFTKV_SCALE_FP16 ? 2 : 1;
#pragma unroll
                    for (int i = 0; i < U; ++i)  // the aligned word that holds the unit's scale
                        ctc::copy<4>(sbase + raw(q, C::RAW16 - 1) + 4 * i,
                                     sd.scales + (((at * ng + ((x0 + 16 * i) >> P.lg_group)) * sb) & ~3ll), n / 4);
                } else {
                    tile::load_piece<D, DP>(sd.codes, sd.scales, row, x0, sd.bits, sd.sfmt, P.lg_group, p);
                }
            }
            if constexpr (C::AHEAD) ctc::commit_copies();
        };
        auto unload = [&](int u, int q) {  // this thread's piece out of the raw ring
            if constexpr (C::AHEAD) {
                const PagedSideK& sd = P.side[u >= per_side];
#pragma unroll
                for (int i = 0; i < C::RAW16 - 1; ++i)
                    if (i < (C::RAW16 - 1) * sd.bits / 8) {
                        const uint4 t = *reinterpret_cast<const uint4*>(smem + raw(q, i));
                        p.w[4 * i] = t.x, p.w[4 * i + 1] = t.y, p.w[4 * i + 2] = t.z, p.w[4 * i + 3] = t.w;
                    }
                // where the scale lies in its word: rows of 1 or 2 scales shift with the row (its slot's low bits)
                int low = 0;
                if (ng < 4) {
                    const int tok = ctc::tile_at(P, u, per_side).t0 + r;
                    low = tok < P.n_tokens ? (int)__ldg(P.slots + tok) * ng : 0;
                }
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const uint32_t w = *reinterpret_cast<const uint32_t*>(smem + raw(q, C::RAW16 - 1) + 4 * i);
                    const int at = low + ((x0 + 16 * i) >> P.lg_group);
                    if (sd.sfmt == SRFTKV_SCALE_FP32) p.sc[i] = __uint_as_float(w);
                    else if (sd.sfmt == SRFTKV_SCALE_FP16)
                        p.sc[i] = __half2float(__ushort_as_half((unsigned short)(w >> (16 * (at & 1)))));
                    else p.sc[i] = __uint_as_float(((w >> (8 * (at & 3))) & 0xFFu) << 23);
                }
            }
        };
#pragma unroll
        for (int j = 0; j < (C::AHEAD ? PD : 1); ++j) load(first + j * step, j, slot_at(first + j * step));
        constexpr int NEXT = C::AHEAD ? PD : 1;
        long long next = slot_at(first + NEXT * step);
        int i_tile = 0;
        for (int u = first; u < total; u += step, ++i_tile) {
            const int s = i_tile % C::ST, use = i_tile / C::ST;
            if constexpr (C::AHEAD) {
                ctc::wait_copies<PD - 1>();
                unload(u, i_tile % PD);
                load(u + PD * step, i_tile % PD, next);  // (the pieces are this thread's own: read before they are replaced)
                next = slot_at(u + (PD + 1) * step);
            }
            if (use > 0 && !__all_sync(0xffffffffu, ptx::mbar_spin_bounded(bar(S::A_EMPTY + s), (use - 1) & 1))) {
                failed = true;
                break;
            }
            uint8_t* a = smem + C::OFF_A + s * C::A_BYTES;
            const PagedSideK& sd = P.side[u >= per_side];
            if constexpr (!C::AHEAD) tile::unpack_scales(p, sd.sfmt);
            if (sd.lambda == nullptr) {
                tile::store_piece_any<D, 128, DP>(a, r, x0, sd.bits, sd.sfmt == SRFTKV_SCALE_FP32, p);
            } else {
                const float* lam = sd.lambda + (long long)ctc::tile_at(P, u, per_side).h * D + x0;
#pragma unroll
                for (int g = 0; g < DP / 8; ++g) {  // eight coordinates, in the order of dq_kperm
                    float f[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t w = sd.bits == 4 ? p.w[g] : p.w[(2 * g + (j >> 2)) % (DP / 4)];
                        const int sh = sd.bits == 4 ? 28 - 4 * j : 24 - 8 * (j & 3);
                        const int c = (int)(w << sh) >> (sd.bits == 4 ? 28 : 24);
                        f[j] = __fdiv_rn((float)c * p.sc[g >> 1], __ldg(lam + 8 * g + j));
                    }
                    const int x = x0 + 8 * g;
                    *reinterpret_cast<uint4*>(a + (x >> 6) * 16384 + r * 128 + ((((x & 63) >> 3) ^ (r & 7)) << 4)) =
                        make_uint4(pack_half2(f[0], f[4]), pack_half2(f[1], f[5]), pack_half2(f[2], f[6]),
                                   pack_half2(f[3], f[7]));
                }
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(S::A_FULL + s));
            if constexpr (!C::AHEAD) {
                load(u + step, 0, next);
                next = slot_at(u + 2 * step);
            }
        }
        if constexpr (C::AHEAD) ctc::wait_copies<0>();
    } else if (warp < C::MMA) {
        // a warp: lanes 32 quarter .., half the columns, of every GROUPSth tile
        constexpr int GROUPS = C::NE / 8;
        const int quarter = warp & 3, c0 = (((warp - C::NL) >> 2) & 1) * (D / 2), group = (warp - C::NL) >> 3;
        uint8_t* stage = smem + C::OFF_OUT + (warp - C::NL) * 2048;
        auto slot_at = [&](int u) { return u < total ? ctc::slot_of(P, ctc::tile_at(P, u, per_side).t0 + 32 * quarter + lane) : -1ll; };
        int i_tile = group;
        long long next = slot_at(first + group * step);
        for (int u = first + group * step; u < total; u += GROUPS * step, i_tile += GROUPS) {
            const int a = i_tile % C::NACC;
            const ctc::Tile t = ctc::tile_at(P, u, per_side);
            const PagedSideK& sd = P.side[t.side];
            const uint32_t rows = __ballot_sync(0xffffffffu, ctc::row_of(P, next, t.h) >= 0);
            next = slot_at(u + GROUPS * step);
            // this lane's place in the coalesced stores: 16-byte piece lane % 4 of rows lane / 4 + 8 j
            uint16_t* x = static_cast<uint16_t*>(sd.x) + (long long)(t.t0 + 32 * quarter + (lane >> 2)) * sd.x_stride +
                          (long long)t.h * D + c0 + 8 * (lane & 3);
            if (!__all_sync(0xffffffffu, ptx::mbar_spin_bounded(bar(S::ACC_FULL + a), (i_tile / C::NACC) & 1))) {
                failed = true;
                break;
            }
            tc::fence_after_sync();
#pragma unroll 1
            for (int k = 0; k < D / 64; ++k) {
                uint32_t v[32], w[16];
                tc::ld_32x32b_x32(tmem + ((uint32_t)(32 * quarter) << 16) + a * D + c0 + 32 * k, v);
                tc::wait_ld(v);
                if (k == D / 64 - 1) {
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(bar(S::ACC_EMPTY + a));
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    if constexpr (DT == SRFTKV_DTYPE_BF16) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                        w[e] = *reinterpret_cast<const uint32_t*>(&b);
                    } else {
                        w[e] = pack_half2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                    }
                }
                // a row's 64 bytes go through shared memory, so that four lanes store them together (a lane storing
                // its own row touched 32 lines an instruction, and the stores were what bounded the kernel)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ ((lane >> 1) & 3)) << 4)) =
                        make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = (lane >> 2) + 8 * j;
                    const uint4 o = *reinterpret_cast<const uint4*>(stage + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
                    if ((rows >> row) & 1) *reinterpret_cast<uint4*>(x + 8ll * j * sd.x_stride + 32 * k) = o;
                }
                __syncwarp();
            }
        }
    } else {
        const bool one = tile::elect();
        int i_tile = 0;
        for (int u = first; u < total; u += step, ++i_tile) {
            const int s = i_tile % C::ST, a = i_tile % C::NACC;
            if (!__all_sync(0xffffffffu, ptx::mbar_spin_bounded(bar(S::A_FULL + s), (i_tile / C::ST) & 1)) ||
                (i_tile >= C::NACC &&
                 !__all_sync(0xffffffffu, ptx::mbar_spin_bounded(bar(S::ACC_EMPTY + a), (i_tile / C::NACC - 1) & 1)))) {
                failed = true;
                break;
            }
            tc::fence_after_sync();
            if (one) {
                const uint32_t ao = tile::desc_k(sbase + C::OFF_A + s * C::A_BYTES), bo = tile::desc_mn(sbase, D * 128);
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc::mma_f16(tmem + a * D, tile::desc(ao + (ks >> 2) * 1024 + (ks & 3) * 2), tile::desc(bo + ks * 128),
                                tile::idesc(128, D, true), ks > 0);
                tc::commit(bar(S::A_EMPTY + s));
                tc::commit(bar(S::ACC_FULL + a));
            }
            __syncwarp();
        }
    }
    if (failed) atomicOr(P.fault, kFaultWait);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == C::MMA) tc::tmem_dealloc(tmem, 512);
}

template <int D>
static int launch_codec_tc(const PagedCodecParams& P, int dtype, bool write, cudaStream_t stream) {
    using CW = ctc::Cfg<D, true, SRFTKV_DTYPE_FP16>;
    using CB = ctc::Cfg<D, true, SRFTKV_DTYPE_BF16>;
    using CR = ctc::Cfg<D, false, SRFTKV_DTYPE_FP16>;
    void (*k)(PagedCodecParams) =
        write ? (dtype == SRFTKV_DTYPE_BF16 ? paged_quantize_tc_kernel<D, SRFTKV_DTYPE_BF16> : paged_quantize_tc_kernel<D, SRFTKV_DTYPE_FP16>)
              : (dtype == SRFTKV_DTYPE_BF16 ? paged_dequantize_tc_kernel<D, SRFTKV_DTYPE_BF16> : paged_dequantize_tc_kernel<D, SRFTKV_DTYPE_FP16>);
    const int smem = !write ? CR::SMEM : dtype == SRFTKV_DTYPE_BF16 ? CB::SMEM : CW::SMEM, split = write ? CW::NSPLIT : 1;
    const int total = (P.n_tokens + 127) / 128 * P.H * P.n_sides, sms = device_sm_count();
    const int ctas = total < sms / split ? total : sms / split;
    static std::atomic<unsigned long long> done[4];
    cudaError_t e = allow_smem(done[2 * write + (dtype == SRFTKV_DTYPE_BF16)], reinterpret_cast<const void*>(k), smem);
    if (e == cudaSuccess) {
        k<<<ctas * split, write ? CW::THREADS : CR::THREADS, smem, stream>>>(P);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess) {
        set_error("paged codec launch failed: %s", cudaGetErrorString(e));
        return SRFTKV_ERR_CUDA;
    }
    return SRFTKV_OK;
}

}  // namespace srftkv
