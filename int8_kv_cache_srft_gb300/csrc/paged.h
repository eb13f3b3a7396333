// paged.h -- what the translation units of the paged cache share (the entry
// points srft_kv_quantize_paged, srft_kv_dequantize_paged and
// q4kv_paged_attention; layouts and rules in include/srftkv.h).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace srftkv {

// Bits of the paged kernels' fault words (srftkv_device_fault shifts them by 16).
constexpr unsigned int kFaultSlot = 1u, kFaultPage = 2u, kFaultWait = 4u;

struct PagedSideK {
    void* x;              // rows [n_tokens][H][d], token stride x_stride elements
    long long x_stride;
    uint8_t* codes;
    uint8_t* scales;
    const float* lambda;  // [H][d] or null
    int bits, transform, sfmt;
};

struct PagedCodecParams {
    PagedSideK side[2];
    int n_sides;
    const int64_t* slots;
    int n_tokens, H, group, lg_group, lg_page;
    uint32_t div_mul;     // division by H as a multiply and a shift (make_fastdiv)
    int div_shift;
    long long n_slots;    // n_pages * page_size
    unsigned int* fault;
    uint32_t sign_mask[128];
};

// A validated codec call; d and dtype choose the kernel.
struct PagedCodecCall {
    PagedCodecParams P;
    int d, dtype;
    cudaStream_t stream;
};
// Many rows on the tensor cores (paged_codec_tc.cuh); both sides of P share the transform
int launch_paged_codec_tc64(const PagedCodecParams& P, int dtype, bool write, cudaStream_t s);
int launch_paged_codec_tc128(const PagedCodecParams& P, int dtype, bool write, cudaStream_t s);
int launch_paged_codec_tc256(const PagedCodecParams& P, int dtype, bool write, cudaStream_t s);
int paged_quantize(const PagedCodecCall& c);
int paged_dequantize(const PagedCodecCall& c);
unsigned int paged_codec_take_fault();

struct PagedAttnParams {
    const void* q;
    void* out;
    long long q_stride, out_stride;
    const uint8_t *kc, *ks, *vc, *vs;
    const float *lam_k, *lam_v;
    const int *table, *seq_lens, *cu_q;
    int B, max_pages, total_q, max_q, max_len;
    int Hq, Hkv, rep, n_pages, lg_page, group, lg_group, sfmt;
    int tr_k, tr_v, window;
    float qscale;  // sm_scale * log2(e)
    unsigned int* fault;
    uint32_t sign_mask[128];
};
struct PagedAttnCall {
    PagedAttnParams P;
    int d, dtype, bits_k, bits_v;
    void* workspace;
    size_t workspace_bytes;
    cudaStream_t stream;
};
// What a launch of the tile kernel (paged_attn_tile.cuh) adds to the call's parameters
struct TileWork {
    int rows_per_block;  // 128 or 256
    int n_splits;        // ranges of the cache a block is split into
    int dual;            // both streams hold the same rows (d <= 128)
    int tps;             // tiles a split
    int n_parts;         // partial results a row: n_splits * (dual ? 2 : 1); 1: the kernel writes `out` itself
    int bits_k, bits_v, dtype;
    uint8_t* images;     // the tiles laid down as fp16, [B * Hkv][tiles][K, V], or null: turned where they are used
    int tiles;           // tiles of max_len
    float* part_ml;      // [total_q * Hq][n_parts][2]: m (log2 units), l
    float* part_acc;     // [total_q * Hq][n_parts][D]
};
int launch_tile64(const PagedAttnParams& P, const TileWork& W, int blocks, cudaStream_t s);
int launch_tile128(const PagedAttnParams& P, const TileWork& W, int blocks, cudaStream_t s);
int launch_tile256(const PagedAttnParams& P, const TileWork& W, int blocks, cudaStream_t s);
// The same for the split kernel (paged_attn_split.cuh)
struct SplitWork {
    int nr;        // groups of four query rows a CTA
    int groups;    // CTAs a (sequence, kv head, split): its rows / (4 nr)
    int n_splits, n_parts;
    int tokens;    // of a split, a multiple of 128
    int chunks;    // the same in chunks of the instance (set at its launch)
    int bits_k, bits_v, dtype;
    float* part_ml;
    float* part_acc;
};
int launch_split64_fp32(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s);
int launch_split64_fp16(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s);
int launch_split64_e8m0(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s);
int launch_split128_fp32(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s);
int launch_split128_fp16(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s);
int launch_split128_e8m0(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s);
int launch_split256_fp32(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s);
int launch_split256_fp16(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s);
int launch_split256_e8m0(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s);
size_t paged_attention_workspace(int d, int Hq, int Hkv, int B, int total_q, int max_q, int max_len, int window);
int paged_attention(const PagedAttnCall& c);
unsigned int paged_attn_take_fault();

}  // namespace srftkv
