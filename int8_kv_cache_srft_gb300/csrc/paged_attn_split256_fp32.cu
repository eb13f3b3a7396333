// paged_attn_split256_fp32.cu -- the paged attention's split kernel at d = 256 with fp32 scales.
#include "paged_attn_split.cuh"

namespace srftkv {
int launch_split256_fp32(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s) {
    return launch_split<256, SRFTKV_SCALE_FP32>(P, W, s);
}
}  // namespace srftkv
