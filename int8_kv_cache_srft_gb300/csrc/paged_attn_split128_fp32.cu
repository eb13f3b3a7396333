// paged_attn_split128_fp32.cu -- the paged attention's split kernel at d = 128 with fp32 scales.
#include "paged_attn_split.cuh"

namespace srftkv {
int launch_split128_fp32(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s) {
    return launch_split<128, SRFTKV_SCALE_FP32>(P, W, s);
}
}  // namespace srftkv
