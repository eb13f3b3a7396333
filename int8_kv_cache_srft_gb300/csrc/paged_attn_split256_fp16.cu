// paged_attn_split256_fp16.cu -- the paged attention's split kernel at d = 256 with fp16 scales.
#include "paged_attn_split.cuh"

namespace srftkv {
int launch_split256_fp16(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s) {
    return launch_split<256, SRFTKV_SCALE_FP16>(P, W, s);
}
}  // namespace srftkv
