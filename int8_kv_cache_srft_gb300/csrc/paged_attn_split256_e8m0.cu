// paged_attn_split256_e8m0.cu -- the paged attention's split kernel at d = 256 with e8m0 scales.
#include "paged_attn_split.cuh"

namespace srftkv {
int launch_split256_e8m0(const PagedAttnParams& P, const SplitWork& W, cudaStream_t s) {
    return launch_split<256, SRFTKV_SCALE_E8M0>(P, W, s);
}
}  // namespace srftkv
