// paged_attn_tile128.cu -- the paged attention's tile kernel at d = 128.
#include "paged_attn_tile.cuh"

namespace srftkv {
int launch_tile128(const PagedAttnParams& P, const TileWork& W, int blocks, cudaStream_t s) {
    return launch_tile<128>(P, W, blocks, s);
}
}  // namespace srftkv
