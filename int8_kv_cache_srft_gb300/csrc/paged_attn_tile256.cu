// paged_attn_tile256.cu -- the paged attention's tile kernel at d = 256.
#include "paged_attn_tile.cuh"

namespace srftkv {
int launch_tile256(const PagedAttnParams& P, const TileWork& W, int blocks, cudaStream_t s) {
    return launch_tile<256>(P, W, blocks, s);
}
}  // namespace srftkv
