// paged_attn_tile64.cu -- the paged attention's tile kernel at d = 64.
#include "paged_attn_tile.cuh"

namespace srftkv {
int launch_tile64(const PagedAttnParams& P, const TileWork& W, int blocks, cudaStream_t s) {
    return launch_tile<64>(P, W, blocks, s);
}
}  // namespace srftkv
