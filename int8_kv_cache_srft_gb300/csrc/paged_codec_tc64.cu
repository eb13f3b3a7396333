// paged_codec_tc64.cu -- the paged codec on the tensor cores at d = 64.
#include "paged_codec_tc.cuh"

namespace srftkv {
int launch_paged_codec_tc64(const PagedCodecParams& P, int dtype, bool write, cudaStream_t s) {
    return launch_codec_tc<64>(P, dtype, write, s);
}
}  // namespace srftkv
