// paged_codec_tc256.cu -- the paged codec on the tensor cores at d = 256.
#include "paged_codec_tc.cuh"

namespace srftkv {
int launch_paged_codec_tc256(const PagedCodecParams& P, int dtype, bool write, cudaStream_t s) {
    return launch_codec_tc<256>(P, dtype, write, s);
}
}  // namespace srftkv
