// decode_paged_scored.cu -- instantiations of the decode kernels with capped,
// biased and masked scores for the paged layout.
#include "decode_launch.cuh"

namespace pkv {

cudaError_t launch_decode_paged_scored(const DecodeParams& p, int group, cudaStream_t stream) {
  return launch_decode<false, true>(p, group, stream);
}

}  // namespace pkv
