// decode_paged_scored.cu -- instantiations of the decode kernels with capped,
// biased and masked scores for the paged layout: small batches, where latency
// counts (one sequence of 1000 positions, 32 / 8 heads: 11.0 us, two launches and
// their chains of dependent reads; its bytes take 0.6), and block sizes that are
// not multiples of 16.
#include "decode_launch.cuh"

namespace pkv {

cudaError_t launch_decode_paged_scored(const DecodeParams& p, int group, cudaStream_t stream) {
  return launch_decode<false, true>(p, group, stream);
}

}  // namespace pkv
