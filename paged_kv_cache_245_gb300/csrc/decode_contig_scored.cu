// decode_contig_scored.cu -- instantiations of the decode kernels with capped,
// biased and masked scores for the contiguous layout.
#include "decode_launch.cuh"

namespace pkv {

cudaError_t launch_decode_contig_scored(const DecodeParams& p, int group, cudaStream_t stream) {
  return launch_decode<true, true>(p, group, stream);
}

cudaError_t room_decode_contig_scored(int group, ClusterRoom* out) {
  return decode_cluster_room<true>(group, out);
}

}  // namespace pkv
