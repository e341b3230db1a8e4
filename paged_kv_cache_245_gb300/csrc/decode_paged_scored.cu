// decode_paged_scored.cu -- instantiations of the decode kernels with capped,
// biased and masked scores for the paged layout: small batches, where latency
// counts, and block sizes that are not multiples of 16.  Where the device holds
// them at once, a pair's splits are a cluster that joins them through
// distributed shared memory: one launch, no partials in memory.  One sequence of
// 1000 positions, 32 / 8 heads (16 CTAs a pair, a tile a warp): 7.3 us, 11.0 with
// the partials and their combine; its bytes take 0.6, the rest is the launch and
// the chain of context, table, rows and join.
#include "decode_launch.cuh"

namespace pkv {

cudaError_t launch_decode_paged_scored(const DecodeParams& p, int group, cudaStream_t stream) {
  return launch_decode<false, true>(p, group, stream);
}

cudaError_t room_decode_paged_scored(int group, ClusterRoom* out) {
  return decode_cluster_room<false>(group, out);
}

}  // namespace pkv
