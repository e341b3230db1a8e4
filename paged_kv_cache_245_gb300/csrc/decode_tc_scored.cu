// decode_tc_scored.cu -- instantiations of the tensor-core decode kernel with
// capped, biased and masked scores.
#include "decode_tc_host.cuh"

namespace pkv {

cudaError_t launch_decode_tc_scored(const CUtensorMap& tk, const CUtensorMap& tv,
                                    const TcParams& p, bool contig, bool eight_heads,
                                    int num_ctas, cudaStream_t stream) {
  if (p.G > kTcHeads) return cudaErrorInvalidValue;
  if (eight_heads)
    return contig ? launch_cfg<true, 10, 2, false, 8, 1, true>(tk, tv, p, num_ctas, stream)
                  : launch_cfg<false, 10, 2, false, 8, 1, true>(tk, tv, p, num_ctas, stream);
  return contig ? launch_cfg<true, 12, 2, false, 4, 1, true>(tk, tv, p, num_ctas, stream)
                : launch_cfg<false, 12, 2, false, 4, 1, true>(tk, tv, p, num_ctas, stream);
}

}  // namespace pkv
