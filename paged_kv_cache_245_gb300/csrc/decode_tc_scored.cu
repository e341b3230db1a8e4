// decode_tc_scored.cu -- instantiations of the tensor-core decode kernel with
// capped, biased and masked scores, for long visible spans (decode_runs.cu: short
// ones).  The scores are capped, biased and masked on the accumulators, under the
// memory's time: 128 sequences of 8000 to 8192 positions in documents of about
// 6000, 56 / 8 heads, capped (1.84 GB): 270 us, 6.8 TB/s, 1.00 of a plain copy;
// 32 contiguous of 100 to 4095, 32 / 4 heads, with slopes (72 MB): 20.0 us, of
// which 10.6 are the bytes; the rest is the launch, the schedule (three dependent
// reads) and the pairs' merges.
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
