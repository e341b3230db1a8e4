// prefill_scored.cu -- the prefill kernel with capped, biased and masked scores.
#include "prefill_kernel.cuh"

namespace pkv {

cudaError_t launch_prefill_scored(const CUtensorMap& tk, const CUtensorMap& tv,
                                  const CUtensorMap& tq, const CUtensorMap& to,
                                  const PrefillParams& p, cudaStream_t stream) {
  if (p.sp.cap2 == 0.f && p.sp.slopes == nullptr)
    return launch_prefill_mode<kPrefillMasked>(tk, tv, tq, to, p, stream);
  if (capped_kernel_serves(p.sp, p.qscale))
    return launch_prefill_mode<kPrefillCapped>(tk, tv, tq, to, p, stream);
  return launch_prefill_mode<kPrefillGeneral>(tk, tv, tq, to, p, stream);
}

}  // namespace pkv
