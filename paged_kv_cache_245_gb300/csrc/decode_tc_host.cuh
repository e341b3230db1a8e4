// decode_tc_host.cuh -- launch of one instantiation of the tensor-core decode
// kernel over a batch, in chunks of at most kTcMaxSeqs sequences.
#pragma once

#include "decode_tc.cuh"

namespace pkv {

template <bool kContig, int W, int S, bool kFuse, int MH = kTcMergeHeads, int NT = 1,
          bool kScored = false>
cudaError_t launch_cfg(const CUtensorMap& tk, const CUtensorMap& tv, const TcParams& p0,
                       int num_ctas, cudaStream_t stream) {
  using L = TcSmem<W, S, NT, MH, kScored>;
  static unsigned long long done_mask = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  auto kernel = decode_tc_kernel<kContig, W, S, NT, kFuse, MH, kScored>;
  if (!(__atomic_load_n(&done_mask, __ATOMIC_ACQUIRE) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
    if (e != cudaSuccess) return e;
    __atomic_fetch_or(&done_mask, bit, __ATOMIC_ACQ_REL);
  }
  const int chunk = tc_chunk_seqs(p0.max_context);
  for (int s0 = 0; s0 < p0.num_seqs; s0 += chunk) {
    TcParams p = p0;
    p.num_seqs = (p0.num_seqs - s0) < chunk ? (p0.num_seqs - s0) : chunk;
    p.q += static_cast<int64_t>(s0) * p.Hq * kHeadDim;
    p.out += static_cast<int64_t>(s0) * p.Hq * kHeadDim;
    if (p.rec_out != nullptr) p.rec_out += static_cast<int64_t>(s0) * p.Hq * kRecStride;
    p.ctx_lens += s0;
    if (p.slot_mapping != nullptr) {
      p.slot_mapping += s0;
      p.k_new += static_cast<int64_t>(s0) * p.Hkv * kHeadDim;
      p.v_new += static_cast<int64_t>(s0) * p.Hkv * kHeadDim;
    }
    if (kScored && p.sp.first_key != nullptr) p.sp.first_key += s0;
    if (kContig) p.req_ids += s0;
    else p.block_tables += static_cast<int64_t>(s0) * p.max_blocks;
    p.tag = next_launch_tag();  // every launch writes its piece records under a fresh tag
    e = launch_pdl_if(pdl_decode_enabled(), kernel, dim3(num_ctas), dim3(W * 32),
                      L::kTotal, stream, tk, tv, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace pkv
