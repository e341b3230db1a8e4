// prefill.cu -- host side of prefill attention (tensor maps, launch) and the
// plain causal kernel (prefill_kernel.cuh).
#include <cudaTypedefs.h>

#include <mutex>

#include "prefill_kernel.cuh"

namespace pkv {

namespace {

PFN_cuTensorMapEncodeTiled_v12000 prefill_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

}  // namespace

bool encode_prefill_runs(CUtensorMap* map, const void* base, int64_t rows, int run_rows) {
  auto enc = prefill_map_encoder();
  if (enc == nullptr || rows % 8 != 0 || run_rows % 8 != 0 || run_rows > 128) return false;
  // dims (innermost first): 64 columns, 8 rows of a group, 2 column halves, groups
  const cuuint64_t dims[4] = {64u, 8u, 2u, static_cast<cuuint64_t>(rows / 8)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(kRowBytes), 128u,
                                 static_cast<cuuint64_t>(8 * kRowBytes)};
  const cuuint32_t box[4] = {64u, 8u, 2u, static_cast<cuuint32_t>(run_rows / 8)};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

bool encode_prefill_rows(CUtensorMap* map, const void* base, int64_t num_tokens, int Hq, int G,
                         int box_rows) {
  auto enc = prefill_map_encoder();
  if (enc == nullptr || G <= 0 || box_rows % G != 0 || box_rows > 128 || box_rows / G > 256 ||
      Hq < G || num_tokens <= 0)
    return false;
  const cuuint64_t dims[4] = {64u, 2u, static_cast<cuuint64_t>(Hq),
                              static_cast<cuuint64_t>(num_tokens)};
  const cuuint64_t strides[3] = {128u, static_cast<cuuint64_t>(kRowBytes),
                                 static_cast<cuuint64_t>(Hq) * kRowBytes};
  const cuuint32_t box[4] = {64u, 1u, static_cast<cuuint32_t>(G),
                            static_cast<cuuint32_t>(box_rows / G)};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

cudaError_t launch_prefill(const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tq,
                           const CUtensorMap& to, const PrefillParams& p, cudaStream_t stream) {
  return launch_prefill_mode<kPrefillPlain>(tk, tv, tq, to, p, stream);
}

}  // namespace pkv
