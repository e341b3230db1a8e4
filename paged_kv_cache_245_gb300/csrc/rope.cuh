// rope.cuh -- parameters and launcher of the rotary append (rope.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pkv.h"

namespace pkv {

struct RopeParams {
  const int32_t* positions;     // [T]
  const int64_t* slot_mapping;  // [T]
  const uint16_t* q;            // token t's heads at q + t * q_stride: [Hq][128]
  const uint16_t* k;            // [Hkv][128] at k + t * k_stride
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;  // elements
  uint16_t* q_out;              // [T][Hq][128] (may be q)
  uint16_t* k_cache;
  uint16_t* v_cache;
  int64_t num_tokens, num_slots, bs;
  int32_t Hq, Hkv;
  pkv_rope rope;
  int32_t checked;
  int* err;
};

cudaError_t launch_rope_append(const RopeParams& p, cudaStream_t stream);

}  // namespace pkv
