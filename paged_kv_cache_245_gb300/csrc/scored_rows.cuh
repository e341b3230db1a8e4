// scored_rows.cuh -- parameters and launcher of the row-by-row scored
// attention (scored_rows.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "score.cuh"

namespace pkv {

struct ScoredRowsParams {
  const uint16_t* q;         // [rows][Hq][128]: decode one row a sequence, prefill packed chunks
  uint16_t* out;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* tables;     // [B][max_blocks]; contiguous: request ids, max_blocks 1
  const int32_t* cu_q;       // prefill: [B + 1]; decode: null
  const int32_t* ctx_lens;   // [B]
  int64_t bs, num_blocks;
  int64_t num_rows;          // rows of q
  int32_t max_blocks, num_seqs, Hq, Hkv;
  int32_t max_context;       // decode: host bound on every context
  int32_t max_q;             // prefill: host bound on every chunk
  float qscale;
  ScoreParams sp;
  int32_t checked;
  int* err;
  int err_code;              // of a table entry out of range
};

cudaError_t launch_scored_rows(const ScoredRowsParams& p, cudaStream_t stream);

}  // namespace pkv
