// q8.cuh -- the 8-bit KV cache: codes (int8 or e4m3) with one fp32 scale for
// every 16 rows of a (block, KV head), value = code * scale.  Parameters and
// launchers of its append (append_q8.cu) and attention kernels.
//
// Row r (pkv_device.cuh: cache_row) holds 128 code bytes at codes + 128 r.
// Block sizes are multiples of 16, so rows 16 n .. 16 n + 15 lie in one
// (block, head): group n, with its scale at scale[n].
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/pkv.h"
#include "decode_tc_launch.h"
#include "rope.cuh"

namespace pkv {

constexpr int kGroupRows = 16;
constexpr int kCodeRowBytes = 128;
constexpr float kInt8Max = 127.f;
constexpr float kE4m3Max = 448.f;
// A scale below this holds zeros (its reciprocal would leave fp32's range).
constexpr float kScaleTiny = 7.888609052210118e-31f;  // 2^-100

struct AppendQ8Params {
  const int64_t* slot_mapping;  // [T]
  const uint16_t* k;            // [Hkv][128] at k + t * k_stride
  const uint16_t* v;
  int64_t k_stride, v_stride;   // elements
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scale;
  float* v_scale;
  int64_t num_slots, bs;
  int32_t num_tokens, Hkv;
  // with rotary positions: the queries' part of the call (no K or V heads), whose
  // positions and plan are the keys' too
  RopeParams queries;
  int32_t checked, sms;
  int* err;
};

// rope: turn queries and keys on the way.
cudaError_t launch_append_q8(const AppendQ8Params& p, bool e4m3, bool rope, cudaStream_t stream);

struct AttentionQ8Params {
  const uint16_t* q;            // [T][Hq][128]
  uint16_t* out;                // [T][Hq][128]
  const int32_t* cu_q;          // prefill [B + 1]; null: one row per sequence
  const int32_t* ctx_lens;      // [B]
  const int32_t* tables;        // [B][max_blocks]; contiguous: request ids, max_blocks 1, bs = S
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const float* k_scale;
  const float* v_scale;
  int64_t bs, num_blocks;
  int32_t max_blocks, num_seqs, Hq, Hkv, G;
  int32_t max_q;                // host bound on any chunk's length (decode: 1)
  int32_t max_context;          // decode: host bound on any context; prefill: what a table holds
  float qscale;                 // scale * log2(e)
  int32_t checked, err_code;    // err_code: of a table entry out of range
  int* err;
};

// Decode (cu_q null), or chunks that chunks_by_runs says: workspace of
// tc_workspace_bytes(num_ctas).
bool chunks_by_runs(int num_tokens, int num_seqs, int max_q, int Hkv, int G, int max_context);
TcStatus launch_decode_q8(const AttentionQ8Params& p, bool e4m3, bool contig, int num_ctas,
                          void* workspace, cudaStream_t stream, cudaError_t* cuda_err);
// The same for small batches: a cluster of 1, 2, 4 or 8 CTAs of 4 or 8 warps a
// (sequence, KV head); no workspace.  The room on the current device for clusters of
// 8-warp CTAs, of which an SM holds one (of 4-warp CTAs: kQ8SmallCtas).
struct ClusterRoom;
constexpr int kQ8SmallCtas = 3;
cudaError_t room_decode_q8_cluster(bool e4m3, ClusterRoom* out);
cudaError_t launch_decode_q8_cluster(const AttentionQ8Params& p, bool e4m3, int cluster, int warps,
                                     cudaStream_t stream);
// Prefill (prefill_q8.cu).  workspace (16-byte aligned): prefill_q8_workspace bytes, if
// that is not 0.
size_t prefill_q8_workspace(int num_tokens, int num_seqs, int max_q, int Hkv, int G, int sms);
TcStatus launch_prefill_q8(const AttentionQ8Params& p, bool e4m3, bool contig, int num_tokens,
                           int sms, void* workspace, cudaStream_t stream, cudaError_t* cuda_err);

#ifdef __CUDACC__

// Two e4m3 codes (the low 16 bits) as two halves; exact, NaN codes stay NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t codes) {
  uint32_t h;
  asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(h) : "r"(codes));
  return h;
}

// Two values as e4m3 codes, `lo` in the low byte: nearest, ties to even,
// saturated; NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(hi), "f"(lo));
  return c;
}

#endif

}  // namespace pkv
