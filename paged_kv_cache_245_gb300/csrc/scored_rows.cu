// scored_rows.cu -- attention with capped, biased and masked scores, one warp
// per (token, query head): the plainest kernel that is right for every case.
// It reads K and V once per query head, so it is bound by L2 at G times the
// traffic the cache needs.
#include "scored_rows.cuh"

namespace pkv {

__global__ void __launch_bounds__(128) scored_rows_kernel(const ScoredRowsParams p) {
  grid_dependency_trigger();
  grid_dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (w >= p.num_rows * p.Hq) return;
  const int64_t row = w / p.Hq;
  const int h = static_cast<int>(w - row * p.Hq);
  const int G = p.Hq / p.Hkv;
  int seq, pos, ctx;
  int64_t cap = static_cast<int64_t>(p.max_blocks) * p.bs;
  if (p.cu_q == nullptr) {
    seq = static_cast<int>(row);
    ctx = p.ctx_lens[seq];
    if (cap > p.max_context) cap = p.max_context;
    if (p.checked && ctx > cap) {
      if (lane == 0) record_error(p.err, kErrContext);
      ctx = static_cast<int>(cap);
    }
    pos = ctx - 1;
  } else {
    int a = 0, b = p.num_seqs - 1;  // the last sequence that starts at or before the row
    while (a < b) {
      const int mid = (a + b + 1) >> 1;
      if (p.cu_q[mid] <= row) a = mid; else b = mid - 1;
    }
    seq = a;
    const int q0 = p.cu_q[seq], Lq = p.cu_q[seq + 1] - q0;
    if (row < q0 || row >= q0 + Lq) return;  // behind the last chunk
    ctx = p.ctx_lens[seq];
    if (p.checked && (Lq > p.max_q || ctx < Lq || ctx > cap)) {
      if (lane == 0) record_error(p.err, kErrContext);
      return;
    }
    pos = ctx - Lq + static_cast<int>(row - q0);
  }
  int lo, hi;
  visible_keys(p.sp, pos, p.sp.first_key ? p.sp.first_key[row] : 0,
               p.cu_q != nullptr && p.sp.prefix ? p.sp.prefix[seq] : 0, ctx, lo, hi);
  KvRows kv;
  kv.k = p.k;
  kv.v = p.v;
  kv.table = p.tables + static_cast<int64_t>(seq) * p.max_blocks;
  kv.bs = p.bs;
  kv.num_blocks = p.num_blocks;
  kv.Hkv = p.Hkv;
  kv.kvh = h / G;
  kv.checked = p.checked;
  kv.err = p.err;
  kv.err_code = p.err_code;
  float o[16];
  attend_row(p.sp, kv, p.q + w * kHeadDim, p.qscale,
             p.sp.slopes ? p.sp.slopes[h] * kLog2e : 0.f, pos, lo, hi, lane, o);
  if (lane < 8) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
      *reinterpret_cast<uint4*>(p.out + w * kHeadDim + c * 64 + lane * 8) =
          make_uint4(pack_bf16x2(o[8 * c], o[8 * c + 1]), pack_bf16x2(o[8 * c + 2], o[8 * c + 3]),
                     pack_bf16x2(o[8 * c + 4], o[8 * c + 5]),
                     pack_bf16x2(o[8 * c + 6], o[8 * c + 7]));
  }
}

cudaError_t launch_scored_rows(const ScoredRowsParams& p, cudaStream_t stream) {
  const int64_t warps = p.num_rows * p.Hq;
  if (warps <= 0) return cudaSuccess;
  if ((warps + 3) / 4 > 0x7fffffffLL) return cudaErrorInvalidValue;
  return launch_pdl(scored_rows_kernel, dim3(static_cast<unsigned>((warps + 3) / 4)), dim3(128), 0,
                    stream, p);
}

}  // namespace pkv
