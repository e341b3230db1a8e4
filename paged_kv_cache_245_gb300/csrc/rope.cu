// rope.cu -- rotary positions on new queries and keys, and the append of the
// turned keys and of the values to the cache, in one pass over the rows.
//
// Pair i of a row at position p is turned by the angle p w_i:
//   (x, y) -> gain (x cos a - y sin a, y cos a + x sin a),  a = p w_i.
// The angle is taken in turns: the plan holds f_i = w_i / 2 pi as a 64-bit
// fraction F_i / 2^64, and p F_i mod 2^64 is the fraction of a turn, exactly,
// for every int32 p -- the integer product wraps as the angle does, so no
// range reduction is needed and far positions lose nothing (the error is
// that of F_i times p: under 2^-34 turns at a million positions).
//
// What bounds it: memory.  Every row is read once and written once (256 bytes
// each way); the 64 sines and cosines of a token are computed once and serve
// all its heads from shared memory.  A row takes 8 lanes of two 16-byte
// chunks; in the half layout a lane's two chunks are partners (chunk c and
// c + rotary_dim / 16), so that no lane needs another's elements.  A row is
// loaded while the one before it is turned, the first while the sines are
// computed; five CTAs an SM keep 80 KiB of rows in flight (three, with the
// registers left alone: 5.4 for 4.2 us at 333 tokens of an odd rotary size).
// The sines are padded so that a row's lanes read different banks (4096 tokens
// 20.5 -> 16.0 us).  16384 tokens of 32 + 2 x 8 heads (403 MB) take 64.6 us, 6.2
// TB/s or 0.92 of a plain copy; 64 tokens 3.2 us and one 2.6 us, a launch and
// three dependent reads (position, sines, row).
#include "rope_rows.cuh"

namespace pkv {

namespace {

template <int kKind, int kTokens>
__global__ void __launch_bounds__(kRopeThreads, 5) rope_append_kernel(const RopeParams p) {
  __shared__ RopeSmem<kKind, kTokens> sm;
  grid_dependency_trigger();
  grid_dependency_wait();
  rope_rows<kKind, kTokens>(p, sm, threadIdx.x, blockIdx.x, blockIdx.y, gridDim.y);
}

template <int kKind>
cudaError_t launch_kind(const RopeParams& p, cudaStream_t stream) {
  const int R = p.Hq + 2 * p.Hkv;
  const unsigned n = static_cast<unsigned>(p.num_tokens);
  const dim3 block(kRopeThreads);
  // Few tokens: one a CTA, its rows over grid y, so that every row of the call
  // is in flight at once (305 tokens x 48 rows 3.4 us, two a CTA 3.8; 512 4.4
  // and 4.1).  Past that a CTA passes over the rows of more tokens: two up to
  // 2048 (1500 tokens 6.1 us, four a CTA 7.0), then four (4096 tokens 16.2 us,
  // two 16.5, eight 17.3).
  if (n <= 400)
    return launch_pdl(rope_append_kernel<kKind, 1>, dim3(n, (R + kRowsPerPass - 1) / kRowsPerPass),
                      block, 0, stream, p);
  if (n <= 2048)
    return launch_pdl(rope_append_kernel<kKind, 2>, dim3((n + 1) / 2), block, 0, stream, p);
  return launch_pdl(rope_append_kernel<kKind, 4>, dim3(n / 4 + (n % 4 != 0)), block, 0, stream, p);
}

}  // namespace

cudaError_t launch_rope_append(const RopeParams& p, cudaStream_t stream) {
  if (p.num_tokens <= 0) return cudaSuccess;
  if (p.rope.interleaved) return launch_kind<0>(p, stream);
  return p.rope.rotary_dim % 16 == 0 ? launch_kind<1>(p, stream) : launch_kind<2>(p, stream);
}

}  // namespace pkv
