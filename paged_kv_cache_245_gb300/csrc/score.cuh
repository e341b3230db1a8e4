// score.cuh -- scores beyond the plain scale * q . k, shared by the decode and
// prefill kernels: the cap by a tanh, the distance bias, and the interval of
// keys a token sees (window, document, prefix); and the attention of one row
// by one warp, which every kernel may fall back on.
//
// Scores are kept in units of log 2 (x = s log2 e), so that exponentials are
// plain powers of two.
#pragma once

#include <stdint.h>

#include "pkv_device.cuh"
#include "score.h"

namespace pkv {

constexpr float kLog2e = 1.4426950408889634f;
// Slope of head h in log-2 units per position.  Past 2^60 either way it would
// only overflow (a row of -inf scores has no maximum); weights that far apart
// are 0 or 1 long before.
constexpr float kMaxSlope = 1152921504606846976.f;
__device__ __forceinline__ float slope_log2(const float* slopes, int h) {
  return fminf(fmaxf(__ldg(slopes + h) * kLog2e, -kMaxSlope), kMaxSlope);
}

__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// softcap * tanh(s / softcap) in log-2 units.  tanh.approx is good to 2^-11
// only, which at a cap of 50 would be an error of 2 % in a probability.
// Above |y| = 1/2: tanh(y) = 1 - 2 / (1 + e^2y) (absolute error 2^-23 of the
// cap; saturates without overflow).  Below, where that form cancels: an odd
// polynomial, the minimax fit of tanh(y) / y over y^2 in [0, 1/4] (relative
// error 2^-26, by Remez exchange).
__device__ __forceinline__ float capped_score(const ScoreParams& sp, float x) {
  const float y = x * sp.inv_cap2;
  const float u = y * y;
  float p = fmaf(u, 0.01713501f, -0.05298608f);
  p = fmaf(u, p, 0.13324779f);
  p = fmaf(u, p, -0.33333069f);
  p = fmaf(u, p, 0.99999999f);
  const float far = fmaf(-2.f * sp.cap2, fast_rcp(1.f + fast_exp2(x * sp.cap_k)), sp.cap2);
  return u <= 0.25f ? x * p : far;
}

// Whether a part of a row (a warp's, a split's, a piece) has nothing in its sum l
// of probabilities.  A NaN score makes its part's sum NaN, which is something:
// the row becomes NaN, as the formula does, wherever the schedule cut it.  (The
// plain kernels leave such parts out.)
template <bool kScored>
__device__ __forceinline__ bool empty_sum(float l) {
  return kScored ? l == 0.f : !(l > 0.f);
}

// What probabilities are taken against: the maximum m, or 0 while every score of
// the part is -inf, so that such a score has no weight (not 2^(-inf + inf)).
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }

// The keys the token at position `pos` sees: lo <= j <= hi, none if lo > hi.
__device__ __forceinline__ void visible_keys(const ScoreParams& sp, int pos, int first, int prefix,
                                             int ctx, int& lo, int& hi) {
  lo = first > 0 ? first : 0;
  if (sp.window > 0 && pos - sp.window + 1 > lo) lo = pos - sp.window + 1;
  const int last = prefix < ctx ? prefix - 1 : ctx - 1;
  hi = pos > last ? pos : last;
  if (hi > ctx - 1) hi = ctx - 1;
}

// Where a sequence's rows of one KV head are.  Contiguous layout: bs = S and
// a one-entry table [reqId].
struct KvRows {
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* table;
  int64_t bs, num_blocks;
  int32_t Hkv, kvh;
  int32_t checked;
  int* err;
  int err_code;
};

// Attention of one query row over its keys [lo, hi] by one warp: four keys at
// a time, 8 lanes a key, 16 head elements a lane; an online softmax per lane
// group, joined at the end.  Reads visible rows only, so nothing that stands
// in masked places matters.  (Few registers on purpose: a larger function called
// from the prefill kernel, though never run, cost that 6 %.)  Result: lane group
// 0's lanes (lane < 8) hold elements 8 lane .. and 64 + 8 lane .. in o[0..7] and
// o[8..15], normalised; zeros for an empty row.
__device__ inline void attend_row(const ScoreParams& sp, const KvRows& kv, const uint16_t* q,
                                  float qscale, float slope2, int pos, int lo, int hi, int lane,
                                  float (&o)[16]) {
  constexpr unsigned kAll = 0xffffffffu;
  const int grp = lane >> 3, sub = lane & 7;
  const uint32_t bs = static_cast<uint32_t>(kv.bs);  // (positions and blocks are below 2^31)
  float qf[16];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint4 a = ld_global_nc_v4(q + w * 64 + sub * 8);
    const uint32_t x[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      qf[8 * w + 2 * e] = bf16_lo(x[e]);
      qf[8 * w + 2 * e + 1] = bf16_hi(x[e]);
    }
  }
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < 16; ++e) o[e] = 0.f;
  for (int64_t j0 = lo; j0 <= hi; j0 += 4) {
    const int64_t j = j0 + grp;
    bool seen = j <= hi;
    int64_t row = 0;
    if (seen) {
      const uint32_t at = static_cast<uint32_t>(j);
      const int32_t blk = kv.table[at / bs];
      if (kv.checked && (blk < 0 || blk >= kv.num_blocks)) {
        record_error(kv.err, kv.err_code);
        seen = false;
      } else {
        row = cache_row(blk, kv.kvh, kv.Hkv, kv.bs, at % bs) * kHeadDim;
      }
    }
    float x = 0.f;
    uint4 vw[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (seen) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const uint4 a = ld_global_nc_v4(kv.k + row + w * 64 + sub * 8);
        vw[w] = ld_global_nc_v4(kv.v + row + w * 64 + sub * 8);
        const uint32_t kx[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x = fmaf(qf[8 * w + 2 * e], bf16_lo(kx[e]), x);
          x = fmaf(qf[8 * w + 2 * e + 1], bf16_hi(kx[e]), x);
        }
      }
    }
    x += __shfl_xor_sync(kAll, x, 1);
    x += __shfl_xor_sync(kAll, x, 2);
    x += __shfl_xor_sync(kAll, x, 4);
    if (!seen) continue;
    x *= qscale;
    if (sp.cap2 > 0.f) x = capped_score(sp, x);
    if (slope2 != 0.f) {
      const float d = static_cast<float>(j < pos ? pos - j : j - pos);
      x = fmaf(-slope2, d, x);
    }
    if (!(x <= m)) {  // a NaN score makes the row NaN, as the formula does
      const float a = fast_exp2(m - x);
      l *= a;
#pragma unroll
      for (int e = 0; e < 16; ++e) o[e] *= a;
      m = x;
    }
    const float pr = x == -INFINITY ? 0.f : fast_exp2(x - m);  // -inf is no score
    l += pr;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint32_t vx[4] = {vw[w].x, vw[w].y, vw[w].z, vw[w].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[8 * w + 2 * e] = fmaf(pr, bf16_lo(vx[e]), o[8 * w + 2 * e]);
        o[8 * w + 2 * e + 1] = fmaf(pr, bf16_hi(vx[e]), o[8 * w + 2 * e + 1]);
      }
    }
  }
  // join the four groups
#pragma unroll
  for (int d = 8; d < 32; d <<= 1) {
    const float mo = __shfl_xor_sync(kAll, m, d), lo2 = __shfl_xor_sync(kAll, l, d);
    const float M = (m != m || mo != mo) ? NAN : fmaxf(m, mo);
    const float a = l == 0.f ? 0.f : fast_exp2(m - M);
    const float b = lo2 == 0.f ? 0.f : fast_exp2(mo - M);
    l = l * a + lo2 * b;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float other = __shfl_xor_sync(kAll, o[e], d);
      o[e] = (a == 0.f ? 0.f : o[e] * a) + (b == 0.f ? 0.f : other * b);
    }
    m = M;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < 16; ++e) o[e] = l == 0.f ? 0.f : o[e] * inv;
}

}  // namespace pkv
