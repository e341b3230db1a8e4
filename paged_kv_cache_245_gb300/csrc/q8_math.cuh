// q8_math.cuh -- arithmetic on 8-bit codes shared by the attention kernels over
// the 8-bit cache: codes as halves, fp16 products of a warp, queries as halves.
#pragma once

#include "pkv_device.cuh"
#include "q8.cuh"

namespace pkv {

// d = a(16x16, row) * b(16x8, col) + c, fp16 inputs, fp32 accumulation.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
      "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_16816_zero(float (&d)[4], const uint32_t (&a)[4],
                                                   uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
      "{%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two probabilities (0 .. 1: against the running maximum) as halves, times 2^15: rounded
// by 2^-11 at most down to 2^-29, and by 2^-40 below.  (As they are, by 2^-11 down to 2^-14
// and to 0 below 2^-25, while their sum kept them: under one key with nearly all of a
// softmax the others' values were lost.)  The products with them are fp32; kPDown goes
// into the values' scale.
constexpr float kPUp = 32768.f, kPDown = 3.0517578125e-05f;
__device__ __forceinline__ uint32_t probabilities_to_half2(float lo, float hi) {
  return pack_half2(lo * kPUp, hi * kPUp);
}

// 1152 in both halves taken off: int8 code + 1152 -> code, exact.
__device__ __forceinline__ uint32_t less_1152(uint32_t h) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
  return r;
}

// Codes (0, 1) and (2, 3) of a word as halves.
template <bool kE4m3>
__device__ __forceinline__ void halves_of(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (kE4m3) {
    lo = e4m3x2_to_half2(w);
    hi = e4m3x2_to_half2(w >> 16);
  } else {
    const uint32_t u = w ^ 0x80808080u;
    lo = less_1152(__byte_perm(u, 0x64646464u, 0x4140));
    hi = less_1152(__byte_perm(u, 0x64646464u, 0x4342));
  }
}

// Codes (0, 2) and (1, 3): one element of two keys each (V).
template <bool kE4m3>
__device__ __forceinline__ void halves_across(uint32_t w, uint32_t& even, uint32_t& odd) {
  if (kE4m3) {
    const uint32_t t = __byte_perm(w, 0u, 0x3120);
    even = e4m3x2_to_half2(t);
    odd = e4m3x2_to_half2(t >> 16);
  } else {
    const uint32_t u = w ^ 0x80808080u;
    even = less_1152(__byte_perm(u, 0x64646464u, 0x4240));
    odd = less_1152(__byte_perm(u, 0x64646464u, 0x4341));
  }
}

// Elements 32 tq .. 32 tq + 31 of query row g (lane 4 g + tq; bf16 as loaded) as the
// B fragments of eight k-steps, times 2^n with n = 14 - the exponent of the row's
// largest element (at most 126).  Returns 2^-n.
__device__ __forceinline__ float queries_to_half(const uint4 (&q)[4], uint32_t (&b)[8][2]) {
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const int n = min(126, 14 + 127 - static_cast<int>(__float_as_uint(top) >> 23));
  const float up = __uint_as_float(static_cast<uint32_t>(n + 127) << 23);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t w[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      b[2 * k + (e >> 1)][e & 1] = pack_half2(bf16_lo(w[e]) * up, bf16_hi(w[e]) * up);
  }
  return __uint_as_float(static_cast<uint32_t>(127 - n) << 23);
}

}  // namespace pkv
