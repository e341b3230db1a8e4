// prefill_scored.cuh -- the softmax of the prefill kernel for capped, biased
// and masked scores: one key tile of one row per thread, S in tensor memory
// in, P = 2^(score - m) as packed bf16 pairs out (over the first 64 columns of
// S in place).
//
// Masks.  What a token sees is one interval of positions, so a row's mask in
// a tile is an interval of columns; a tile that every row of the warp sees
// whole takes the path without masks.
//
// Capped scores (kPrefillCapped).  |score| <= cap, so no running maximum is
// needed: P is taken against a fixed m, chosen so that the lowest score keeps
// 2^-100 (26 binary digits above the smallest normal number) and the highest
// stays at 2^50 or less, and O and l are never rescaled.  That leaves one pass
// over S.  The tanh: three special-function operations an element (two
// exponentials, a reciprocal) would take three times the tensor cores' time,
// and tanh.approx is too coarse (2^-11); so where every score of the warp's
// half tile is within the cap (|s| <= cap, |tanh| <= 0.76) it is an odd
// polynomial on packed pairs, s (c0 + c1 w + .. + c4 w^4), w = s^2: the minimax
// fit of tanh(y) / y over y^2 in [0, 1] (relative error 2^-17, by Remez
// exchange; the probabilities are rounded to 2^-9 after it).  A half tile with
// a larger score is done again with exponentials.
#pragma once

#include <limits.h>

#include "prefill.cuh"
#include "score.cuh"
#include "umma.cuh"

namespace pkv {

struct ScoredRow {
  int lo, hi;    // columns the row sees, counted from the item's first key (none: lo > hi)
  int pos;       // the row's own position, counted the same
  float slope2;  // its head's slope, log-2 units
};

struct ScoredConsts {
  float sc;         // scale * log2 e
  ScoreParams sp;
  // kPrefillCapped
  uint64_t c[5];    // the polynomial in the raw product's square, as pairs
  uint64_t neg_m2;  // -m as a pair
  float w_max;      // squares up to this are in the polynomial's range
  float exp_k, neg_2cap, cap_m;  // 2^(exp_k s) = e^(2y); cap - m
};

// The offset m of capped scores |x| <= cap2 (cap2 <= 75): see above.
__host__ __device__ inline float capped_offset(float cap2) {
  return cap2 <= 50.f ? cap2 : 100.f - cap2;
}

// Whether the capped kernel serves these scores: a cap whose range fits the
// fixed offset, no bias, and a raw product at the cap (cap / scale) whose
// eighth power neither overflows nor underflows in fp32.
inline bool capped_kernel_serves(const ScoreParams& sp, float qscale) {
  if (!(sp.cap2 > 0.f) || sp.cap2 > 75.f || sp.slopes != nullptr) return false;
  const float r = qscale * sp.inv_cap2 < 0.f ? -qscale * sp.inv_cap2 : qscale * sp.inv_cap2;
  return r >= 1.220703125e-4f && r <= 8192.f;  // 2^-13 .. 2^13
}

template <int kMode>
__device__ __forceinline__ ScoredConsts scored_consts(const PrefillParams& p) {
  using namespace umma;
  ScoredConsts k;
  k.sc = p.qscale;
  k.sp = p.sp;
  if (kMode == kPrefillCapped) {
    const float r = k.sc * p.sp.inv_cap2;
    const float fit[5] = {0.99999309f, -0.33298065f, 0.13036811f, -0.04481755f, 0.00903642f};
    float power = k.sc;
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const uint32_t b = __float_as_uint(fit[i] * power);
      k.c[i] = f2_pack(b, b);
      power *= r * r;
    }
    const float m = capped_offset(p.sp.cap2);
    k.neg_m2 = f2_pack(__float_as_uint(-m), __float_as_uint(-m));
    k.w_max = 1.f / (r * r);
    k.exp_k = k.sc * p.sp.cap_k;
    k.neg_2cap = -2.f * p.sp.cap2;
    k.cap_m = p.sp.cap2 - m;
  }
  return k;
}

// Bits c of columns 32 w + c that lie in [a, b].
__device__ __forceinline__ uint32_t span_bits(int a, int b, int w) {
  const int lo = max(a - 32 * w, 0), hi = min(b - 32 * w, 31);
  return lo <= hi ? (0xffffffffu << lo) & (0xffffffffu >> (31 - hi)) : 0u;
}

// O *= alpha for the warp's rows.
__device__ __forceinline__ void rescale_o(uint32_t o_tm, float alpha) {
  using namespace umma;
#pragma unroll 1
  for (int c0 = 0; c0 < kHeadDim; c0 += 32) {
    uint32_t w[32];
    tmem_ld32(w, o_tm + c0);
    tmem_wait_ld(w);
#pragma unroll
    for (int c = 0; c < 32; ++c) w[c] = __float_as_uint(__uint_as_float(w[c]) * alpha);
    tmem_st32(o_tm + c0, w);
  }
}

// The row's running maximum takes in the tile's; O and l are rescaled when it
// grows by more than 2^kRescaleLog2.  Returns the offset P is taken against
// (0 while the row has seen nothing, where every P is masked).
__device__ __forceinline__ float take_max(float tmax, bool first, uint32_t o_tm, float& m_used,
                                          float& l) {
  using namespace umma;
  const float m_new = fmaxf(m_used, tmax);
  if (first) {
    m_used = m_new;
  } else {
    const bool grow = m_new > m_used + kRescaleLog2;  // always, from -inf
    if (__any_sync(kFull, grow)) {
      const float alpha = grow ? fast_exp2(m_used - m_new) : 1.f;
      if (grow) {
        l *= alpha;
        m_used = m_new;
      }
      rescale_o(o_tm, alpha);
    }
  }
  return m_used == -INFINITY ? 0.f : m_used;
}

// P of 64 columns from their scores: e(c) for column c, packed and summed.
template <typename Score>
__device__ __forceinline__ float masked_half(uint32_t s_tm, int h, uint32_t lo, uint32_t hi,
                                             Score score) {
  using namespace umma;
  uint32_t a[32], b[32], pk[32];
  tmem_ld32(a, s_tm + 64 * h);
  tmem_ld32(b, s_tm + 64 * h + 32);
  tmem_wait_ld(a);
  tmem_ready(b);
  float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    const uint32_t u0 = c < 16 ? a[2 * c] : b[2 * c - 32];
    const uint32_t u1 = c < 16 ? a[2 * c + 1] : b[2 * c - 31];
    float e0 = fast_exp2(score(__uint_as_float(u0)));
    float e1 = fast_exp2(score(__uint_as_float(u1)));
    const uint32_t bits = c < 16 ? lo : hi;
    e0 = (bits >> ((2 * c) & 31)) & 1u ? e0 : 0.f;
    e1 = (bits >> ((2 * c + 1) & 31)) & 1u ? e1 : 0.f;
    ls[c & 3] += e0 + e1;
    pk[c] = pack_bf16x2(e0, e1);
  }
  tmem_st32(s_tm + 32 * h, pk);
  return (ls[0] + ls[1]) + (ls[2] + ls[3]);
}

__device__ __forceinline__ void zero_half(uint32_t s_tm, int h) {
  uint32_t pz[32];
#pragma unroll
  for (int c = 0; c < 32; ++c) pz[c] = 0u;
  umma::tmem_st32(s_tm + 32 * h, pz);
}

// One half (64 columns) under the cap: the polynomial, or, where a score is
// out of its range, the exponentials.
template <bool kMasked>
__device__ __forceinline__ float capped_half(const ScoredConsts& k, uint32_t s_tm, int h,
                                             uint32_t lo, uint32_t hi) {
  using namespace umma;
  uint32_t a[32], b[32], pk[32];
  tmem_ld32(a, s_tm + 64 * h);
  tmem_ld32(b, s_tm + 64 * h + 32);
  tmem_wait_ld(a);
  tmem_ready(b);
  uint64_t ls2[2] = {0ull, 0ull};
  float top[2] = {0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    const uint64_t s2 = c < 16 ? f2_pack(a[2 * c], a[2 * c + 1]) : f2_pack(b[2 * c - 32], b[2 * c - 31]);
    const uint64_t w2 = f2_mul(s2, s2);
    float w0, w1;
    f2_unpack(w2, w0, w1);
    top[c & 1] = fmax3(top[c & 1], w0, w1);
    uint64_t q = f2_fma(w2, k.c[4], k.c[3]);
    q = f2_fma(w2, q, k.c[2]);
    q = f2_fma(w2, q, k.c[1]);
    q = f2_fma(w2, q, k.c[0]);
    float x0, x1;
    f2_unpack(f2_fma(s2, q, k.neg_m2), x0, x1);
    float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
    if (kMasked) {
      const uint32_t bits = c < 16 ? lo : hi;
      e0 = (bits >> ((2 * c) & 31)) & 1u ? e0 : 0.f;
      e1 = (bits >> ((2 * c + 1) & 31)) & 1u ? e1 : 0.f;
    }
    ls2[c & 1] = f2_add(ls2[c & 1], f2_pack(__float_as_uint(e0), __float_as_uint(e1)));
    pk[c] = pack_bf16x2(e0, e1);
  }
  if (__any_sync(kFull, fmaxf(top[0], top[1]) > k.w_max)) {
    const uint32_t all = 0xffffffffu;
    return masked_half(s_tm, h, kMasked ? lo : all, kMasked ? hi : all, [&](float s) {
      return fmaf(k.neg_2cap, fast_rcp(1.f + fast_exp2(s * k.exp_k)), k.cap_m);
    });
  }
  tmem_st32(s_tm + 32 * h, pk);
  float l0, l1;
  f2_unpack(f2_add(ls2[0], ls2[1]), l0, l1);
  return l0 + l1;
}

// One key tile: kt is its first column counted from the item's first key.
template <int kMode>
__device__ __forceinline__ void scored_tile(const ScoredConsts& k, const ScoredRow& r,
                                            uint32_t s_tm, uint32_t o_tm, int kt, bool first,
                                            float& m_used, float& l) {
  using namespace umma;
  // columns of this tile the row sees (kt is far below 2^31 where hi is not)
  const int c0 = r.lo > kt ? (r.lo - kt > 128 ? 128 : r.lo - kt) : 0;
  const int c1 = r.hi < kt ? -1 : (r.hi - kt > 127 ? 127 : r.hi - kt);
  const bool masked = __any_sync(kFull, c0 > 0 || c1 < 127);
  const float sc = k.sc;

  if (kMode == kPrefillCapped) {
    if (!masked) {
#pragma unroll
      for (int h = 0; h < 2; ++h) l += capped_half<false>(k, s_tm, h, 0u, 0u);
    } else {
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const uint32_t lo = span_bits(c0, c1, 2 * h), hi = span_bits(c0, c1, 2 * h + 1);
        if (!__any_sync(kFull, (lo | hi) != 0u)) zero_half(s_tm, h);
        else l += capped_half<true>(k, s_tm, h, lo, hi);
      }
    }
    return;
  }

  if (kMode == kPrefillMasked && !masked && sc >= 0.f) {
    // (a negative scale: the maximum of the scaled scores is not the scaled maximum)
    float mx[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) mx[u] = -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t a[32], b[32];
      tmem_ld32(a, s_tm + 64 * h);
      tmem_ld32(b, s_tm + 64 * h + 32);
      tmem_wait_ld(a);
      tmem_ready(b);
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        mx[c & 3] = fmax3(mx[c & 3], __uint_as_float(a[2 * c]), __uint_as_float(a[2 * c + 1]));
        mx[(c + 2) & 3] =
            fmax3(mx[(c + 2) & 3], __uint_as_float(b[2 * c]), __uint_as_float(b[2 * c + 1]));
      }
    }
    const float tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
    const float m = take_max(tmax, first, o_tm, m_used, l);
    const uint64_t sc2 = f2_pack(__float_as_uint(sc), __float_as_uint(sc));
    const uint64_t nm2 = f2_pack(__float_as_uint(-m), __float_as_uint(-m));
    uint64_t ls2[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) ls2[u] = 0ull;  // (+0, +0)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t a[32], b[32], pk[32];
      tmem_ld32(a, s_tm + 64 * h);
      tmem_ld32(b, s_tm + 64 * h + 32);
      tmem_wait_ld(a);
      tmem_ready(b);
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        const uint64_t s2 =
            c < 16 ? f2_pack(a[2 * c], a[2 * c + 1]) : f2_pack(b[2 * c - 32], b[2 * c - 31]);
        float x0, x1;
        f2_unpack(f2_fma(s2, sc2, nm2), x0, x1);
        const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
        ls2[c & 3] = f2_add(ls2[c & 3], f2_pack(__float_as_uint(e0), __float_as_uint(e1)));
        pk[c] = pack_bf16x2(e0, e1);
      }
      tmem_st32(s_tm + 32 * h, pk);
    }
    float l0, l1, l2, l3;
    f2_unpack(f2_add(ls2[0], ls2[1]), l0, l1);
    f2_unpack(f2_add(ls2[2], ls2[3]), l2, l3);
    l += (l0 + l2) + (l1 + l3);
    return;
  }

  // Any score, any mask.  Pass 1: the row's maximum; where a score costs more
  // than a product it is written back over S for pass 2.
  constexpr bool kStore = kMode == kPrefillGeneral;
  float mx[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) mx[u] = -INFINITY;
  const float posf = static_cast<float>(r.pos - kt);
#pragma unroll 1
  for (int w = 0; w < 4; ++w) {
    const uint32_t bits = span_bits(c0, c1, w);
    if (!__any_sync(kFull, bits != 0u)) continue;
    uint32_t a[32];
    tmem_ld32(a, s_tm + 32 * w);
    tmem_wait_ld(a);
    const float at = posf - static_cast<float>(32 * w);
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      float x = __uint_as_float(a[c]) * sc;
      if (kStore) {
        if (k.sp.cap2 > 0.f) x = capped_score(k.sp, x);
        x = fmaf(-r.slope2, fabsf(at - static_cast<float>(c)), x);
        a[c] = __float_as_uint(x);
      }
      mx[c & 3] = (bits >> c) & 1u ? fmaxf(mx[c & 3], x) : mx[c & 3];
    }
    if (kStore) tmem_st32(s_tm + 32 * w, a);
  }
  if (kStore) tmem_wait_st();
  const float m = take_max(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), first, o_tm, m_used, l);
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = span_bits(c0, c1, 2 * h), hi = span_bits(c0, c1, 2 * h + 1);
    if (!__any_sync(kFull, (lo | hi) != 0u)) zero_half(s_tm, h);
    else
      l += masked_half(s_tm, h, lo, hi,
                       [&](float s) { return kStore ? s - m : fmaf(s, sc, -m); });
  }
}

// Whether all 128 elements of this thread's row of O are finite.
__device__ __forceinline__ bool finite_row(uint32_t o_tm) {
  using namespace umma;
  float z = 0.f;  // 0 x is 0 for a finite x, else NaN
#pragma unroll 1
  for (int c0 = 0; c0 < kHeadDim; c0 += 32) {
    uint32_t w[32];
    tmem_ld32(w, o_tm + c0);
    tmem_wait_ld(w);
#pragma unroll
    for (int c = 0; c < 32; ++c) z = fmaf(__uint_as_float(w[c]), 0.f, z);
  }
  return z == 0.f;
}

// Computes and writes the rows flagged in the warp, one by one.
static __device__ __noinline__ void repair_rows(const PrefillParams& p, const KvRows& kv, bool flagged,
                                         int64_t qrow, const ScoredRow& r, int k0, int lane) {
  for (uint32_t left = __ballot_sync(umma::kFull, flagged); left != 0u; left &= left - 1) {
    const int src = __ffs(left) - 1;
    const int64_t row = __shfl_sync(umma::kFull, qrow, src);
    const int lo = __shfl_sync(umma::kFull, r.lo, src), hi = __shfl_sync(umma::kFull, r.hi, src);
    const int pos = __shfl_sync(umma::kFull, r.pos, src);
    const float slope2 = __shfl_sync(umma::kFull, r.slope2, src);
    float o[16];
    attend_row(p.sp, kv, p.q + row * kHeadDim, p.qscale, slope2, pos + k0, hi < 0 ? 0 : lo + k0,
               hi < 0 ? -1 : hi + k0, lane, o);
    if (lane < 8) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        *reinterpret_cast<uint4*>(p.out + row * kHeadDim + c * 64 + lane * 8) = make_uint4(
            pack_bf16x2(o[8 * c], o[8 * c + 1]), pack_bf16x2(o[8 * c + 2], o[8 * c + 3]),
            pack_bf16x2(o[8 * c + 4], o[8 * c + 5]), pack_bf16x2(o[8 * c + 6], o[8 * c + 7]));
    }
  }
}

}  // namespace pkv
