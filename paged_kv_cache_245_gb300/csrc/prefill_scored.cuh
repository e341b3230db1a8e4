// prefill_scored.cuh -- the softmax of the scored prefill kernel
// (prefill_scored.cu): one key tile of one row per thread, S in tensor memory
// in, P = 2^(score - m) as packed bf16 pairs out, over the first 64 columns of
// S in place.
//
// Masks.  What a token sees is one interval of positions, so a row's mask in
// a tile is an interval of columns.  A tile that every row of the warp sees
// whole takes straight-line code; the others a loop over halves of 64 columns,
// with bit tests, that skips a half no row sees.  (A loop, and one body for
// every kind of half: code that runs once or twice an item comes out of a cold
// instruction cache.  Unrolled over the row it cost 8 x 2048 tokens 253 -> 323
// us, although one tile in eight takes it.)
//
// Capped scores (kPrefillCapped).  |score| <= cap, so no running maximum is
// needed, and one pass over S does: P is taken against a fixed m, chosen so that
// the lowest score keeps 2^-100 (26 binary digits above the smallest normal
// number) and the highest stays at 2^50 or less, and O and l are never rescaled.  The tanh: three
// special-function operations an element (two exponentials, a reciprocal)
// would take longer than the tensor cores, and tanh.approx is too coarse
// (2^-11); so where every score is within the cap (|s| <= cap, |tanh| <= 0.76)
// it is an odd polynomial on packed pairs, s (c0 + c1 w + .. + c4 w^4), w = s^2:
// the minimax fit of tanh(y) / y over y^2 in [0, 1] (relative error 2^-17, by
// Remez exchange; the probabilities are rounded to 2^-9 after it).  Half tiles
// with a larger score take the exponentials, after the polynomial that told so.
// Caps below 11 always do: 64 scores of 0 fall outside the sums that tile_capped
// accepts, and below 8.2 no sum is inside.  8 x 2048 tokens: caps of 2 to 10 554
// us whatever the scores; 12 and 15 285 us for scores of 0.25 and 554 for scores
// of 4 (most half tiles hold one beyond the cap); 30 and 50 273 us.
//
// Biased scores (kPrefillBiased).  Up to the row's own position the bias is
// linear in the column: one packed addition and one fused product a pair.  The
// key tiles come last first, so that the bias only falls (8 x 2048 tokens 288 ->
// 272 us).  Capped and biased (kPrefillCappedBiased): the bias of the nearest key
// stands in for the maximum, and again one pass does (522 -> 335 us).
#pragma once

#include <limits.h>

#include "prefill.cuh"
#include "score.cuh"
#include "umma.cuh"

namespace pkv {

// A thread's row of an item.
struct ScoredRow {
  int lo, hi;     // columns the row sees, counted from the item's first key (none: lo > hi)
  int pos;        // the row's own position, counted the same
  float slope2;   // its head's slope, log-2 units
  int64_t qrow;   // row of q and out
  bool valid;     // a row of the chunk (else padding)
};

struct SoftState {
  float m;  // what P is taken against (running maximum)
  float l;  // sum of P
};

// The capped scores' polynomial in registers: packed products take no
// operand from constant memory, and reloading them cost 15 % of the kernel.
struct CappedRegs {
  uint64_t c[5], neg_m2;
};

template <int kMode>
__device__ __forceinline__ CappedRegs capped_regs(const PrefillParams& p) {
  CappedRegs k;
  if (kMode == kPrefillCapped || kMode == kPrefillCappedBiased || kMode == kPrefillGeneral) {
#pragma unroll
    for (int i = 0; i < 5; ++i) asm volatile("mov.b64 %0, %1;" : "=l"(k.c[i]) : "l"(p.cap.c[i]));
    asm volatile("mov.b64 %0, %1;" : "=l"(k.neg_m2) : "l"(p.cap.neg_m2));
  }
  return k;
}

// Bits c of columns 32 w + c that lie in [a, b].
__device__ __forceinline__ uint32_t span_bits(int a, int b, int w) {
  const int lo = max(a - 32 * w, 0), hi = min(b - 32 * w, 31);
  return lo <= hi ? (0xffffffffu << lo) & (0xffffffffu >> (31 - hi)) : 0u;
}

constexpr int kRing = 4;  // item descriptors in flight

// The kernel's mbarriers.
struct ScoredBars {
  uint64_t kfull[2];    // K of a stage landed
  uint64_t vfull[2];    // V of a stage landed
  uint64_t kempty[2];   // both S products reading a stage's K completed
  uint64_t vempty[2];   // both P V products reading a stage's V completed
  uint64_t sfull[2];    // S_t of the next key tile (and PV_t before it) done
  uint64_t pfull[2];    // P_t written (one arrival per warp)
  uint64_t ofull[2];    // an item's last PV_t completed
  uint64_t qfull[2];    // a Q slot written (every lane of warp 10 arrives)
  uint64_t qempty[2];   // the last S product reading a Q slot completed
  uint64_t ifull[kRing];   // an item descriptor published
  uint64_t iempty[kRing];  // every reader is done with it
  uint64_t drain;       // the MMA thread's final wait
  uint64_t taken;       // an answer to the request for another CTA's item
  uint32_t tmem;        // tensor-memory address
  volatile int abort;   // a wait gave up
  int pairs;            // of the sorted list
  int joined;           // the cluster's item is in parts
};

// Wait for phase `parity` of `bar`; give up when another role has given up (*abort)
// or after p.wait_ns (then set *abort and record the timeout).
__device__ __forceinline__ bool wait_role(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          const PrefillParams& p) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    if (global_timer_ns() - t0 > p.wait_ns) {
      *abort = 1;
      record_error(p.err, kErrTimeout);
      return false;
    }
  }
  return true;
}

// The row's running maximum takes in the tile's; O and l are rescaled when it
// grows by more than 2^kRescaleLog2.  Returns the offset P is taken against
// (0 while the row has seen nothing, where every P is masked).
__device__ __forceinline__ float take_max(float tmax, bool first, uint32_t o_tm, SoftState& st) {
  using namespace umma;
  const float m_new = fmaxf(st.m, tmax);
  if (first) {
    st.m = m_new;
  } else {
    const bool grow = m_new > st.m + kRescaleLog2;  // always, from -inf
    if (__any_sync(kFull, grow)) {
      const float alpha = grow ? fast_exp2(st.m - m_new) : 1.f;
      if (grow) {
        st.l *= alpha;
        st.m = m_new;
      }
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t w[32];
        tmem_ld32(w, o_tm + 32 * c);
        tmem_wait_ld(w);
#pragma unroll
        for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * alpha);
        tmem_st32(o_tm + 32 * c, w);
      }
    }
  }
  return st.m == -INFINITY ? 0.f : st.m;
}

// ---- 32 columns ("chunk") of a row, as 16 pairs in registers.  f(i, pair)
// gives pair i's scores; called in order of i.
__device__ __forceinline__ bool bit_of(uint32_t bits, int c) { return (bits >> c) & 1u; }

template <bool kMask, typename F>
__device__ __forceinline__ void chunk_max(const uint32_t (&a)[32], uint32_t bits, F&& f,
                                          float (&mx)[4]) {
  using namespace umma;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x0, x1;
    f2_unpack(f(i, f2_pack(a[2 * i], a[2 * i + 1])), x0, x1);
    if (kMask) {
      x0 = bit_of(bits, 2 * i) ? x0 : -INFINITY;
      x1 = bit_of(bits, 2 * i + 1) ? x1 : -INFINITY;
    }
    mx[i & 3] = fmax3(mx[i & 3], x0, x1);
  }
}

// The largest product of the columns in `bits`.  (The others hold whatever
// stands in rows of K that were not loaded: no choice may hang on it.)
__device__ __forceinline__ float seen_abs_max(const uint32_t (&a)[32], uint32_t bits) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    top = umma::fmax3_abs(top, bit_of(bits, 2 * i) ? __uint_as_float(a[2 * i]) : 0.f,
                          bit_of(bits, 2 * i + 1) ? __uint_as_float(a[2 * i + 1]) : 0.f);
  return top;
}

__device__ __forceinline__ float abs_max(const uint32_t (&a)[32]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    top = umma::fmax3_abs(top, __uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1]));
  return top;
}

// P = 2^f, packed into pk[0..15], summed into ls: where columns are masked, as
// rounded to bf16, so that the rounding cancels in a row that sees few keys
// (one key's output is its value); over whole tiles before it (two operations
// a pair less), where the roundings average out.
template <bool kMask, typename F>
__device__ __forceinline__ void chunk_p(const uint32_t (&a)[32], uint32_t bits, F&& f,
                                        uint32_t* pk, uint64_t (&ls)[4]) {
  using namespace umma;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x0, x1;
    f2_unpack(f(i, f2_pack(a[2 * i], a[2 * i + 1])), x0, x1);
    float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
    if (kMask) {
      e0 = bit_of(bits, 2 * i) ? e0 : 0.f;
      e1 = bit_of(bits, 2 * i + 1) ? e1 : 0.f;
    }
    pk[i] = pack_bf16x2(e0, e1);
    ls[i & 3] = f2_add(ls[i & 3], kMask ? f2_pack(pk[i] << 16, pk[i] & 0xffff0000u)
                                        : f2_pack(__float_as_uint(e0), __float_as_uint(e1)));
  }
}

__device__ __forceinline__ float sum_of(const uint64_t (&ls)[4]) {
  using namespace umma;
  float l0, l1, l2, l3;
  f2_unpack(f2_add(ls[0], ls[1]), l0, l1);
  f2_unpack(f2_add(ls[2], ls[3]), l2, l3);
  return (l0 + l2) + (l1 + l3);
}

// A tile as a row sees it (columns c0 .. c1) and as the rows of its warp do.
struct TileMask {
  int c0, c1;
  bool whole;    // every row sees every column
  bool none[2];  // no row sees a column of this half
  __device__ __forceinline__ uint32_t bits(int chunk) const { return span_bits(c0, c1, chunk); }
};

__device__ __forceinline__ TileMask tile_mask(const ScoredRow& r, int kt) {
  using namespace umma;
  TileMask m;  // (kt is far below 2^31 where hi is not)
  m.c0 = r.lo > kt ? (r.lo - kt > 128 ? 128 : r.lo - kt) : 0;
  m.c1 = r.hi < kt ? -1 : (r.hi - kt > 127 ? 127 : r.hi - kt);
  m.whole = __all_sync(kFull, m.c0 == 0 && m.c1 == 127);
  m.none[0] = m.none[1] = false;
  if (!m.whole) {
    m.none[0] = !__any_sync(kFull, m.c0 < 64 && m.c1 >= 0 && m.c0 <= m.c1);
    m.none[1] = !__any_sync(kFull, m.c1 >= 64 && m.c0 <= m.c1);
  }
  return m;
}

// A whole row of S, in one tensor-memory round trip (335 to 375 cycles).
struct Row128 {
  uint32_t a[32], b[32], c[32], d[32];
  __device__ __forceinline__ explicit Row128(uint32_t s_tm) {
    using namespace umma;
    tmem_ld32(a, s_tm);
    tmem_ld32(b, s_tm + 32);
    tmem_ld32(c, s_tm + 64);
    tmem_ld32(d, s_tm + 96);
    tmem_wait_ld(a);
    tmem_ready(b);
    tmem_ready(c);
    tmem_ready(d);
  }
};

__device__ __forceinline__ void load_half(uint32_t (&a)[32], uint32_t (&b)[32], uint32_t tm) {
  using namespace umma;
  tmem_ld32(a, tm);
  tmem_ld32(b, tm + 32);
  tmem_wait_ld(a);
  tmem_ready(b);
}

__device__ __forceinline__ uint64_t f2_both(float x) {
  return umma::f2_pack(__float_as_uint(x), __float_as_uint(x));
}

// The linear bias of consecutive pairs: start + slope (2i, 2i + 1), along four
// chains of additions.
struct BiasPairs {
  uint64_t t[4], step;
  __device__ __forceinline__ BiasPairs(float start, float slope) {
    using namespace umma;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      t[k] = f2_pack(__float_as_uint(fmaf(slope, static_cast<float>(2 * k), start)),
                     __float_as_uint(fmaf(slope, static_cast<float>(2 * k + 1), start)));
    const uint32_t s8 = __float_as_uint(8.f * slope);
    step = f2_pack(s8, s8);
  }
  __device__ __forceinline__ uint64_t next(int i) {
    const uint64_t r = t[i & 3];
    t[i & 3] = umma::f2_add(r, step);
    return r;
  }
};

__device__ __forceinline__ void zero_p(uint32_t (&pk)[32]) {
#pragma unroll
  for (int i = 0; i < 32; ++i) pk[i] = 0u;
}

// The largest raw product of 32 columns.
template <bool kMask>
__device__ __forceinline__ float chunk_top(const uint32_t (&a)[32], uint32_t bits) {
  float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  chunk_max<kMask>(a, bits, [](int, uint64_t s2) { return s2; }, mx);
  return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// Whether a row's bias is too steep for the paths that add it up along a row or
// take it from m in one rounding.  Sums along a row are off by the slope times
// 2^-17, and the rounding of m by the largest bias times 2^-25: of slopes of a
// million either moves the key of the largest score by many units, and its P
// underflows.  Such a row's scores are each rounded once, where m is found and
// where it is subtracted, so the largest is m to the bit.
__device__ __forceinline__ bool steep_row(const ScoredRow& r) { return fabsf(r.slope2) > 2.f; }

// A tile against the running maximum; scale >= 0, no cap.  Two passes over S:
// with the row held in registers between them the kernel spills (measured a
// quarter slower).
//
// With a bias the maximum is a bound: the largest product of 32 columns and
// their largest bias, at most 31 slopes above the largest score (2^-62 keeps P
// far from underflow; steeper slopes take the scores one by one, see steep_row).  The scores'
// own maximum costs two more operations a pair (8 x 2048 tokens 305 us).
template <int kMode>
__device__ __forceinline__ void tile_running_max(const PrefillParams& p, const ScoredRow& r,
                                                 uint32_t s_tm, uint32_t o_tm, int kt, bool first,
                                                 SoftState& st) {
  using namespace umma;
  constexpr bool kBias = kMode == kPrefillBiased;
  const TileMask mask = tile_mask(r, kt);
  const uint64_t sc2 = f2_pack(__float_as_uint(p.qscale), __float_as_uint(p.qscale));
  const float at = static_cast<float>(r.pos - kt);  // distance of column 0
  uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
  // past a row's own position (seen under a prefix only) the distance grows
  // again; up to it the bias is linear in the column
  const bool bent = kBias && __any_sync(kFull, r.hi > r.pos && r.pos < kt + 127);
  const bool steep = kBias && __any_sync(kFull, steep_row(r));
  // the largest score there can be in columns c .. c + 31, by their largest product
  auto bound = [&](float top, int c) {
    if (!kBias) return top * p.qscale;
    const float d0 = fabsf(at - c), d1 = fabsf(at - (c + 31));
    const float far = fmaxf(d0, d1);
    const float near = at >= c && at <= c + 31 ? 0.f : fminf(d0, d1);
    return fmaf(top, p.qscale, -r.slope2 * (r.slope2 >= 0.f ? near : far));
  };
  if (mask.whole && !bent && !steep) {
    // Loads of S take 335 to 375 cycles.  The maximum comes from one load of
    // the row; its last chunk stays in registers, and the others come again,
    // each during the exponentials of the one before.
    Row128 s(s_tm);
    float tmax;
    if (kBias) {
      tmax = fmaxf(fmaxf(bound(chunk_top<false>(s.a, 0u), 0), bound(chunk_top<false>(s.b, 0u), 32)),
                   fmaxf(bound(chunk_top<false>(s.c, 0u), 64), bound(chunk_top<false>(s.d, 0u), 96)));
    } else {
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      auto raw = [](int, uint64_t s2) { return s2; };
      chunk_max<false>(s.a, 0u, raw, mx);
      chunk_max<false>(s.b, 0u, raw, mx);
      chunk_max<false>(s.c, 0u, raw, mx);
      chunk_max<false>(s.d, 0u, raw, mx);
      tmax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.qscale;
    }
    const float m = take_max(tmax, first, o_tm, st);
    uint32_t x[32], y[32], p0[32], p1[32];
    tmem_ld32(x, s_tm);
    const uint64_t nm2 = f2_pack(__float_as_uint(-m), __float_as_uint(-m));
    BiasPairs bias(fmaf(-r.slope2, at - 96.f, -m), r.slope2);
    auto f = [&](int i, uint64_t s2) { return f2_fma(s2, sc2, kBias ? bias.next(i) : nm2); };
    chunk_p<false>(s.d, 0u, f, p1 + 16, ls);
    bias = BiasPairs(fmaf(-r.slope2, at, -m), r.slope2);
    tmem_wait_ld(x);
    tmem_ld32(y, s_tm + 32);
    chunk_p<false>(x, 0u, f, p0, ls);
    tmem_wait_ld(y);
    tmem_ld32(x, s_tm + 64);
    chunk_p<false>(y, 0u, f, p0 + 16, ls);
    tmem_wait_ld(x);
    tmem_st32(s_tm, p0);
    chunk_p<false>(x, 0u, f, p1, ls);
    tmem_st32(s_tm + 32, p1);
    st.l += sum_of(ls);
    return;
  }
  // the scores of columns from `from` away of the row on, either side of it, less
  // `less` in the bias's rounding, and less `after` when they are rounded
  auto exactly = [&](float from, float less, float after) {
    return [=, &p, &r](int i, uint64_t s2) {
      float x0, x1;
      f2_unpack(s2, x0, x1);
      x0 = fmaf(x0, p.qscale, fmaf(-r.slope2, fabsf(from - static_cast<float>(2 * i)), -less));
      x1 = fmaf(x1, p.qscale, fmaf(-r.slope2, fabsf(from - static_cast<float>(2 * i + 1)), -less));
      return f2_add(f2_pack(__float_as_uint(x0), __float_as_uint(x1)), f2_both(-after));
    };
  };
  float tmax = -INFINITY;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    if (h == 0 ? mask.none[0] : mask.none[1]) continue;
    uint32_t a[32], b[32];
    load_half(a, b, s_tm + 64 * h);
    if (steep) {
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      chunk_max<true>(a, mask.bits(2 * h), exactly(at - 64.f * h, 0.f, 0.f), mx);
      chunk_max<true>(b, mask.bits(2 * h + 1), exactly(at - 64.f * h - 32.f, 0.f, 0.f), mx);
      tmax = fmaxf(tmax, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
    } else {
      tmax = fmaxf(tmax, fmaxf(bound(chunk_top<true>(a, mask.bits(2 * h)), 64 * h),
                               bound(chunk_top<true>(b, mask.bits(2 * h + 1)), 64 * h + 32)));
    }
  }
  const float m = take_max(tmax, first, o_tm, st);
  const uint64_t nm2 = f2_pack(__float_as_uint(-m), __float_as_uint(-m));
  auto plain = [&](int, uint64_t s2) { return f2_fma(s2, sc2, nm2); };
  const float less = steep ? 0.f : m, after = steep ? m : 0.f;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t pk[32];
    if (h == 0 ? mask.none[0] : mask.none[1]) {
      zero_p(pk);
    } else {
      uint32_t a[32], b[32];
      load_half(a, b, s_tm + 64 * h);
      const float from = at - 64.f * h;
      if (kBias && !bent && !steep) {
        BiasPairs bias(fmaf(-r.slope2, from, -m), r.slope2);
        auto biased = [&](int i, uint64_t s2) { return f2_fma(s2, sc2, bias.next(i)); };
        chunk_p<true>(a, mask.bits(2 * h), biased, pk, ls);
        chunk_p<true>(b, mask.bits(2 * h + 1), biased, pk + 16, ls);
      } else if (kBias) {
        chunk_p<true>(a, mask.bits(2 * h), exactly(from, less, after), pk, ls);
        chunk_p<true>(b, mask.bits(2 * h + 1), exactly(from - 32.f, less, after), pk + 16, ls);
      } else {
        chunk_p<true>(a, mask.bits(2 * h), plain, pk, ls);
        chunk_p<true>(b, mask.bits(2 * h + 1), plain, pk + 16, ls);
      }
    }
    tmem_st32(s_tm + 32 * h, pk);
  }
  st.l += sum_of(ls);
}

// Any score: it is written back over S in the first pass, for the second.  A
// chunk whose products are all within the cap takes the polynomial.
__device__ __forceinline__ void tile_general(const PrefillParams& p, const CappedRegs& k,
                                             const ScoredRow& r, uint32_t s_tm, uint32_t o_tm,
                                             int kt, bool first, SoftState& st) {
  using namespace umma;
  const TileMask mask = tile_mask(r, kt);
  const uint64_t sc2 = f2_pack(__float_as_uint(p.qscale), __float_as_uint(p.qscale));
  float mx[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) mx[i] = -INFINITY;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    if (c < 2 ? mask.none[0] : mask.none[1]) continue;
    const uint32_t bits = mask.bits(c);
    uint32_t a[32];
    tmem_ld32(a, s_tm + 32 * c);
    tmem_wait_ld(a);
    if (p.sp.cap2 > 0.f && !__all_sync(kFull, seen_abs_max(a, bits) <= p.cap.s_max)) {
#pragma unroll
      for (int e = 0; e < 32; ++e)
        a[e] = __float_as_uint(capped_score(p.sp, __uint_as_float(a[e]) * p.qscale));
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint64_t s2 = f2_pack(a[2 * i], a[2 * i + 1]);
        const uint64_t w2 = f2_mul(s2, s2);
        uint64_t q = f2_fma(w2, k.c[4], k.c[3]);
        q = f2_fma(w2, q, k.c[2]);
        q = f2_fma(w2, q, k.c[1]);
        q = f2_fma(w2, q, k.c[0]);
        float x0, x1;
        f2_unpack(p.sp.cap2 > 0.f ? f2_mul(s2, q) : f2_mul(s2, sc2), x0, x1);
        a[2 * i] = __float_as_uint(x0);
        a[2 * i + 1] = __float_as_uint(x1);
      }
    }
    const float at = static_cast<float>(r.pos - kt - 32 * c);
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const float v = fmaf(-r.slope2, fabsf(at - static_cast<float>(e)), __uint_as_float(a[e]));
      a[e] = __float_as_uint(v);
      mx[e & 3] = bit_of(bits, e) ? fmaxf(mx[e & 3], v) : mx[e & 3];
    }
    tmem_st32(s_tm + 32 * c, a);
  }
  tmem_wait_st();
  const float m = take_max(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), first, o_tm, st);
  const uint64_t nm2 = f2_pack(__float_as_uint(-m), __float_as_uint(-m));
  uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
  auto less_m = [&](int, uint64_t s2) { return f2_add(s2, nm2); };
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t pk[32];
    if (h == 0 ? mask.none[0] : mask.none[1]) {
      zero_p(pk);
    } else {
      uint32_t a[32], b[32];
      load_half(a, b, s_tm + 64 * h);
      chunk_p<true>(a, mask.bits(2 * h), less_m, pk, ls);
      chunk_p<true>(b, mask.bits(2 * h + 1), less_m, pk + 16, ls);
    }
    tmem_st32(s_tm + 32 * h, pk);
  }
  st.l += sum_of(ls);
}

// Under the cap, in one pass: the polynomial, or, where a half tile holds a
// score out of its range, the exponentials.  Past the range the polynomial
// keeps rising (falling), so the sum of P that a row takes from a half tells:
// one product above the cap alone makes it p_high or more, and products below
// -cap, whatever the polynomial gives for them, are lost in a sum of p_low or
// more (64 of them are under 2^-12 of it).  Masked columns add 0, so that
// nothing that stands in them can sway the choice.  (By the largest product
// instead, 8 x 2048 tokens took 300 us for 270.)
__device__ __forceinline__ void tile_capped(const PrefillParams& p, const CappedRegs& k,
                                            const ScoredRow& r, uint32_t s_tm, int kt,
                                            SoftState& st) {
  using namespace umma;
  const TileMask mask = tile_mask(r, kt);
  auto poly = [&](int, uint64_t s2) {
    const uint64_t w2 = f2_mul(s2, s2);
    uint64_t q = f2_fma(w2, k.c[4], k.c[3]);
    q = f2_fma(w2, q, k.c[2]);
    q = f2_fma(w2, q, k.c[1]);
    q = f2_fma(w2, q, k.c[0]);
    return f2_fma(s2, q, k.neg_m2);
  };
  auto in_range = [&](float sum) { return sum >= p.cap.p_low && sum <= p.cap.p_high; };
  bool done[2] = {false, false};
  float sum1 = 0.f;
  uint32_t p1[32];
  if (mask.whole) {
    uint32_t x[32], y[32], p0[32];
    uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
    load_half(x, y, s_tm);
    chunk_p<false>(x, 0u, poly, p0, ls);
    chunk_p<false>(y, 0u, poly, p0 + 16, ls);
    const float sum0 = sum_of(ls);
    done[0] = __all_sync(kFull, in_range(sum0));
    if (done[0]) {
      tmem_st32(s_tm, p0);
      st.l += sum0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) ls[i] = 0ull;
    load_half(x, y, s_tm + 64);
    chunk_p<false>(x, 0u, poly, p1, ls);
    chunk_p<false>(y, 0u, poly, p1 + 16, ls);
    sum1 = sum_of(ls);
    done[1] = __all_sync(kFull, in_range(sum1));
  }
  if (!done[0] || !done[1]) {
    auto far = [&](int, uint64_t s2) {
      float x0, x1;
      f2_unpack(s2, x0, x1);
      x0 = fmaf(p.cap.neg_2cap, fast_rcp(1.f + fast_exp2(x0 * p.cap.exp_k)), p.cap.cap_m);
      x1 = fmaf(p.cap.neg_2cap, fast_rcp(1.f + fast_exp2(x1 * p.cap.exp_k)), p.cap.cap_m);
      return f2_pack(__float_as_uint(x0), __float_as_uint(x1));
    };
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      if (h == 0 ? done[0] : done[1]) continue;
      uint32_t pk[32];
      if (h == 0 ? mask.none[0] : mask.none[1]) {
        zero_p(pk);
      } else {
        const uint32_t bits0 = mask.bits(2 * h), bits1 = mask.bits(2 * h + 1);
        float sum = 0.f;
        bool near = !mask.whole;
        if (near) {
          uint32_t a[32], b[32];
          load_half(a, b, s_tm + 64 * h);
          uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
          chunk_p<true>(a, bits0, poly, pk, ls);
          chunk_p<true>(b, bits1, poly, pk + 16, ls);
          sum = sum_of(ls);
          near = __all_sync(kFull, in_range(sum) || (bits0 | bits1) == 0u);
        }
        if (!near) {
          uint32_t a[32], b[32];
          load_half(a, b, s_tm + 64 * h);
          uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
          chunk_p<true>(a, bits0, far, pk, ls);
          chunk_p<true>(b, bits1, far, pk + 16, ls);
          sum = sum_of(ls);
        }
        st.l += sum;
      }
      tmem_st32(s_tm + 32 * h, pk);
    }
  }
  if (done[1]) {  // (over S of the first half, which is read by now)
    tmem_st32(s_tm + 32, p1);
    st.l += sum1;
  }
}

// Capped and biased, in one pass: a score is at most the cap and the bias of
// the key the row sees at the smallest distance (at the largest, where the
// slope is negative), and its largest is at least -cap and that bias.  So the
// running maximum is that bias alone, known without S, and the cap's offset
// keeps P in range as it does without a bias.
__device__ __forceinline__ void tile_capped_biased(const PrefillParams& p, const CappedRegs& k,
                                                   const ScoredRow& r, uint32_t s_tm,
                                                   uint32_t o_tm, int kt, bool first,
                                                   SoftState& st) {
  using namespace umma;
  const TileMask mask = tile_mask(r, kt);
  const int ati = r.pos - kt;  // distance of column 0
  const float at = static_cast<float>(ati);
  const int near_d = max(max(mask.c0 - ati, ati - mask.c1), 0);
  const int far_d = max(abs(ati - mask.c0), abs(ati - mask.c1));
  const float top_bias =
      mask.c0 <= mask.c1 ? -r.slope2 * static_cast<float>(r.slope2 >= 0.f ? near_d : far_d)
                         : -INFINITY;
  const float m = take_max(top_bias, first, o_tm, st);
  const bool bent = __any_sync(kFull, r.hi > r.pos && r.pos < kt + 127);
  const bool steep = __any_sync(kFull, steep_row(r));
  const bool linear_bias = !bent && !steep;
  float neg_m, unused;
  f2_unpack(k.neg_m2, neg_m, unused);
  BiasPairs bias(0.f, 0.f);
  auto poly = [&](int i, uint64_t s2) {
    const uint64_t w2 = f2_mul(s2, s2);
    uint64_t q = f2_fma(w2, k.c[4], k.c[3]);
    q = f2_fma(w2, q, k.c[2]);
    q = f2_fma(w2, q, k.c[1]);
    q = f2_fma(w2, q, k.c[0]);
    return f2_fma(s2, q, bias.next(i));
  };
  // (bias - m, at 64 h, of a row whose bias is linear over the tile)
  auto linear = [&](int h) { return BiasPairs(fmaf(-r.slope2, at - 64.f * h, neg_m - m), r.slope2); };
  bool done[2] = {false, false};
  uint32_t p1[32];
  float sum1 = 0.f;
  if (mask.whole && linear_bias) {
    uint32_t x[32], y[32], p0[32];
    uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
    load_half(x, y, s_tm);
    bias = linear(0);
    const float top0 = fmaxf(abs_max(x), abs_max(y));
    chunk_p<false>(x, 0u, poly, p0, ls);
    chunk_p<false>(y, 0u, poly, p0 + 16, ls);
    done[0] = __all_sync(kFull, top0 <= p.cap.s_max);
    if (done[0]) {
      tmem_st32(s_tm, p0);
      st.l += sum_of(ls);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) ls[i] = 0ull;
    load_half(x, y, s_tm + 64);
    bias = linear(1);
    const float top1 = fmaxf(abs_max(x), abs_max(y));
    chunk_p<false>(x, 0u, poly, p1, ls);
    chunk_p<false>(y, 0u, poly, p1 + 16, ls);
    sum1 = sum_of(ls);
    done[1] = __all_sync(kFull, top1 <= p.cap.s_max);
  }
  if (!done[0] || !done[1]) {
    const float less = steep ? 0.f : m, after = steep ? m : 0.f;
    auto each = [&](float from) {
      return [=, &p, &r](int i, uint64_t s2) {
        float x0, x1;
        f2_unpack(s2, x0, x1);
        const float b0 = fmaf(-r.slope2, fabsf(from - static_cast<float>(2 * i)), -less);
        const float b1 = fmaf(-r.slope2, fabsf(from - static_cast<float>(2 * i + 1)), -less);
        x0 = fmaf(p.cap.neg_2cap, fast_rcp(1.f + fast_exp2(x0 * p.cap.exp_k)), p.cap.cap_m);
        x1 = fmaf(p.cap.neg_2cap, fast_rcp(1.f + fast_exp2(x1 * p.cap.exp_k)), p.cap.cap_m);
        return f2_add(f2_pack(__float_as_uint(x0), __float_as_uint(x1)),
                      f2_add(f2_pack(__float_as_uint(b0), __float_as_uint(b1)), f2_both(-after)));
      };
    };
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      if (h == 0 ? done[0] : done[1]) continue;
      uint32_t pk[32];
      if (h == 0 ? mask.none[0] : mask.none[1]) {
        zero_p(pk);
      } else {
        const uint32_t bits0 = mask.bits(2 * h), bits1 = mask.bits(2 * h + 1);
        uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
        uint32_t a[32], b[32];
        load_half(a, b, s_tm + 64 * h);
        const bool near = !mask.whole && linear_bias &&
                          fmaxf(seen_abs_max(a, bits0), seen_abs_max(b, bits1)) <= p.cap.s_max;
        if (__all_sync(kFull, near)) {
          bias = linear(h);
          chunk_p<true>(a, bits0, poly, pk, ls);
          chunk_p<true>(b, bits1, poly, pk + 16, ls);
        } else {
          chunk_p<true>(a, bits0, each(at - 64.f * h), pk, ls);
          chunk_p<true>(b, bits1, each(at - 64.f * h - 32.f), pk + 16, ls);
        }
        st.l += sum_of(ls);
      }
      tmem_st32(s_tm + 32 * h, pk);
    }
  }
  if (done[1]) {  // (over S of the first half, which is read by now)
    tmem_st32(s_tm + 32, p1);
    st.l += sum1;
  }
}

// One key tile: kt is its first key counted from the item's.
template <int kMode>
__device__ __forceinline__ void scored_tile(const PrefillParams& p, const CappedRegs& k, const ScoredRow& r,
                                            uint32_t s_tm, uint32_t o_tm, int kt, bool first,
                                            SoftState& st) {
  if constexpr (kMode == kPrefillCapped) tile_capped(p, k, r, s_tm, kt, st);
  else if constexpr (kMode == kPrefillCappedBiased)
    tile_capped_biased(p, k, r, s_tm, o_tm, kt, first, st);
  else if constexpr (kMode == kPrefillGeneral) tile_general(p, k, r, s_tm, o_tm, kt, first, st);
  else tile_running_max<kMode>(p, r, s_tm, o_tm, kt, first, st);
}

// Adds 0 where all 32 values are finite, NaN where one is not.
__device__ __forceinline__ void add_finite(uint64_t& z, const uint32_t (&w)[32]) {
#pragma unroll
  for (int c = 0; c < 16; ++c) z = umma::f2_fma(umma::f2_pack(w[2 * c], w[2 * c + 1]), 0ull, z);
}

__device__ __forceinline__ bool is_zero(uint64_t z) {
  float z0, z1;
  umma::f2_unpack(z, z0, z1);
  return z0 == 0.f && z1 == 0.f;
}

// 64 columns of a row, times inv, as bf16: chunk c (0..7) of 16 bytes.
__device__ __forceinline__ uint4 out_chunk(const uint32_t (&a)[32], const uint32_t (&b)[32],
                                           float inv, int c) {
  const uint32_t* x = c < 4 ? a + 8 * c : b + 8 * (c - 4);
  return make_uint4(pack_bf16x2(__uint_as_float(x[0]) * inv, __uint_as_float(x[1]) * inv),
                    pack_bf16x2(__uint_as_float(x[2]) * inv, __uint_as_float(x[3]) * inv),
                    pack_bf16x2(__uint_as_float(x[4]) * inv, __uint_as_float(x[5]) * inv),
                    pack_bf16x2(__uint_as_float(x[6]) * inv, __uint_as_float(x[7]) * inv));
}

// Column half h of the warp's 32 rows (row = lane) through its 4 KiB of
// staging, 128-byte swizzled, and one tensor store.
__device__ __forceinline__ void store_half_tma(const CUtensorMap* tmo, unsigned char* stg, int lane,
                                               float inv, const uint32_t (&a)[32],
                                               const uint32_t (&b)[32], int h, int head0,
                                               int tok0) {
  using namespace umma;
  if (lane == 0) bulk_wait_read();  // the warp's last store has read the staging
  __syncwarp();
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(stg + lane * 128 + ((c ^ (lane & 7)) << 4)) = out_chunk(a, b, inv, c);
  fence_proxy_async_smem();  // the tensor store reads the staging through the async proxy
  __syncwarp();
  if (lane == 0) {
    tma_store_4d_at(tmo, stg, 0, h, head0, tok0);
    bulk_commit();
  }
}

// 64 columns of one row by plain stores; v8: dst is 32-byte aligned, whole
// 32-byte sectors.
__device__ __forceinline__ void store_half(uint4* dst, float inv, const uint32_t (&a)[32],
                                           const uint32_t (&b)[32], bool v8) {
#pragma unroll
  for (int c = 0; c < 8; c += 2) {
    const uint4 x = out_chunk(a, b, inv, c), y = out_chunk(a, b, inv, c + 1);
    if (v8) {
      umma::st_global_v8(dst + c, x, y);
    } else {
      dst[c] = x;
      dst[c + 1] = y;
    }
  }
}

// 128 columns as bits: column d is bit d / 4 of word d % 4.
struct Columns {
  uint32_t w[4];
};

// The columns of this thread's row of O that are not finite (whole warp).
__device__ __forceinline__ Columns bad_columns(uint32_t o_tm) {
  Columns bad = {};
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t x[32];
    umma::tmem_ld32(x, o_tm + 32 * c);
    umma::tmem_wait_ld(x);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      bad.w[e & 3] |= (x[e] & 0x7f800000u) == 0x7f800000u ? 1u << (8 * c + (e >> 2)) : 0u;
  }
  return bad;
}

// What a row sees in V that is not finite, by column.
struct SeenValues {
  Columns nan, pos, neg;
};

// Looks through the V rows that the warp's flagged rows see, until a NaN is found
// for each of their bad columns.  16 positions at a time (one block: their size is a
// multiple of 16), two a load, 16 lanes each.
static __device__ __noinline__ SeenValues scan_values(const KvRows& kv, bool flagged,
                                                      const Columns& bad, int lo, int hi,
                                                      int lane) {
  constexpr unsigned kAll = 0xffffffffu;
  SeenValues seen = {};
  const bool on = flagged && lo <= hi;
  const int first = __reduce_min_sync(kAll, on ? lo : INT_MAX);
  const int last = __reduce_max_sync(kAll, on ? hi : -1);
  const uint32_t bs = static_cast<uint32_t>(kv.bs);
  const int half = lane >> 4, chunk = lane & 15;  // columns 8 chunk .. 8 chunk + 7
  for (int64_t j0 = first & ~15; j0 <= last; j0 += 16) {
    // (a block that no flagged row sees is not read, nor its table entry)
    if (!__any_sync(kAll, on && lo < j0 + 16 && hi >= j0)) continue;
    const uint32_t at = static_cast<uint32_t>(j0);
    const int32_t blk = kv.table[at / bs];
    if (kv.checked && (blk < 0 || blk >= kv.num_blocks)) {
      record_error(kv.err, kv.err_code);
      continue;
    }
    const uint16_t* v = kv.v + (cache_row(blk, kv.kvh, kv.Hkv, kv.bs, at % bs) + half) * kHeadDim +
                        chunk * 8;
    // an exponent of all ones carries into the sign's place
    auto ones_of = [](const uint4& x) {
      return ((((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
               ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u)) &
              0x80008000u);
    };
    uint32_t hit = 0u;  // loads that bring a value that is not finite
#pragma unroll
    for (int g = 0; g < 8; g += 4) {
      uint4 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = ld_global_nc_v4(v + 2 * (g + u) * kHeadDim);
#pragma unroll
      for (int u = 0; u < 4; ++u) hit |= ones_of(x[u]) != 0u ? 1u << (g + u) : 0u;
    }
    for (hit = __reduce_or_sync(kAll, hit); hit != 0u; hit &= hit - 1) {
      const int u = __ffs(hit) - 1;
      const uint4 x = ld_global_nc_v4(v + 2 * u * kHeadDim);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      Columns nan = {}, pos = {}, neg = {};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = (e & 1 ? w[e >> 1] >> 16 : w[e >> 1]) & 0xffffu;
        const uint32_t bit = 1u << (2 * chunk + (e >> 2));
        if ((b & 0x7fffu) > 0x7f80u) nan.w[e & 3] |= bit;
        else if (b == 0x7f80u) pos.w[e & 3] |= bit;
        else if (b == 0xff80u) neg.w[e & 3] |= bit;
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {  // position j0 + 2 u + r
        const int64_t j = j0 + 2 * u + r;
        const bool sees = on && lo <= j && j <= hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t n = __reduce_or_sync(kAll, half == r ? nan.w[i] : 0u);
          const uint32_t p = __reduce_or_sync(kAll, half == r ? pos.w[i] : 0u);
          const uint32_t m = __reduce_or_sync(kAll, half == r ? neg.w[i] : 0u);
          if (sees) {
            seen.nan.w[i] |= n;
            seen.pos.w[i] |= p;
            seen.neg.w[i] |= m;
          }
        }
      }
      uint32_t open = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) open |= bad.w[i] & ~seen.nan.w[i];
      if (!__any_sync(kAll, on && open != 0u)) return seen;
    }
  }
  return seen;
}

// Puts the warp's flagged rows (a thread's row each, `bad` its columns that are
// not finite) right.  Such a column holds what the formula gives where the row
// sees a value of V that is not finite: that value (NaN where it sees several
// kinds), which is written.  Else it met one that it does not see (0 times a
// NaN or an infinity is NaN), and the row is computed again by itself.
//
// So the rows computed again are those beside a masked value that is not finite,
// in a column where they see none: a value that every later token sees costs its
// own work item the rows before it, and the items after it one look through V.
// (Each row that is not finite computed again, one NaN in a prompt's first tokens
// cost every later row its whole context.)
static __device__ __noinline__ void repair_rows(const PrefillParams& p, const KvRows& kv,
                                                bool flagged, const Columns& bad,
                                                const ScoredRow& r, int k0, int lane) {
  const bool sees = r.lo <= r.hi;
  const SeenValues seen = scan_values(kv, flagged, bad, sees ? r.lo + k0 : 0,
                                      sees ? r.hi + k0 : -1, lane);
  uint32_t unexplained = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    unexplained |= bad.w[i] & ~(seen.nan.w[i] | seen.pos.w[i] | seen.neg.w[i]);
  if (flagged && unexplained == 0u) {
    uint16_t* out = p.out + r.qrow * kHeadDim;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      for (uint32_t left = bad.w[i]; left != 0u; left &= left - 1) {
        const int b = __ffs(left) - 1;
        const bool nan = (seen.nan.w[i] | (seen.pos.w[i] & seen.neg.w[i])) >> b & 1u;
        out[4 * b + i] = nan ? 0x7fffu : seen.pos.w[i] >> b & 1u ? 0x7f80u : 0xff80u;
      }
  }
  for (uint32_t left = __ballot_sync(umma::kFull, flagged && unexplained != 0u); left != 0u;
       left &= left - 1) {
    const int src = __ffs(left) - 1;
    const int64_t row = __shfl_sync(umma::kFull, r.qrow, src);
    const int lo = __shfl_sync(umma::kFull, r.lo, src), hi = __shfl_sync(umma::kFull, r.hi, src);
    const int pos = __shfl_sync(umma::kFull, r.pos, src);
    const float slope2 = __shfl_sync(umma::kFull, r.slope2, src);
    const bool none = lo > hi;
    float o[16];
    attend_row(p.sp, kv, p.q + row * kHeadDim, p.qscale, slope2, pos + k0, none ? 0 : lo + k0,
               none ? -1 : hi + k0, lane, o);
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
