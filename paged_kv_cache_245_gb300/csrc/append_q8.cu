// append_q8.cu -- new keys and values quantised into the 8-bit cache, with or
// without rotary positions on the way.
//
// For each group of 16 slots that the call writes to, each head, K and V by
// themselves:
//   a   = max |x| over the new rows' finite elements
//   old = 0 if the group's first row is new (the group starts anew), else its scale
//   s   = max(old, a / qmax), qmax = 127 (int8) or 448 (e4m3);  inv = 1 / s
//   new rows x:  code = round(x inv);  kept rows: code = round(code old inv)
// all in fp32, each product rounded once, so that the codes are the formula's
// bit for bit.  Kept rows change only when the scale grows; rows of a group that
// starts anew and that the call does not write become zero.
//
// Tokens may come in any order.  A CTA takes a tile of tokens, enters their
// groups into a hash table in shared memory and passes once over the call's
// slots, which gives each group's first token and, row by row, the last token
// that writes it.  The CTA that holds a group's first token does the whole
// group; so no two CTAs touch one group, and the result does not depend on
// their order.
//
// A warp takes a (group, head, K or V): 16 rows x 256 bytes are 64 elements a
// lane, all in registers between the maximum and the rounding, so that every row
// is read once.
#include <cuda_bf16.h>

#include "pkv_device.cuh"
#include "q8.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTile = 64;           // tokens a CTA
constexpr int kTable = 4 * kMaxTile;   // hash slots (a power of two)
constexpr int kBatch = 2;              // groups whose sines are in shared memory at once
constexpr unsigned kFull = 0xffffffffu;

// (cos, sin) of pair i of a token at cs_at(i): padded so that lanes that read
// 8 (half layout) or 4 (interleaved) pairs apart meet different banks.
__device__ __forceinline__ constexpr int cs_at(int pair) { return pair + (pair >> 3) * 2; }
constexpr int kSines = cs_at(64);

__device__ __forceinline__ float2 sines(const pkv_rope& rope, int32_t position, int pair) {
  if (pair >= (rope.rotary_dim >> 1)) return make_float2(1.f, 0.f);
  // position times turns, exact modulo a turn; a signed fraction in units of 2^-63 half turns
  const int64_t turn = static_cast<int64_t>(static_cast<uint64_t>(static_cast<int64_t>(position)) *
                                            rope.turn[pair]);
  float2 c;
  sincospif(static_cast<float>(turn) * 1.0842021724855044e-19f, &c.y, &c.x);
  return make_float2(c.x * rope.gain, c.y * rope.gain);
}

// An element of a turned pair; y is the other one, negated for the first.
__device__ __forceinline__ float turned(float x, float y, float2 cs) {
  return __fmaf_rn(x, cs.x, __fmul_rn(y, cs.y));
}

// Eight elements of a row, chunk c of the 16 lanes that hold it, turned.  Every
// lane of the warp calls; a row lies in one half of the warp.
__device__ __forceinline__ void turn_chunk(const pkv_rope& rope, const float2* cs, int c,
                                           float (&x)[8]) {
  const int rd = rope.rotary_dim, half = rd >> 1;
  if (rope.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pair = c * 4 + i;
      if (pair < half) {
        const float2 f = cs[cs_at(pair)];
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = turned(a, -b, f);
        x[2 * i + 1] = turned(b, a, f);
      }
    }
    return;
  }
  // partner of element e: e + half below half, e - half from there to rd.  It is
  // element (e +- half) & 7 of chunk (e +- half) >> 3 of the same row.
  float y[8];
  const int lane = threadIdx.x & 31;
  if ((half & 7) == 0) {
    const int by = half >> 3;
    const int other = c < by ? c + by : (c < 2 * by ? c - by : c);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(kFull, x[i], (lane & 16) | other);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = c * 8 + i;
      const int want = e < half ? e + half : (e < rd ? e - half : e);
      float got = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float v = __shfl_sync(kFull, x[j], (lane & 16) | (want >> 3));
        if (j == (want & 7)) got = v;
      }
      y[i] = got;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = c * 8 + i;
    if (e < rd) {
      const bool lower = e < half;
      const float2 f = cs[cs_at(lower ? e : e - half)];
      x[i] = turned(x[i], lower ? -y[i] : y[i], f);
    }
  }
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(u[i]);
    x[2 * i + 1] = bf16_hi(u[i]);
  }
}

// Four values in units of the scale as codes.
template <bool kE4m3>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  if (kE4m3) return to_e4m3x2(a, b) | (to_e4m3x2(c, d) << 16);
  // rint by the addition of 1.5 2^23, whose low byte is then the code; NaN: 0
  const float x[4] = {a, b, c, d};
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float y = fminf(fmaxf(x[i], -kInt8Max), kInt8Max);
    const uint32_t u = __float_as_uint(__fadd_rn(x[i] == x[i] ? y : 0.f, 12582912.f));
    r |= (u & 255u) << (8 * i);
  }
  return r;
}

template <bool kE4m3>
__device__ __forceinline__ float code_value(uint32_t byte) {
  if (kE4m3) {
    const uint32_t h = e4m3x2_to_half2(byte & 255u);
    float f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h));
    return f;
  }
  return static_cast<float>(static_cast<int8_t>(byte));
}

struct GroupTable {
  unsigned long long key[kTable];  // group + 1, or 0
  int32_t first[kTable];           // lowest token of the group
  int32_t token[kTable][kGroupRows];  // token that writes the row, or -1
  int32_t owned[kTable];           // table slots of the groups that this CTA does
  int32_t num_owned;
};

__device__ __forceinline__ int hash_of(unsigned long long key) {
  return static_cast<int>((key * 0x9E3779B97F4A7C15ull) >> 40) & (kTable - 1);
}

// One (group, head, tensor) of the call, by a warp.
template <bool kE4m3, bool kRope>
__device__ __forceinline__ void put_unit(const AppendQ8Params& p, const int32_t* token,
                                         const float2 (*cs)[kSines], int64_t group, int h,
                                         bool is_v) {
  constexpr float kMax = kE4m3 ? kE4m3Max : kInt8Max;
  const int lane = threadIdx.x & 31, c = lane & 15, odd = lane >> 4;
  const uint16_t* src = (is_v ? p.v : p.k) + h * kHeadDim + c * 8;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  const int64_t slot = group * kGroupRows;
  const int64_t row0 = cache_row(slot / p.bs, h, p.Hkv, p.bs, slot % p.bs);
  uint8_t* dst = (is_v ? p.v_codes : p.k_codes) + row0 * kCodeRowBytes + c * 8;
  float* scale = (is_v ? p.v_scale : p.k_scale) + row0 / kGroupRows;
  const bool started = token[0] >= 0;
  float old = started ? 0.f : *scale;
  if (!(old > 0.f && old <= 3.402823466e38f)) old = 0.f;

  uint4 raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int t = token[2 * i + odd];
    raw[i] = t >= 0 ? ld_global_nc_v4(src + t * stride) : make_uint4(0u, 0u, 0u, 0u);
  }
  float x[8][8];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    unpack8(raw[i], x[i]);
    if (kRope && !is_v) turn_chunk(p.rope, cs[2 * i + odd], c, x[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = fabsf(x[i][j]);
      top = fmaxf(top, a <= 3.402823466e38f ? a : 0.f);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  const float s = fmaxf(old, __fdiv_rn(top, kMax));
  const float inv = s >= kScaleTiny ? __frcp_rn(s) : 0.f;
  if (lane == 0) *scale = s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = 2 * i + odd;
    uint2* at = reinterpret_cast<uint2*>(dst + row * kCodeRowBytes);
    float y[8];
    if (token[row] >= 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = __fmul_rn(x[i][j], inv);
    } else if (started) {
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = 0.f;
    } else {
      if (s == old) continue;
      const uint2 held = *at;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        y[j] = __fmul_rn(__fmul_rn(code_value<kE4m3>((j < 4 ? held.x : held.y) >> (8 * (j & 3))), old),
                         inv);
    }
    *at = make_uint2(codes4<kE4m3>(y[0], y[1], y[2], y[3]), codes4<kE4m3>(y[4], y[5], y[6], y[7]));
  }
}

// Query rows of tokens t0 .. t0 + n - 1 turned into q_out.
__device__ __forceinline__ void turn_queries(const AppendQ8Params& p, int t0, int n,
                                             float2 (*cs)[kSines]) {
  for (int e = threadIdx.x; e < n * 64; e += kThreads)
    cs[e >> 6][cs_at(e & 63)] = sines(p.rope, p.positions[t0 + (e >> 6)], e & 63);
  __syncthreads();
  const int c = threadIdx.x & 15;
  const int rows = n * p.Hq;
  // whole warps take part in the shuffles of turn_chunk
  for (int r0 = (threadIdx.x >> 5) * 2; r0 < rows; r0 += kWarps * 2) {
    const int r = min(r0 + ((threadIdx.x >> 4) & 1), rows - 1);
    const int tok = r / p.Hq;
    const int64_t t = t0 + tok;
    const int h = r - tok * p.Hq;
    const uint4 w = *reinterpret_cast<const uint4*>(p.q + t * p.q_stride + h * kHeadDim + c * 8);
    float x[8];
    unpack8(w, x);
    turn_chunk(p.rope, cs[tok], c, x);
    if (r0 + ((threadIdx.x >> 4) & 1) < rows)
      *reinterpret_cast<uint4*>(p.q_out + (t * p.Hq + h) * kHeadDim + c * 8) =
          make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                     pack_bf16x2(x[6], x[7]));
  }
}

constexpr int kQueryTokens = 4;  // tokens of a CTA that turns queries

template <bool kE4m3, bool kRope>
__global__ void __launch_bounds__(kThreads)
    append_q8_kernel(const __grid_constant__ AppendQ8Params p, int tile, int kv_ctas) {
  __shared__ GroupTable g;
  __shared__ __align__(16) float2 cs[kRope ? kBatch * kGroupRows : 1][kSines];
  grid_dependency_trigger();
  grid_dependency_wait();
  const int tid = threadIdx.x;
  if constexpr (kRope) {
    if (static_cast<int>(blockIdx.x) >= kv_ctas) {
      const int t0 = (static_cast<int>(blockIdx.x) - kv_ctas) * kQueryTokens;
      turn_queries(p, t0, min(kQueryTokens, p.num_tokens - t0), cs);
      return;
    }
  }
  const int t0 = blockIdx.x * tile;
  const int t1 = min(t0 + tile, p.num_tokens);
  for (int i = tid; i < kTable; i += kThreads) {
    g.key[i] = 0ull;
    g.first[i] = 0x7fffffff;
#pragma unroll
    for (int r = 0; r < kGroupRows; ++r) g.token[i][r] = -1;
  }
  if (tid == 0) g.num_owned = 0;
  __syncthreads();
  // the slot's group + 1, or 0: a token whose rows go nowhere
  auto key_of = [&](int64_t slot) -> unsigned long long {
    if (slot < 0 || (p.checked && slot >= p.num_slots)) return 0ull;
    return static_cast<unsigned long long>(slot / kGroupRows) + 1ull;
  };
  for (int t = t0 + tid; t < t1; t += kThreads) {
    const int64_t slot = p.slot_mapping[t];
    if (p.checked && slot >= p.num_slots) record_error(p.err, kErrSlot);
    const unsigned long long key = key_of(slot);
    if (key == 0ull) continue;
    int at = hash_of(key);
    while (true) {  // at most kMaxTile of kTable slots are taken
      const unsigned long long was = atomicCAS(&g.key[at], 0ull, key);
      if (was == 0ull || was == key) break;
      at = (at + 1) & (kTable - 1);
    }
  }
  __syncthreads();
  for (int t = tid; t < p.num_tokens; t += kThreads) {
    const int64_t slot = p.slot_mapping[t];
    const unsigned long long key = key_of(slot);
    if (key == 0ull) continue;
    int at = hash_of(key);
    unsigned long long have;
    while ((have = g.key[at]) != key && have != 0ull) at = (at + 1) & (kTable - 1);
    if (have == key) {
      atomicMin(&g.first[at], t);
      atomicMax(&g.token[at][slot % kGroupRows], t);
    }
  }
  __syncthreads();
  for (int i = tid; i < kTable; i += kThreads)
    if (g.key[i] != 0ull && g.first[i] >= t0) g.owned[atomicAdd(&g.num_owned, 1)] = i;
  __syncthreads();
  const int n = g.num_owned;
  const int per = 2 * p.Hkv;
  const int warp = tid >> 5;
  if constexpr (!kRope) {
    for (int u = warp; u < n * per; u += kWarps) {
      const int at = g.owned[u / per], e = u % per;
      put_unit<kE4m3, false>(p, g.token[at], nullptr, static_cast<int64_t>(g.key[at] - 1ull),
                             e >> 1, e & 1);
    }
  } else {
  for (int b0 = 0; b0 < n; b0 += kBatch) {
    const int nb = min(kBatch, n - b0);
    for (int e = tid; e < nb * kGroupRows * 64; e += kThreads) {
      const int row = e >> 6;
      const int t = g.token[g.owned[b0 + row / kGroupRows]][row % kGroupRows];
      if (t >= 0) cs[row][cs_at(e & 63)] = sines(p.rope, p.positions[t], e & 63);
    }
    __syncthreads();
    for (int u = warp; u < nb * per; u += kWarps) {
      const int b = u / per, e = u % per;
      const int at = g.owned[b0 + b];
      put_unit<kE4m3, true>(p, g.token[at],
                            &cs[b * kGroupRows],
                            static_cast<int64_t>(g.key[at] - 1ull), e >> 1, e & 1);
    }
    __syncthreads();
  }
  }
}

template <bool kE4m3, bool kRope>
cudaError_t launch(const AppendQ8Params& p, cudaStream_t stream) {
  // A few hundred CTAs where there are tokens for them, up to 32 tokens each;
  // more past 32768, so that the passes over all slots stay few.
  int tile = (p.num_tokens + 303) / 304;
  tile = tile < 1 ? 1 : (tile > 32 ? 32 : tile);
  if (p.num_tokens > 32768) tile = kMaxTile;
  const int kv = (p.num_tokens + tile - 1) / tile;
  const int qs = kRope ? (p.num_tokens + kQueryTokens - 1) / kQueryTokens : 0;
  return launch_pdl(append_q8_kernel<kE4m3, kRope>, dim3(static_cast<unsigned>(kv) + qs),
                    dim3(kThreads), 0, stream, p, tile, kv);
}

}  // namespace

cudaError_t launch_append_q8(const AppendQ8Params& p, bool e4m3, bool rope, cudaStream_t stream) {
  if (p.num_tokens <= 0) return cudaSuccess;
  if (e4m3) return rope ? launch<true, true>(p, stream) : launch<true, false>(p, stream);
  return rope ? launch<false, true>(p, stream) : launch<false, false>(p, stream);
}

}  // namespace pkv
