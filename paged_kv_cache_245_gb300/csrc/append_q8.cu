// append_q8.cu -- new keys and values quantised into the 8-bit cache, with or
// without rotary positions on the way.
//
// For each group of 16 slots that the call writes to, each head, K and V by
// themselves:
//   a   = max |x| over the new rows' finite elements
//   old = 0 if the group's first row is new (the group starts anew), else its scale
//   s   = max(old, a r), r = 1 / qmax in fp32, qmax = 127 (int8) or 448 (e4m3);  inv = 1 / s
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
// their order.  In the pass a bit for each of the table's groups turns most
// slots away before the table is looked at.
//
// A warp takes a (group, head, K or V): 16 rows x 256 bytes are 64 elements a
// lane, all in registers between the maximum and the rounding, so that every row
// is read once.  8 lanes hold a row, each two chunks of 8 elements, as in
// rope_rows.cuh: a lane has both elements of its turned pairs.
//
// What bounds it: for few tokens three dependent reads (slot, slots, rows) and the scale;
// for prompts the wait for rows (a warp loads a unit, takes its maximum, rounds and stores
// it, and only then asks for the next; DRAM is at 42 % of its peak).  One CTA an SM, as
// large as the registers allow, keeps the passes over the slots few and every SM as busy
// as the next; with 32 tokens a CTA and three CTAs an SM 16384 tokens took 32 us.  The
// maximum on the bf16 bits, two at a time, took the larger part of the arithmetic away (75
// to 32 us with the filter).  8 KV heads, us: 1 token 4.1, 64 of as many sequences 4.4, 256
// 5.8; prompts of 1000 5.1, 4096 10.1, 16384 21.6 (101 MB: 4.7 TB/s, 0.69 of a plain copy),
// 65536 70 (5.7 TB/s, 0.85).  With rotary positions and 32 query heads: 1 5.7, 300 7.3, 1000
// 11.8, 4096 27, 16384 77 (369 MB: 4.8 TB/s, 0.71); there the keys' turn, in fp32 until
// they are rounded, takes some 120 registers a thread.
#include <cuda_bf16.h>

#include "decode_launch.cuh"
#include "pkv_device.cuh"
#include "q8.cuh"
#include "rope_rows.cuh"
#include "umma.cuh"

namespace pkv {

namespace {

constexpr int kMaxTile = 512;          // tokens a CTA
constexpr int kMaxTable = 2 * kMaxTile;  // hash slots (a power of two)
constexpr int kMinTable = 64;
constexpr int kFilter = 4096;          // bits
constexpr int kScan = 8;               // slots that a thread has on the way
// Tokens whose queries are turned by CTAs of the same launch; past that by a launch of
// rope.cu's, of whose CTAs an SM holds five (256 tokens 7.3 us for 9.7, 600 8.4 for 11.3,
// 1000 11.5 for 12.3; 1300 15.2 for 13.9, 4096 38.8 for 27.2).
constexpr int kTogether = 1000;
constexpr int kBatch = 4;              // groups whose sines are in shared memory at once
constexpr unsigned kFull = 0xffffffffu;

// Threads of a CTA, one an SM: what the registers of a unit leave room for.
__host__ __device__ constexpr int threads_of(int kind) { return kind < 0 ? 768 : 512; }

// (cos, sin) times gain of a pair at a position.  position times turns is exact modulo
// a turn, in units of 2^-64 turns; less the nearest quarter turn it is at most 2^61 of
// them, 1/4 half turn, and what its conversion to fp32 leaves (2^-27 half turns at most)
// goes in by the first term of the series: a key that lies next to the border of two
// codes shall fall on the side of its exact value as seldom wrong as the products allow
// (rope_rows, whose results are rounded to bf16, converts the whole fraction).
__device__ __forceinline__ float2 rope_sines(const pkv_rope& rope, int32_t position, int pair) {
  if (pair >= (rope.rotary_dim >> 1)) return make_float2(1.f, 0.f);
  const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(position)) * rope.turn[pair];
  const int quarter = static_cast<int>((turn + (uint64_t{1} << 61)) >> 62);
  const int64_t rest = static_cast<int64_t>(turn - (static_cast<uint64_t>(quarter) << 62));
  const float high = static_cast<float>(rest);
  const float low = static_cast<float>(rest - static_cast<int64_t>(high));
  float s, c;
  sincospif(high * 1.0842021724855044e-19f, &s, &c);  // 2^-63
  const float by = low * 3.406121578e-19f;            // pi 2^-63
  const float s1 = fmaf(c, by, s), c1 = fmaf(-s, by, c);
  float2 r = quarter & 1 ? make_float2(-s1, c1) : make_float2(c1, s1);
  if (quarter & 2) r = make_float2(-r.x, -r.y);
  return make_float2(r.x * rope.gain, r.y * rope.gain);
}

// An element of a turned pair; y is the other one, negated for the first.
__device__ __forceinline__ float turned_one(float x, float y, float2 cs) {
  return __fmaf_rn(x, cs.x, __fmul_rn(y, cs.y));
}

__device__ __forceinline__ void turn_pair(float& x, float& y, float2 cs) {
  const float a = turned_one(x, -y, cs);
  y = turned_one(y, x, cs);
  x = a;
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
  unsigned long long key[kMaxTable];  // group + 1, or 0
  int32_t first[kMaxTable];           // lowest token of the group
  uint32_t filter[kFilter / 32];      // a bit for each group of the table
  int32_t owned[kMaxTile];            // table slots of the groups that this CTA does
  int32_t num_owned;
  // last, as only a launch's table is asked for: the token that writes a row, or -1
  alignas(16) int32_t token[kMaxTable][kGroupRows];
};

__device__ __forceinline__ int hash_of(unsigned long long key, int mask) {
  return static_cast<int>((key * 0x9E3779B97F4A7C15ull) >> 40) & mask;
}

// Bit of the filter of a slot's group.
__device__ __forceinline__ uint32_t filter_bit(int64_t slot) {
  return (static_cast<uint32_t>(slot >> 4) * 0x9E3779B9u) >> 20;
}
static_assert(kGroupRows == 16 && kFilter == 1 << 12, "filter_bit");

// A unit of the call: a (group, head, K or V), by a warp.  Lane 8 r + l holds rows
// 4 i + r, of each two chunks of 8 elements.
struct Unit {
  const int32_t* token;  // [16]
  const uint16_t* src;   // the head's elements of token 0
  int64_t stride;
  uint8_t* codes;        // of the group's first row
  float* scale;
};

__device__ __forceinline__ Unit unit_at(const AppendQ8Params& p, const int32_t* token, int64_t group,
                                        int h, bool is_v) {
  const int64_t slot = group * kGroupRows;
  const int64_t row = cache_row(slot / p.bs, h, p.Hkv, p.bs, slot % p.bs);
  Unit u;
  u.token = token;
  u.src = (is_v ? p.v : p.k) + h * kHeadDim;
  u.stride = is_v ? p.v_stride : p.k_stride;
  u.codes = (is_v ? p.v_codes : p.k_codes) + row * kCodeRowBytes;
  u.scale = (is_v ? p.v_scale : p.k_scale) + row / kGroupRows;
  return u;
}

// The group's scale before the call; 0 if it starts anew, or if no append wrote it.
__device__ __forceinline__ float scale_before(const Unit& u) {
  const float old = u.token[0] >= 0 ? 0.f : *u.scale;
  return old > 0.f && old <= 3.402823466e38f ? old : 0.f;
}

// Eight finite values x / scale as codes: |x inv| is at most qmax (1 + 2^-21), which
// rounds to qmax.  v: pairs.
template <bool kE4m3>
__device__ __forceinline__ uint2 codes8(const uint64_t (&v)[4], uint64_t inv2) {
  uint32_t r[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float x, y, z, w;
    umma::f2_unpack(umma::f2_mul(v[2 * k], inv2), x, y);
    umma::f2_unpack(umma::f2_mul(v[2 * k + 1], inv2), z, w);
    if (kE4m3) {
      r[k] = to_e4m3x2(x, y) | (to_e4m3x2(z, w) << 16);
    } else {
      // rint by the addition of 1.5 2^23, whose low byte is then the code (one by one:
      // a packed addition came out in one rounding with its product)
      constexpr float kMagic = 12582912.f;
      const uint32_t a = __float_as_uint(__fadd_rn(x, kMagic)), b = __float_as_uint(__fadd_rn(y, kMagic));
      const uint32_t c = __float_as_uint(__fadd_rn(z, kMagic)), d = __float_as_uint(__fadd_rn(w, kMagic));
      r[k] = __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
    }
  }
  return make_uint2(r[0], r[1]);
}

// The rows' codes: chunk(i, half, y) gives the values of chunk `half` (0, 1) of row
// 4 i + r.  at0, at1: the chunks' places in a row.
template <bool kE4m3, typename Chunk>
__device__ __forceinline__ void put_rows(const Unit& u, float old, float s, bool finite, int at0,
                                         int at1, Chunk chunk) {
  const int r = (threadIdx.x & 31) >> 3;
  const bool started = u.token[0] >= 0;
  const float inv = s >= kScaleTiny ? __frcp_rn(s) : 0.f;
  const uint64_t inv2 = umma::f2_pack(__float_as_uint(inv), __float_as_uint(inv));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 4 * i + r;
    uint2* const at[2] = {reinterpret_cast<uint2*>(u.codes + row * kCodeRowBytes + 8 * at0),
                          reinterpret_cast<uint2*>(u.codes + row * kCodeRowBytes + 8 * at1)};
    if (u.token[row] >= 0) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint64_t v[4];
        chunk(i, k, v);
        if (finite) {
          *at[k] = codes8<kE4m3>(v, inv2);
        } else {
          float y[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            umma::f2_unpack(v[j], y[2 * j], y[2 * j + 1]);
            y[2 * j] = __fmul_rn(y[2 * j], inv);
            y[2 * j + 1] = __fmul_rn(y[2 * j + 1], inv);
          }
          *at[k] = make_uint2(codes4<kE4m3>(y[0], y[1], y[2], y[3]),
                              codes4<kE4m3>(y[4], y[5], y[6], y[7]));
        }
      }
    } else if (started) {
      *at[0] = *at[1] = make_uint2(0u, 0u);
    } else if (s != old) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint2 held = *at[k];
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          y[j] = __fmul_rn(
              __fmul_rn(code_value<kE4m3>((j < 4 ? held.x : held.y) >> (8 * (j & 3))), old), inv);
        *at[k] = make_uint2(codes4<kE4m3>(y[0], y[1], y[2], y[3]),
                            codes4<kE4m3>(y[4], y[5], y[6], y[7]));
      }
    }
  }
}

__device__ __forceinline__ void pairs_of(const uint4& w, uint64_t (&v)[4]) {
  v[0] = umma::f2_pack(w.x << 16, w.x & 0xffff0000u);
  v[1] = umma::f2_pack(w.y << 16, w.y & 0xffff0000u);
  v[2] = umma::f2_pack(w.z << 16, w.z & 0xffff0000u);
  v[3] = umma::f2_pack(w.w << 16, w.w & 0xffff0000u);
}

// Rows as they come.  The maximum is taken on the bf16 bits: without the sign they
// order as the values do, infinities and NaN above all others.
template <bool kE4m3>
__device__ __forceinline__ void put_unit(const Unit& u) {
  constexpr float kMax = kE4m3 ? kE4m3Max : kInt8Max;
  const int lane = threadIdx.x & 31, l = lane & 7, r = lane >> 3;
  const float old = scale_before(u);
  uint4 raw[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = u.token[4 * i + r];
    const uint16_t* src = u.src + t * u.stride + l * 8;
    raw[i][0] = t >= 0 ? ld_global_nc_v4(src) : make_uint4(0u, 0u, 0u, 0u);
    raw[i][1] = t >= 0 ? ld_global_nc_v4(src + 64) : make_uint4(0u, 0u, 0u, 0u);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint4& w = raw[i >> 1][i & 1];
    m = __vmaxu2(__vmaxu2(m, w.x & 0x7fff7fffu), w.y & 0x7fff7fffu);
    m = __vmaxu2(__vmaxu2(m, w.z & 0x7fff7fffu), w.w & 0x7fff7fffu);
  }
  uint32_t top = __reduce_max_sync(kFull, max(m << 16, m & 0xffff0000u));
  const bool finite = top < 0x7f800000u;
  if (!finite) {
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4& w = raw[i >> 1][i & 1];
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = (x[j] << 16) & 0x7fffffffu, b = x[j] & 0x7fff0000u;
        top = max(top, a < 0x7f800000u ? a : 0u);
        top = max(top, b < 0x7f800000u ? b : 0u);
      }
    }
    top = __reduce_max_sync(kFull, top);
  }
  const float s = fmaxf(old, __fmul_rn(__uint_as_float(top), 1.f / kMax));
  put_rows<kE4m3>(u, old, s, finite, l, l + 8,
                  [&](int i, int k, uint64_t (&v)[4]) { pairs_of(raw[i][k], v); });
  if (lane == 0) *u.scale = s;
}

// The largest of three sizes, NaN if one is.
__device__ __forceinline__ float larger_size(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Keys, turned; cs: the sines of the 16 rows.  kKind as for rope_rows: interleaved, half
// with partners in whole chunks (which a lane holds both), half with others (read one
// by one).
template <bool kE4m3, int kKind>
__device__ __forceinline__ void put_turned(const Unit& u, const float2 (*cs)[cs_at(64)],
                                           int rotary_dim) {
  constexpr float kMax = kE4m3 ? kE4m3Max : kInt8Max;
  const int lane = threadIdx.x & 31, l = lane & 7, r = lane >> 3;
  const int half = rotary_dim >> 1;
  int ca = 2 * l, cb = 2 * l + 1;
  if (kKind == 1 && l < (rotary_dim >> 4)) {
    ca = l;
    cb = l + (rotary_dim >> 4);
  }
  const float old = scale_before(u);
  uint4 raw[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = u.token[4 * i + r];
    const uint16_t* src = u.src + t * u.stride;
    raw[i][0] = t >= 0 ? ld_global_nc_v4(src + 8 * ca) : make_uint4(0u, 0u, 0u, 0u);
    raw[i][1] = t >= 0 ? ld_global_nc_v4(src + 8 * cb) : make_uint4(0u, 0u, 0u, 0u);
  }
  float x[4][16];
  float size = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = u.token[4 * i + r];
    const float2* f = cs[4 * i + r];
    const uint32_t w[8] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w,
                           raw[i][1].x, raw[i][1].y, raw[i][1].z, raw[i][1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[i][2 * j] = bf16_lo(w[j]);
      x[i][2 * j + 1] = bf16_hi(w[j]);
    }
    if (t >= 0) {
      if (kKind == 2) {
        const uint16_t* src = u.src + t * u.stride;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int e = 16 * l + j;
          if (e >= rotary_dim) continue;
          const bool lower = e < half;
          const int other = lower ? e + half : e - half;
          const float y = bf16_lo(src[other]);
          const float2 c = f[cs_at(lower ? e : other)];
          x[i][j] = turned_one(x[i][j], lower ? -y : y, c);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float4 c = *reinterpret_cast<const float4*>(&f[cs_at(8 * l) + j]);
          const float2 c0 = make_float2(c.x, c.y), c1 = make_float2(c.z, c.w);
          if (kKind == 0) {
            if (8 * l + j < half) turn_pair(x[i][2 * j], x[i][2 * j + 1], c0);
            if (8 * l + j + 1 < half) turn_pair(x[i][2 * j + 2], x[i][2 * j + 3], c1);
          } else if (8 * l < half) {
            turn_pair(x[i][j], x[i][8 + j], c0);
            turn_pair(x[i][j + 1], x[i][8 + j + 1], c1);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 16; j += 2) size = larger_size(size, x[i][j], x[i][j + 1]);
  }
  // (as bits they order as the values do, infinities and NaN above all others)
  uint32_t top = __reduce_max_sync(kFull, __float_as_uint(size));
  const bool finite = top < 0x7f800000u;
  if (!finite) {
    top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const uint32_t a = __float_as_uint(x[i][j]) & 0x7fffffffu;
        top = max(top, a < 0x7f800000u ? a : 0u);
      }
    top = __reduce_max_sync(kFull, top);
  }
  const float s = fmaxf(old, __fmul_rn(__uint_as_float(top), 1.f / kMax));
  put_rows<kE4m3>(u, old, s, finite, ca, cb, [&](int i, int k, uint64_t (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = umma::f2_pack(__float_as_uint(x[i][8 * k + 2 * j]),
                           __float_as_uint(x[i][8 * k + 2 * j + 1]));
  });
  if (lane == 0) *u.scale = s;
}

// What a CTA has in shared memory.
template <int kKind>
struct KvSmem {
  alignas(16) float2 cs[kKind >= 0 ? kBatch * kGroupRows : 1][cs_at(64)];
  GroupTable g;
};

// kKind: -1 without rotary positions, else rope_rows'.  table: hash slots, a power of
// two, at least 2 tile.
template <bool kE4m3, int kKind>
__global__ void __launch_bounds__(threads_of(kKind), 1)
    append_q8_kernel(const __grid_constant__ AppendQ8Params p, int tile, int table, int kv_ctas,
                     int per_token) {
  constexpr bool kRope = kKind >= 0;
  constexpr int kRowsKind = kRope ? kKind : 0;
  constexpr int kThreads = threads_of(kKind), kWarps = kThreads / 32;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  grid_dependency_trigger();
  grid_dependency_wait();
  const int tid = threadIdx.x;
  if constexpr (kRope) {
    if (static_cast<int>(blockIdx.x) >= kv_ctas) {
      const int part = tid / kRopeThreads;
      const int b = (static_cast<int>(blockIdx.x) - kv_ctas) * (kThreads / kRopeThreads) + part;
      rope_rows<kRowsKind, 1>(p.queries, reinterpret_cast<RopeSmem<kRowsKind, 1>*>(smem_raw)[part],
                              tid % kRopeThreads, b / per_token, b % per_token, per_token);
      return;
    }
  }
  KvSmem<kKind>& smem = *reinterpret_cast<KvSmem<kKind>*>(smem_raw);
  GroupTable& g = smem.g;
  const int mask = table - 1;
  const int t0 = blockIdx.x * tile;
  const int t1 = min(t0 + tile, p.num_tokens);
  for (int i = tid; i < table * kGroupRows / 4; i += kThreads)
    reinterpret_cast<int4*>(g.token)[i] = make_int4(-1, -1, -1, -1);
  for (int i = tid; i < table; i += kThreads) {
    g.key[i] = 0ull;
    g.first[i] = 0x7fffffff;
  }
  for (int i = tid; i < kFilter / 32; i += kThreads) g.filter[i] = 0u;
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
    const uint32_t bit = filter_bit(slot);
    atomicOr(&g.filter[bit >> 5], 1u << (bit & 31));
    int at = hash_of(key, mask);
    while (true) {  // at most half of the slots are taken
      const unsigned long long was = atomicCAS(&g.key[at], 0ull, key);
      if (was == 0ull || was == key) break;
      at = (at + 1) & mask;
    }
  }
  __syncthreads();
  for (int base = tid; base < p.num_tokens; base += kScan * kThreads) {
    int64_t slot[kScan];
    uint32_t hits = 0;
#pragma unroll
    for (int j = 0; j < kScan; ++j) {
      const int t = base + j * kThreads;
      slot[j] = t < p.num_tokens ? __ldg(p.slot_mapping + t) : -1;
    }
#pragma unroll
    for (int j = 0; j < kScan; ++j) {
      const uint32_t bit = filter_bit(slot[j]);
      hits |= (g.filter[bit >> 5] >> (bit & 31) & 1u) << j;
    }
    if (hits == 0u) continue;
#pragma unroll
    for (int j = 0; j < kScan; ++j) {
      if (!(hits >> j & 1u)) continue;
      const unsigned long long key = key_of(slot[j]);
      if (key == 0ull) continue;
      int at = hash_of(key, mask);
      unsigned long long have;
      while ((have = g.key[at]) != key && have != 0ull) at = (at + 1) & mask;
      if (have == key) {
        atomicMin(&g.first[at], base + j * kThreads);
        atomicMax(&g.token[at][slot[j] % kGroupRows], base + j * kThreads);
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < table; i += kThreads)
    if (g.key[i] != 0ull && g.first[i] >= t0) g.owned[atomicAdd(&g.num_owned, 1)] = i;
  __syncthreads();
  const int n = g.num_owned;
  const int warp = tid >> 5;
  // unit u of groups b0 .. b0 + nb - 1 of the CTA's: K's heads first (turning takes longer)
  auto put = [&](int b0, int nb, int u) {
    const bool is_v = u >= nb * p.Hkv;
    if (is_v) u -= nb * p.Hkv;
    const int b = static_cast<uint32_t>(u) / static_cast<uint32_t>(p.Hkv), h = u - b * p.Hkv;
    const int at = g.owned[b0 + b];
    const int64_t group = static_cast<int64_t>(g.key[at] - 1ull);
    if (!kRope || is_v)
      put_unit<kE4m3>(unit_at(p, g.token[at], group, h, is_v));
    else
      put_turned<kE4m3, kRowsKind>(unit_at(p, g.token[at], group, h, false),
                                   &smem.cs[b * kGroupRows], p.queries.rope.rotary_dim);
  };
  if constexpr (!kRope) {
    for (int u = warp; u < n * 2 * p.Hkv; u += kWarps) put(0, n, u);
  } else {
    for (int b0 = 0; b0 < n; b0 += kBatch) {
      const int nb = min(kBatch, n - b0);
      for (int e = tid; e < nb * kGroupRows * 64; e += kThreads) {
        const int row = e >> 6;
        const int t = g.token[g.owned[b0 + row / kGroupRows]][row % kGroupRows];
        if (t >= 0)
          smem.cs[row][cs_at(e & 63)] = rope_sines(p.queries.rope, p.queries.positions[t], e & 63);
      }
      __syncthreads();
      for (int u = warp; u < nb * 2 * p.Hkv; u += kWarps) put(b0, nb, u);
      __syncthreads();
    }
  }
}

template <bool kE4m3, int kKind>
cudaError_t launch(const AppendQ8Params& p, cudaStream_t stream) {
  // one CTA an SM, or several rounds of them (what they cost: above)
  const int64_t most = static_cast<int64_t>(p.sms) * kMaxTile;
  const int64_t ctas = p.sms * ((p.num_tokens + most - 1) / most);
  const int tile = static_cast<int>((p.num_tokens + ctas - 1) / ctas);
  const int kv = (p.num_tokens + tile - 1) / tile;
  int table = kMinTable;
  while (table < 2 * tile) table *= 2;
  constexpr size_t kRow = sizeof(GroupTable::token[0]);
  constexpr size_t kSmem = sizeof(KvSmem<kKind>), kRest = kSmem - kMaxTable * kRow;
  static_assert(kKind < 0 || sizeof(RopeSmem<kKind < 0 ? 0 : kKind, 1>) *
                                     (threads_of(kKind) / kRopeThreads) <= kRest, "queries fit too");
  static unsigned long long done_mask = 0;
  auto kernel = append_q8_kernel<kE4m3, kKind>;
  const cudaError_t se = ensure_smem_limit(kernel, static_cast<int>(kSmem), &done_mask);
  if (se != cudaSuccess) return se;
  int queries = 0, per_token = 0;
  if (kKind >= 0) {
    if (p.num_tokens <= kTogether) {
      per_token = (p.queries.Hq + kRowsPerPass - 1) / kRowsPerPass;
      constexpr int kParts = threads_of(kKind) / kRopeThreads;
      queries = (p.num_tokens * per_token + kParts - 1) / kParts;
    } else {
      const cudaError_t e = launch_rope_append(p.queries, stream);
      if (e != cudaSuccess) return e;
    }
  }
  return launch_pdl(kernel, dim3(static_cast<unsigned>(kv + queries)), dim3(threads_of(kKind)),
                    kRest + table * kRow, stream, p, tile, table, kv, per_token);
}

template <bool kE4m3>
cudaError_t launch_kind(const AppendQ8Params& p, bool rope, cudaStream_t stream) {
  if (!rope) return launch<kE4m3, -1>(p, stream);
  if (p.queries.rope.interleaved) return launch<kE4m3, 0>(p, stream);
  return p.queries.rope.rotary_dim % 16 == 0 ? launch<kE4m3, 1>(p, stream)
                                             : launch<kE4m3, 2>(p, stream);
}

}  // namespace

cudaError_t launch_append_q8(const AppendQ8Params& p, bool e4m3, bool rope, cudaStream_t stream) {
  if (p.num_tokens <= 0) return cudaSuccess;
  return e4m3 ? launch_kind<true>(p, rope, stream) : launch_kind<false>(p, rope, stream);
}

}  // namespace pkv
