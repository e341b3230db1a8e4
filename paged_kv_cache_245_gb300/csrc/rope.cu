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
#include "rope.cuh"

#include "pkv_device.cuh"

namespace pkv {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRowsPerPass = kRopeThreads / 8;

// The turned pair (x, y) as bf16: the only rounding on the way.
__device__ __forceinline__ float2 turned(float x, float y, float2 cs) {
  return make_float2(x * cs.x - y * cs.y, y * cs.x + x * cs.y);
}

// Plain (coherent) load: the output may be the query tensor itself.
__device__ __forceinline__ uint4 ld_row16(const uint16_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}

// Eight pairs, then 16 bytes of padding: lanes that read 8 pairs apart meet
// different banks.
__device__ __forceinline__ constexpr int cs_at(int pair) { return pair + (pair >> 3) * 2; }

// A row's two chunks of this lane, its token of the CTA and its row of R.
struct RopeRow {
  uint4 a, b;
  int tok, h;
};

// kKind 0: interleaved pairs (2i, 2i + 1); 1: half layout, rotary_dim a
// multiple of 16 (whole chunks are partners); 2: half layout, any even
// rotary_dim (partners from shared memory, one by one).
template <int kKind, int kTokens>
__global__ void __launch_bounds__(kRopeThreads, 5) rope_append_kernel(const RopeParams p) {
  // (cos, sin) times gain of the rotated pairs; pair i at cs_at(i)
  __shared__ __align__(16) float2 cs[kTokens][cs_at(64)];
  __shared__ uint32_t rows[kKind == 2 ? kRowsPerPass : 1][66];  // a row of every 8 lanes
  __shared__ int64_t row0[kTokens];    // cache row of KV head 0, or -1: k and v go nowhere
  grid_dependency_trigger();
  grid_dependency_wait();
  const int tid = threadIdx.x;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kTokens;
  const int ntok = static_cast<int>(min(static_cast<int64_t>(kTokens), p.num_tokens - t0));
  const int rd = p.rope.rotary_dim;
  const int half = rd >> 1;

  const int l = tid & 7;
  const int R = p.Hq + 2 * p.Hkv;
  const int nrows = ntok * R;
  // the two chunks of this lane: rotated rows, and copied ones (v)
  int ca = 2 * l, cb = 2 * l + 1;
  if (kKind == 1) {
    const int parts = rd >> 4;  // partner pairs of chunks
    ca = l < parts ? l : 2 * l;  // past the rotated part: chunks 2 parts + 2 (l - parts), + 1
    cb = l < parts ? l + parts : 2 * l + 1;
  }
  if (kKind == 2) {
    ca = l;  // (fewer bank conflicts than neighbours)
    cb = l + 8;
  }
  auto fetch = [&](int r) -> RopeRow {
    RopeRow row;
    row.tok = kTokens == 1 ? 0 : r / R;
    row.h = r - row.tok * R;
    const int64_t t = t0 + row.tok;
    const int hk = row.h - p.Hq;
    const uint16_t* src = hk < 0 ? p.q + t * p.q_stride + row.h * kHeadDim
                        : hk < p.Hkv ? p.k + t * p.k_stride + hk * kHeadDim
                                     : p.v + t * p.v_stride + (hk - p.Hkv) * kHeadDim;
    row.a = ld_row16(src + ca * 8);
    row.b = ld_row16(src + cb * 8);
    return row;
  };
  // a row is in flight while the one before it is turned; the first while the
  // sines are computed
  const int step = gridDim.y * kRowsPerPass;
  int r = blockIdx.y * kRowsPerPass + (tid >> 3);
  RopeRow cur;
  if (r < nrows) cur = fetch(r);

  for (int e = tid; e < kTokens * 64; e += kRopeThreads) {
    const int tok = e >> 6, i = e & 63;
    float2 c = make_float2(1.f, 0.f);
    if (tok < ntok && i < half) {
      const int64_t pos = p.positions[t0 + tok];
      const int64_t turn = static_cast<int64_t>(static_cast<uint64_t>(pos) * p.rope.turn[i]);
      // a signed fraction of a turn in units of 2^-64 is 2^-63 half turns
      sincospif(static_cast<float>(turn) * 1.0842021724855044e-19f, &c.y, &c.x);
      c.x *= p.rope.gain;
      c.y *= p.rope.gain;
    }
    cs[tok][cs_at(i)] = c;
  }
  if (tid < ntok) {
    const int64_t slot = p.slot_mapping[t0 + tid];
    int64_t r = -1;
    if (slot >= 0) {
      if (p.checked && slot >= p.num_slots) {
        if (blockIdx.y == 0) record_error(p.err, kErrSlot);
      } else {
        r = cache_row(slot / p.bs, 0, p.Hkv, p.bs, slot % p.bs);
      }
    }
    row0[tid] = r;
  }
  __syncthreads();

  for (; r < nrows; r += step) {
    const RopeRow row = cur;
    const int tok = row.tok;
    if (r + step < nrows) cur = fetch(r + step);
    const int h = row.h;
    const int64_t t = t0 + tok;
    uint16_t* dst;
    bool move = true;
    if (h < p.Hq) {
      dst = p.q_out + (t * p.Hq + h) * kHeadDim;
    } else {
      const bool is_v = h >= p.Hq + p.Hkv;
      const int64_t kv_row = row0[tok];
      dst = (is_v ? p.v_cache : p.k_cache) +
            (kv_row + (h - p.Hq - (is_v ? p.Hkv : 0)) * p.bs) * kHeadDim;
      move = kv_row >= 0;
    }
    uint32_t wa[4] = {row.a.x, row.a.y, row.a.z, row.a.w};
    uint32_t wb[4] = {row.b.x, row.b.y, row.b.z, row.b.w};
    if (h < p.Hq + p.Hkv) {
      if (kKind == 0) {  // a 32-bit word is a pair
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t& w = i < 4 ? wa[i] : wb[i - 4];
          const int pair = (i < 4 ? ca : cb) * 4 + (i & 3);
          if (pair < half) {
            const float2 f = turned(bf16_lo(w), bf16_hi(w), cs[tok][cs_at(pair)]);
            w = pack_bf16x2(f.x, f.y);
          }
        }
      } else if (kKind == 1) {
        if (l < (rd >> 4)) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(&cs[tok][cs_at(l * 8) + 2 * i]);
            const float2 r0 = turned(bf16_lo(wa[i]), bf16_lo(wb[i]), make_float2(f.x, f.y));
            const float2 r1 = turned(bf16_hi(wa[i]), bf16_hi(wb[i]), make_float2(f.z, f.w));
            wa[i] = pack_bf16x2(r0.x, r1.x);
            wb[i] = pack_bf16x2(r0.y, r1.y);
          }
        }
      } else {  // rotary_dim is even: a word is turned whole or not at all
        const unsigned lanes = 0xffu << (tid & 24);  // the row's own
        uint32_t* stage = rows[tid >> 3];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          stage[ca * 4 + i] = wa[i];
          stage[cb * 4 + i] = wb[i];
        }
        __syncwarp(lanes);
        const uint16_t* elems = reinterpret_cast<const uint16_t*>(stage);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t& w = i < 4 ? wa[i] : wb[i - 4];
          const int at = (i < 4 ? ca : cb) * 8 + 2 * (i & 3);
          if (at >= rd) continue;
          float o[2];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const float x = b == 0 ? bf16_lo(w) : bf16_hi(w);
            const bool lower = at + b < half;
            const int other = lower ? at + b + half : at + b - half;
            const float y = bf16_lo(elems[other]);
            const float2 f = cs[tok][cs_at(lower ? at + b : other)];
            o[b] = lower ? turned(x, y, f).x : turned(y, x, f).y;
          }
          w = pack_bf16x2(o[0], o[1]);
        }
        __syncwarp(lanes);  // read before the next row comes in
      }
    }
    if (move) {
      *reinterpret_cast<uint4*>(dst + ca * 8) = make_uint4(wa[0], wa[1], wa[2], wa[3]);
      *reinterpret_cast<uint4*>(dst + cb * 8) = make_uint4(wb[0], wb[1], wb[2], wb[3]);
    }
  }
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
