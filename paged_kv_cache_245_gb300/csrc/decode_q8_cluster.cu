// decode_q8_cluster.cu -- decode attention over the 8-bit KV cache for small
// batches: each (sequence, KV head) is one thread-block cluster, whose warps take
// its 16-token tiles in turn and join their parts through distributed shared
// memory, in one launch.  sm_103a.
//
// What counts here is the chain of dependent reads.  Warp w takes tiles w, w + N,
// ... (N warps in the cluster), so which tiles are its own does not depend on the
// context, and a tile's table entry is read beside the context and the queries;
// then come K, V and the scales, straight into the registers that the products
// take them from (no shared memory, no barrier); then two joins.  A tile costs a
// warp about 1 us (its loads wait for one another more than its products do; two
// or three more tiles in flight, or two tiles a step, did not change that), so the
// host takes this kernel only where a warp has few tiles.  8 KV heads, us a call,
// this kernel / decode_q8.cu: 1 sequence of 1000 5.2 / 14.7, of 8000 11.2 / 17.8, 4
// of 1000 5.8 / 11.3, 8 of 512 5.6 / 10.3, 16 of 512 6.2 / 11.2, 8 of 2000 10.8 /
// 14.0.
//
// Math of a tile: as in decode_q8.cu.  A lane's part of K is 32 elements of rows
// g and g + 8; of V, 16 elements (16 g ..) of keys 2 tq, 2 tq + 1, 2 tq + 8 and 2 tq
// + 9, so that rows g and g + 8 of product i stand for elements 16 g + 2 i and + 1.
#include "cluster.cuh"
#include "decode_launch.cuh"
#include "q8.cuh"
#include "q8_math.cuh"
#include "umma.cuh"

namespace pkv {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRec = 132;  // o[128], m, l, pad

struct Tile {
  uint4 k[4];  // row g: chunks 2 tq, 2 tq + 1; row g + 8
  uint4 v[4];  // keys 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9: chunk g
  float ks, vs;
};

template <bool kE4m3, int kWarps>
__global__ void __launch_bounds__(kWarps * 32, kWarps == 8 ? 1 : kQ8SmallCtas)
    decode_q8_cluster_kernel(const __grid_constant__ AttentionQ8Params p, int cluster) {
  __shared__ __align__(16) float part[kWarps][8][kRec];  // each warp's heads
  __shared__ __align__(16) float joined[8][kRec];        // the CTA's
  constexpr int kJoinHeads = 8 / kWarps;                 // heads that a warp joins
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, tq = lane & 3;
  const int seq = blockIdx.z, kvh = blockIdx.y, G = p.G;
  const int rank = blockIdx.x;
  const int N = cluster * kWarps;

  grid_dependency_wait();
  grid_dependency_trigger();

  // ---- context, first table entry and queries, side by side
  const uint32_t bs = static_cast<uint32_t>(p.bs);
  const int32_t* table = p.tables + static_cast<int64_t>(seq) * p.max_blocks;
  auto entry_of = [&](int tile) -> int32_t {
    const uint32_t at = static_cast<uint32_t>(tile) * 16 / bs;
    return at < static_cast<uint32_t>(p.max_blocks) ? __ldg(table + at) : 0;
  };
  int tile = rank * kWarps + warp;
  const int32_t entry = entry_of(tile);
  int32_t next_entry = entry_of(tile + N);
  int ctx = max(__ldg(p.ctx_lens + seq), 0);
  uint4 qn[4];
  {
    const uint4* row = reinterpret_cast<const uint4*>(
        p.q + (static_cast<int64_t>(seq) * p.Hq + kvh * G + (g < G ? g : 0)) * kHeadDim + 32 * tq);
#pragma unroll
    for (int k = 0; k < 4; ++k) qn[k] = g < G ? __ldg(row + k) : make_uint4(0u, 0u, 0u, 0u);
  }
  if (p.checked && ctx > p.max_context) {
    if (threadIdx.x == 0 && rank == 0) record_error(p.err, kErrContext);
    ctx = p.max_context;
  }
  const int ntiles = (ctx + 15) >> 4;

  auto fetch = [&](int n, int32_t e, Tile& t) {
    if (p.checked && (e < 0 || e >= p.num_blocks)) {
      if (lane == 0) record_error(p.err, p.err_code);
#pragma unroll
      for (int i = 0; i < 4; ++i) t.k[i] = t.v[i] = make_uint4(0u, 0u, 0u, 0u);
      t.ks = t.vs = 0.f;
      return;
    }
    const int64_t row = cache_row(e, kvh, p.Hkv, bs, static_cast<uint32_t>(n) * 16 % bs);
    const uint8_t* k = p.k_codes + (row + g) * kCodeRowBytes + 32 * tq;
    const uint8_t* v = p.v_codes + (row + 2 * tq) * kCodeRowBytes + 16 * g;
    t.k[0] = ld_global_nc_v4(k);
    t.k[1] = ld_global_nc_v4(k + 16);
    t.k[2] = ld_global_nc_v4(k + 8 * kCodeRowBytes);
    t.k[3] = ld_global_nc_v4(k + 8 * kCodeRowBytes + 16);
    t.ks = __ldg(p.k_scale + row / kGroupRows);
    t.v[0] = ld_global_nc_v4(v);
    t.v[1] = ld_global_nc_v4(v + kCodeRowBytes);
    t.v[2] = ld_global_nc_v4(v + 8 * kCodeRowBytes);
    t.v[3] = ld_global_nc_v4(v + 9 * kCodeRowBytes);
    t.vs = __ldg(p.v_scale + row / kGroupRows);
  };

  // O^T of elements 16 g + 2 i (0) and + 1 (1): heads 2 tq and 2 tq + 1 as a pair
  uint64_t acc[8][2];
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = 0ull;
  Tile next;
  if (tile < ntiles) fetch(tile, entry, next);
  uint32_t qb[8][2];
  const float down = queries_to_half(qn, qb);
  // score units of heads 2 tq and 2 tq + 1
  const float qs0 = __shfl_sync(kFull, down, 8 * tq) * p.qscale;
  const float qs1 = __shfl_sync(kFull, down, 8 * tq + 4) * p.qscale;

  for (; tile < ntiles; tile += N) {
    Tile t = next;
    if (tile + N < ntiles) {
      fetch(tile + N, next_entry, next);
      next_entry = entry_of(tile + 2 * N);
    }
    const int nvalid = ctx - tile * 16;
    if (kE4m3 && nvalid < 16) {  // rows past the context may hold NaN: 0 * NaN
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (2 * tq + (i & 1) + 8 * (i >> 1) >= nvalid) t.v[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    // ---- S^T = K . Q^T: keys g and g + 8, heads 2tq and 2tq + 1
    float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint32_t w0[4] = {t.k[half].x, t.k[half].y, t.k[half].z, t.k[half].w};
      const uint32_t w1[4] = {t.k[2 + half].x, t.k[2 + half].y, t.k[2 + half].z, t.k[2 + half].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t a[4];
        halves_of<kE4m3>(w0[e], a[0], a[2]);
        halves_of<kE4m3>(w1[e], a[1], a[3]);
        const int ks = 4 * half + e;
        if (ks & 1) mma_f16_16816(sb, a, qb[ks][0], qb[ks][1]);
        else mma_f16_16816(sa, a, qb[ks][0], qb[ks][1]);
      }
    }
    const float f0 = qs0 * t.ks, f1 = qs1 * t.ks;
    const bool v0 = g < nvalid, v1 = g + 8 < nvalid;
    const float s0 = v0 ? (sa[0] + sb[0]) * f0 : -INFINITY;
    const float s1 = v0 ? (sa[1] + sb[1]) * f1 : -INFINITY;
    const float s2 = v1 ? (sa[2] + sb[2]) * f0 : -INFINITY;
    const float s3 = v1 ? (sa[3] + sb[3]) * f1 : -INFINITY;
    float mx0 = fmaxf(m0, fmaxf(s0, s2)), mx1 = fmaxf(m1, fmaxf(s1, s3));
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, o));
      mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, o));
    }
    if (mx0 > m0 || mx1 > m1) {
      const float a0 = mx0 > m0 ? fast_exp2(m0 - mx0) : 1.f;
      const float a1 = mx1 > m1 ? fast_exp2(m1 - mx1) : 1.f;
      const uint64_t a2 = umma::f2_pack(__float_as_uint(a0), __float_as_uint(a1));
      l0 *= a0;
      l1 *= a1;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[i][0] = umma::f2_mul(acc[i][0], a2);
        acc[i][1] = umma::f2_mul(acc[i][1], a2);
      }
      m0 = mx0;
      m1 = mx1;
    }
    const float p0 = fast_exp2(s0 - m0), p2 = fast_exp2(s2 - m0);
    const float p1 = fast_exp2(s1 - m1), p3 = fast_exp2(s3 - m1);
    l0 += p0 + p2;
    l1 += p1 + p3;
    // P^T as the B operand, rounded to fp16 once
    const uint32_t b0 = movmatrix_trans(probabilities_to_half2(p0, p1));  // keys 0..7
    const uint32_t b1 = movmatrix_trans(probabilities_to_half2(p2, p3));  // keys 8..15

    // ---- O^T += vs (V^T . P^T)
    const float vs = t.vs * kPDown;
    const uint64_t vs2 = umma::f2_pack(__float_as_uint(vs), __float_as_uint(vs));
    const uint32_t* k0 = &t.v[0].x;
    const uint32_t* k1 = &t.v[1].x;
    const uint32_t* k8 = &t.v[2].x;
    const uint32_t* k9 = &t.v[3].x;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // elements 2 i and 2 i + 1 of both keys of a pair
      const unsigned pick = i & 1 ? 0x7632u : 0x5410u;
      uint32_t a[4];
      halves_across<kE4m3>(__byte_perm(k0[i >> 1], k1[i >> 1], pick), a[0], a[1]);
      halves_across<kE4m3>(__byte_perm(k8[i >> 1], k9[i >> 1], pick), a[2], a[3]);
      float d[4];
      mma_f16_16816_zero(d, a, b0, b1);
      acc[i][0] = umma::f2_fma(umma::f2_pack(__float_as_uint(d[0]), __float_as_uint(d[1])), vs2,
                               acc[i][0]);
      acc[i][1] = umma::f2_fma(umma::f2_pack(__float_as_uint(d[2]), __float_as_uint(d[3])), vs2,
                               acc[i][1]);
    }
  }

  // ---- the warps' parts, joined head by head
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    l0 += __shfl_xor_sync(kFull, l0, o);
    l1 += __shfl_xor_sync(kFull, l1, o);
  }
  {
    float e0[16], e1[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      umma::f2_unpack(acc[i][0], e0[2 * i], e1[2 * i]);
      umma::f2_unpack(acc[i][1], e0[2 * i + 1], e1[2 * i + 1]);
    }
    float* r0 = part[warp][2 * tq];
    float* r1 = part[warp][2 * tq + 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (2 * tq < G)
        *reinterpret_cast<float4*>(r0 + 16 * g + 4 * i) =
            make_float4(e0[4 * i], e0[4 * i + 1], e0[4 * i + 2], e0[4 * i + 3]);
      if (2 * tq + 1 < G)
        *reinterpret_cast<float4*>(r1 + 16 * g + 4 * i) =
            make_float4(e1[4 * i], e1[4 * i + 1], e1[4 * i + 2], e1[4 * i + 3]);
    }
    if (g == 0) {
      r0[128] = m0;
      r0[129] = l0;
      r1[128] = m1;
      r1[129] = l1;
    }
  }
  __syncthreads();
  // (o, m, l) of n records, as one: weights 2^(m_k - M) for the lanes k < n
  auto weights = [&](float mk, float lk, float& M, float& L) -> float {
    M = mk;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    const float f = lk == 0.f ? 0.f : fast_exp2(mk - M);
    L = lk * f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) L += __shfl_xor_sync(kFull, L, o);
    return f;
  };
  auto write_out = [&](int h, float4 o4, float L) {
    const float inv = L != 0.f ? 1.f / L : 0.f;
    *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(seq) * p.Hq + kvh * G + h) * kHeadDim +
                              lane * 4) =
        make_uint2(pack_bf16x2(o4.x * inv, o4.y * inv), pack_bf16x2(o4.z * inv, o4.w * inv));
  };
  auto add = [](float4& o4, float x, const float4& v) {
    o4.x = fmaf(x, v.x, o4.x);
    o4.y = fmaf(x, v.y, o4.y);
    o4.z = fmaf(x, v.z, o4.z);
    o4.w = fmaf(x, v.w, o4.w);
  };
  const int k = lane & 15;
#pragma unroll
  for (int j = 0; j < kJoinHeads; ++j) {
    const int h = warp + j * kWarps;
    if (h >= G) break;
    float M, L;
    const float f = weights(k < kWarps ? part[k][h][128] : -INFINITY,
                            k < kWarps ? part[k][h][129] : 0.f, M, L);
    float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      add(o4, __shfl_sync(kFull, f, w), *reinterpret_cast<const float4*>(&part[w][h][lane * 4]));
    if (cluster == 1) {
      write_out(h, o4, L);
    } else {
      *reinterpret_cast<float4*>(&joined[h][lane * 4]) = o4;
      if (lane == 0) {
        joined[h][128] = M;
        joined[h][129] = L;
      }
    }
  }
  if (cluster == 1) return;
  // then the CTAs': CTA 0 reads the others'
  cluster_sync();
  if (rank == 0) {
#pragma unroll
    for (int j = 0; j < kJoinHeads; ++j) {
      const int h = warp + j * kWarps;
      if (h >= G) break;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (k < cluster) ml = ld_cluster_f2(in_cta(&joined[h][128], k));
      float M, L;
      const float f = weights(ml.x, ml.y, M, L);
      float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int c = 0; c < cluster; ++c)
        add(o4, __shfl_sync(kFull, f, c), ld_cluster_f4(in_cta(&joined[h][lane * 4], c)));
      write_out(h, o4, L);
    }
  }
  cluster_sync();  // no CTA leaves while its memory is read
}

template <bool kE4m3, int kWarps>
cudaError_t launch(const AttentionQ8Params& p, int cluster, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster, p.Hkv, p.num_seqs);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_decode_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, decode_q8_cluster_kernel<kE4m3, kWarps>, p, cluster);
}

template <bool kE4m3, int kWarps>
cudaError_t room(ClusterRoom* out) {
  static unsigned long long asked = 0;
  static ClusterRoom rooms[64];
  return cluster_room(decode_q8_cluster_kernel<kE4m3, kWarps>, kWarps * 32, 0, rooms, &asked, out);
}

}  // namespace

cudaError_t room_decode_q8_cluster(bool e4m3, ClusterRoom* out) {
  return e4m3 ? room<true, 8>(out) : room<false, 8>(out);
}

cudaError_t launch_decode_q8_cluster(const AttentionQ8Params& p, bool e4m3, int cluster, int warps,
                                     cudaStream_t stream) {
  if (warps == 4)
    return e4m3 ? launch<true, 4>(p, cluster, stream) : launch<false, 4>(p, cluster, stream);
  return e4m3 ? launch<true, 8>(p, cluster, stream) : launch<false, 8>(p, cluster, stream);
}

}  // namespace pkv
