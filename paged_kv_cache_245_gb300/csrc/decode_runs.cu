// decode_runs.cu -- decode attention with capped, biased and masked scores
// (score.cuh) over a paged (block size a multiple of 16) or contiguous KV
// cache, for batches of short visible spans: warp-level tensor-core math on
// 16-token tiles and a persistent schedule balanced over every warp of the GPU.
// sm_103a.
//
// For sequence i, query head h, KV head h / G and the positions lo .. ctx - 1
// its newest token sees: out[i][h] = sum_j softmax_j(score(q . K_j)) V_j.
// Tiles before the one that holds lo do not exist here, so a window's or a
// document's cost is its own.
//
// Schedule.  The work is the flattened list of tiles of every (sequence, KV
// head) pair, pair p = seq * Hkv + kvh in order, cut evenly over the warps of
// the grid (one CTA per SM; tc_unit_to_tile, a pair counting as seg_cost
// tiles more): each warp takes a contiguous run.  A pair that lies whole in a
// warp's run is written by that warp.  A run's first and last tiles may be
// pieces of a pair that other warps share: a piece's (o, m, l) goes to shared
// memory, and the CTA joins them once, after its warps' runs.  A pair that is
// cut by CTAs is joined by the last of them, through tagged records (decode_tc.cuh).
// The kernel of long spans (decode_tc.cuh) deals a CTA's tiles round-robin to
// its warps, which all meet at the end of every pair, so a pair of a few tiles
// costs it 3 to 4 us; here it costs one warp its own tiles.  Both are bound by
// HBM in between: 64 ragged sequences up to 8192 under a window of 1024, 32 / 8
// heads (115 MB, 17.0 us at the rate of a copy) take 25.6 us, of which 2 go by
// before the runs are known, 2 more until the first tiles are asked for, and 2.6
// at the end for the joins.  256 sequences of 128: 30.2 us; by pairs 62.
//
// Data movement and the math of a tile are that kernel's: TMA boxes into
// a per-warp ring, S^T = K Q^T and O^T += V^T P^T by mma.m16n8k16, an online
// softmax in base 2 on the accumulator fragment.
#include "decode_tc.cuh"

namespace pkv {

namespace {

// W warps, S stages each; MH query heads of a KV head (4, or 8).
template <int W, int S, int MH>
struct RunsSmem {
  static constexpr int kPieceFloats = MH * kRecStride;  // o[128], m, l of each head
  static constexpr int kStagesOff = 0;                  // (a run's last piece goes over its stages)
  static constexpr int kBarsOff = W * S * kTcStageBytes;
  static constexpr int kFirstOff = kBarsOff + W * S * 8;           // a run's first piece
  static constexpr int kRunOff = kFirstOff + W * kPieceFloats * 4;   // the CTA's tiles [lo, hi)
  static constexpr int kPairOff = kRunOff + 2 * 8;                   // pairs of the pieces [W][2]
  static constexpr int kCtxOff = kPairOff + W * 2 * 4;
  static constexpr int kReqOff = kCtxOff + kTcMaxSeqs * 4;
  static constexpr int kLowOff = kReqOff + kTcMaxSeqs * 4;
  static constexpr int kPrefixOff = kLowOff + kTcMaxSeqs * 4;
  static constexpr int kTotal = kPrefixOff + (kTcMaxSeqs + 1) * 4 + 1024;  // + 1 KiB alignment
  static_assert(kTotal <= 232448, "shared memory per CTA exceeds 227 KiB");
  static_assert(kPieceFloats * 4 <= S * kTcStageBytes, "a piece fits a warp's stages");
  static_assert(kFirstOff % 16 == 0 && kRecStride % 4 == 0, "float4 records");
};

}  // namespace

template <bool kContig, int W, int S, int MH>
__global__ void __launch_bounds__(W * 32, 1)
    decode_runs_kernel(const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv,
                       const __grid_constant__ TcParams p) {
  using L = RunsSmem<W, S, MH>;
  constexpr unsigned kFull = 0xffffffffu;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int tid = threadIdx.x;
  const int c = blockIdx.x;
  const int P = gridDim.x;
  const int B = p.num_seqs;
  const int G = p.G;
  const int Hkv = p.Hkv;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarsOff) + warp * S;
  int64_t* cta_run = reinterpret_cast<int64_t*>(smem + L::kRunOff);
  int32_t* piece_pair = reinterpret_cast<int32_t*>(smem + L::kPairOff);  // [W][first, last]
  int32_t* ctx_s = reinterpret_cast<int32_t*>(smem + L::kCtxOff);
  int32_t* req_s = reinterpret_cast<int32_t*>(smem + L::kReqOff);
  int32_t* low_s = reinterpret_cast<int32_t*>(smem + L::kLowOff);
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + L::kPrefixOff);
  // the record of head h of a run's first (0) or last (1) piece
  auto piece = [&](int w, int last, int h) -> float* {
    unsigned char* base = last ? smem + L::kStagesOff + w * S * kTcStageBytes
                               : smem + L::kFirstOff + w * L::kPieceFloats * 4;
    return reinterpret_cast<float*>(base) + h * kRecStride;
  };

  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&bars[s], 1);
    fence_barrier_init();
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
    piece_pair[2 * warp] = piece_pair[2 * warp + 1] = -1;
  }
  // wait for the previous kernel in the stream before reading any input, then
  // let the next one get scheduled (no-ops without the launch attribute)
  grid_dependency_wait();
  grid_dependency_trigger();

  // ---- visible positions, tile counts and their prefix over sequences
  for (int i = tid; i < B; i += W * 32) {
    int ctx = tc_context(p, i, kContig, c == 0);
    low_s[i] = tc_first_visible(p, i, ctx);
    ctx_s[i] = ctx;
    if (kContig) req_s[i] = ctx > 0 ? p.req_ids[i] : 0;
  }
  __syncthreads();
  auto seq_tiles = [&](int i) -> int { return ((ctx_s[i] + 15) >> 4) - (low_s[i] >> 4); };
  // position of the first row of tile n of sequence i
  auto tile_pos = [&](int i, int64_t n) -> int64_t { return (n + (low_s[i] >> 4)) * 16; };
  if (warp == 0) {
    const int per = (B + 31) / 32;
    const int i0 = lane * per;
    int sum = 0;
    for (int i = i0; i < i0 + per && i < B; ++i) sum += seq_tiles(i);
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    int run = incl - sum;
    for (int i = i0; i < i0 + per && i < B; ++i) {
      prefix[i] = run;
      run += seq_tiles(i);
    }
    if (lane == 31) prefix[B] = incl;
  }
  __syncthreads();

  // outputs of sequences that see nothing are zeros (c, c + P, ... of this CTA)
  for (int i = c; i < B; i += P) {
    if (ctx_s[i] != 0) continue;
    uint4* o = reinterpret_cast<uint4*>(p.out + static_cast<int64_t>(i) * p.Hq * kHeadDim);
    for (int k = tid; k < p.Hq * kHeadDim / 8; k += W * 32) o[k] = make_uint4(0u, 0u, 0u, 0u);
  }

  // ---- this warp's run of tiles [lo, hi): that of its share of the units
  const int64_t V = tc_vseq(prefix, B, Hkv, p.seg_cost);
  int64_t lo, hi;
  int seq_lo;  // the sequence that holds tile lo
  const int64_t share = static_cast<int64_t>(c) * W + warp;
  if (V < (int64_t{1} << 20) && P * W < 4096) {
    // in 32 bits, even lanes for the run's start and odd ones for its end (the
    // general form below takes 1 us longer)
    const uint32_t units = static_cast<uint32_t>(V), H = Hkv, cost = p.seg_cost;
    const uint32_t u = (static_cast<uint32_t>(share) + (lane & 1)) * units / (P * W);
    const uint32_t u0 = __shfl_sync(kFull, u, 0), u1 = __shfl_sync(kFull, u, 1);
    int a0 = 0, a1 = 0;  // the last sequences whose units start at or before them
    for (int i = lane; i < B; i += 32) {
      const uint32_t start = H * (prefix[i] + cost * i);
      if (start <= u0) a0 = i;
      if (start <= u1) a1 = i;
    }
    a0 = __reduce_max_sync(kFull, a0);
    a1 = __reduce_max_sync(kFull, a1);
    const int a = lane & 1 ? a1 : a0;
    const uint32_t n = prefix[a + 1] - prefix[a];
    const uint32_t r = u - H * (prefix[a] + cost * a);
    const uint32_t h = r / (n + cost), o = r - h * (n + cost);
    const uint32_t tile = u >= units ? H * prefix[B] : H * prefix[a] + h * n + (o > cost ? o - cost : 0);
    lo = __shfl_sync(kFull, tile, 0);
    hi = __shfl_sync(kFull, tile, 1);
    seq_lo = a0;
  } else {
    const int64_t parts = static_cast<int64_t>(P) * W;
    lo = tc_unit_to_tile(share * V / parts, prefix, B, Hkv, p.seg_cost);
    hi = tc_unit_to_tile((share + 1) * V / parts, prefix, B, Hkv, p.seg_cost);
    seq_lo = lo < hi ? tc_find_seg(lo, hi, prefix, B, Hkv).seq : 0;
  }
  if (lane == 0 && warp == 0) cta_run[0] = lo;
  if (lane == 0 && warp == W - 1) cta_run[1] = hi;
  // (an empty sequence's units hold no tile: the next one's first)
  while (lo < hi && static_cast<int64_t>(Hkv) * prefix[seq_lo + 1] <= lo) ++seq_lo;

  const uint32_t bs32 = static_cast<uint32_t>(p.bs);  // paged: a 32-bit block size
  const uint64_t policy = l2_policy_evict_first();
  unsigned char* stage0 = smem + L::kStagesOff + warp * S * kTcStageBytes;
  const int g = lane >> 2;   // accumulator row group
  const int tq = lane & 3;   // accumulator column pair

  // Q^T fragments of one pair straight from global memory: b0 = Q[g][16ks +
  // 2tq, +1], b1 = Q[g][16ks + 2tq + 8, +9] (heads >= G are 0).
  auto load_q = [&](uint32_t (&qf)[8][2], int seq, int kvh) {
    const uint32_t* qrow = reinterpret_cast<const uint32_t*>(
        p.q + (static_cast<int64_t>(seq) * p.Hq + kvh * G + (g < G ? g : 0)) * kHeadDim);
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      qf[ks][0] = g < G ? __ldg(qrow + ks * 8 + tq) : 0u;
      qf[ks][1] = g < G ? __ldg(qrow + ks * 8 + 4 + tq) : 0u;
    }
  };
  // the pair after `sg` (its tiles start at sg.pend < hi)
  auto next_seg = [&](const TcSeg& sg) -> TcSeg {
    int a = sg.seq;
    if (sg.kvh + 1 == Hkv)
      do ++a; while (prefix[a + 1] == prefix[a]);
    return tc_seg_at(sg.pend, hi, a, prefix, Hkv);
  };

  int issued = 0, consumed = 0;
  bool dead = false;
  if (lo < hi) {
    // ---- the issue cursor: tile ix of pair iseg
    TcSeg iseg = tc_seg_at(lo, hi, seq_lo, prefix, Hkv);
    int64_t ix = lo;
    // The next pair's Q fragments are fetched into qn when the cursor first
    // reaches it (if qn is free), so its start does not wait on them.
    uint32_t qn[8][2];
    int64_t qn_pair = -1;
    auto load_entry = [&]() -> int32_t {  // block-table entry of tile ix (lane 0)
      if (kContig || lane != 0 || ix >= hi) return 0;
      const int64_t pos = tile_pos(iseg.seq, ix - iseg.pstart);
      return __ldg(p.block_tables + static_cast<int64_t>(iseg.seq) * p.max_blocks +
                   static_cast<uint32_t>(pos) / bs32);
    };
    auto issue = [&](int stage, int32_t entry) {
      if (ix == iseg.x0 && qn_pair < 0) {  // whole warp
        load_q(qn, iseg.seq, iseg.kvh);
        qn_pair = iseg.pstart;
      }
      if (lane == 0) {
        unsigned char* st = stage0 + stage * kTcStageBytes;
        const int64_t pos = tile_pos(iseg.seq, ix - iseg.pstart);
        bool kv_ok = true;
        int64_t row;
        if (kContig) {
          row = cache_row(req_s[iseg.seq], iseg.kvh, Hkv, p.bs, pos);
        } else {
          if (p.checked && (entry < 0 || entry >= p.num_blocks)) {
            record_error(p.err, kErrBlockId);
            kv_ok = false;  // skip the copy: stale rows, undefined output, no fault
          }
          row = cache_row(entry, iseg.kvh, Hkv, p.bs, static_cast<uint32_t>(pos) % bs32);
        }
        mbar_arrive_expect_tx(&bars[stage], kv_ok ? 4u * kBoxBytes : 0u);
        if (kv_ok) {
          const int32_t y = static_cast<int32_t>(row);
          tma_load_2d(st, &tmk, 0, y, &bars[stage], policy);
          tma_load_2d(st + kBoxBytes, &tmk, 64, y, &bars[stage], policy);
          tma_load_2d(st + 2 * kBoxBytes, &tmv, 0, y, &bars[stage], policy);
          tma_load_2d(st + 3 * kBoxBytes, &tmv, 64, y, &bars[stage], policy);
        }
      }
      ++issued;
      if (++ix >= iseg.x1 && ix < hi) iseg = next_seg(iseg);
    };

    // Prologue: lane s fetches the table entry of tile lo + s (one memory
    // latency for all of them), then the stages fill.
    int32_t pre = 0;
    if (!kContig) {
      TcSeg cs = iseg;
      for (int s = 0; s < S && lo + s < hi; ++s) {
        if (lo + s >= cs.x1) cs = next_seg(cs);
        if (lane == s) {
          const int64_t pos = tile_pos(cs.seq, lo + s - cs.pstart);
          pre = __ldg(p.block_tables + static_cast<int64_t>(cs.seq) * p.max_blocks +
                      static_cast<uint32_t>(pos) / bs32);
        }
      }
    }
    for (int s = 0; s < S && ix < hi; ++s) issue(s, __shfl_sync(kFull, pre, s));
    int32_t next_entry = load_entry();

    // ---- per-lane ldmatrix offsets inside a 128-byte-swizzled 16 x 128 B box
    uint32_t koff[4], voff[4];
    {
      const int rk = (lane & 7) + 8 * ((lane >> 3) & 1), hk = lane >> 4;
      const int rv = (lane & 7) + 8 * (lane >> 4), hv = (lane >> 3) & 1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        koff[j] = rk * 128 + ((((2 * j + hk) ^ (rk & 7))) << 4);
        voff[j] = rv * 128 + ((((2 * j + hv) ^ (rv & 7))) << 4);
      }
    }

    TcSeg seg = tc_seg_at(lo, hi, seq_lo, prefix, Hkv);
    while (true) {
      uint32_t qb[8][2];
      if (qn_pair == seg.pstart) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          qb[ks][0] = qn[ks][0];
          qb[ks][1] = qn[ks][1];
        }
        qn_pair = -1;
      } else {
        load_q(qb, seg.seq, seg.kvh);
      }
      const int ctx = ctx_s[seg.seq];
      const int low = low_s[seg.seq];
      float slope0 = 0.f, slope1 = 0.f;  // of heads 2tq, 2tq + 1
      if (p.sp.slopes != nullptr) {
        slope0 = 2 * tq < G ? slope_log2(p.sp.slopes, seg.kvh * G + 2 * tq) : 0.f;
        slope1 = 2 * tq + 1 < G ? slope_log2(p.sp.slopes, seg.kvh * G + 2 * tq + 1) : 0.f;
      }
      float acc[8][4];
      float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;

      for (int64_t x = seg.x0; x < seg.x1 && !dead; ++x) {
        const int stage = consumed % S;
        if (!__all_sync(kFull, mbar_wait_bounded(&bars[stage],
                                                 static_cast<uint32_t>(consumed / S) & 1u))) {
          dead = true;
          if (lane == 0) record_error(p.err, kErrTimeout);
          break;
        }
        ++consumed;
        unsigned char* st = stage0 + stage * kTcStageBytes;
        const uint32_t kaddr = smem_addr(st);
        const uint32_t vaddr = kaddr + 2 * kBoxBytes;
        const int row0 = static_cast<int>(tile_pos(seg.seq, x - seg.pstart));
        const int nvalid = min(16, ctx - row0);
        const int nlow = max(0, low - row0);  // rows before the first visible
        if (nvalid < 16 || nlow > 0) {  // masked rows must not feed p.V (0 * NaN)
          for (int idx = lane; idx < (nlow + 16 - nvalid) * 16; idx += 32) {
            const int r = idx >> 4;
            const int rr = r < nlow ? r : nvalid + r - nlow;
            const int ch = idx & 15;
            *reinterpret_cast<uint4*>(st + 2 * kBoxBytes + (ch >> 3) * kBoxBytes + rr * 128 +
                                      (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          __syncwarp();
        }

        // ---- S^T = K . Q^T  (two accumulation chains)
        float sa[4] = {0.f, 0.f, 0.f, 0.f}, sb[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          uint32_t a[4];
          ldmatrix_x4(a, kaddr + (ks >> 2) * kBoxBytes + koff[ks & 3]);
          if (ks & 1) mma_bf16_16816(sb, a, qb[ks][0], qb[ks][1]);
          else mma_bf16_16816(sa, a, qb[ks][0], qb[ks][1]);
        }
        // scores of tokens g (x0, x1) and g + 8 (x2, x3), heads 2tq and 2tq + 1
        float x0 = (sa[0] + sb[0]) * p.qscale, x1 = (sa[1] + sb[1]) * p.qscale;
        float x2 = (sa[2] + sb[2]) * p.qscale, x3 = (sa[3] + sb[3]) * p.qscale;
        if (p.sp.cap2 > 0.f) {
          x0 = capped_score(p.sp, x0);
          x1 = capped_score(p.sp, x1);
          x2 = capped_score(p.sp, x2);
          x3 = capped_score(p.sp, x3);
        }
        if (p.sp.slopes != nullptr) {
          const float d0 = static_cast<float>(ctx - 1 - (row0 + g));
          const float d1 = static_cast<float>(ctx - 1 - (row0 + g + 8));
          x0 = fmaf(-slope0, d0, x0);
          x1 = fmaf(-slope1, d0, x1);
          x2 = fmaf(-slope0, d1, x2);
          x3 = fmaf(-slope1, d1, x3);
        }
        const bool v0 = g < nvalid && g >= nlow, v1 = g + 8 < nvalid && g + 8 >= nlow;
        const float s0 = v0 ? x0 : -INFINITY, s1 = v0 ? x1 : -INFINITY;
        const float s2 = v1 ? x2 : -INFINITY, s3 = v1 ? x3 : -INFINITY;

        // ---- online softmax, per head column
        float mx0 = fmaxf(s0, s2), mx1 = fmaxf(s1, s3);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, o));
          mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, o));
        }
        const float n0 = fmaxf(m0, mx0), n1 = fmaxf(m1, mx1);
        if (n0 > m0) {
          const float a = fast_exp2(m0 - n0);
          l0 *= a;
#pragma unroll
          for (int i = 0; i < 8; ++i) { acc[i][0] *= a; acc[i][2] *= a; }
          m0 = n0;
        }
        if (n1 > m1) {
          const float a = fast_exp2(m1 - n1);
          l1 *= a;
#pragma unroll
          for (int i = 0; i < 8; ++i) { acc[i][1] *= a; acc[i][3] *= a; }
          m1 = n1;
        }
        const float f0 = finite_max(m0), f1 = finite_max(m1);
        const float p0 = fast_exp2(s0 - f0), p2 = fast_exp2(s2 - f0);
        const float p1 = fast_exp2(s1 - f1), p3 = fast_exp2(s3 - f1);
        // P^T as the B operand, rounded to bf16 (V's type) once; l sums what was
        // rounded, so that it cancels where few keys are seen
        const uint32_t w01 = pack_bf16x2(p0, p1), w23 = pack_bf16x2(p2, p3);
        l0 += bf16_lo(w01) + bf16_lo(w23);
        l1 += bf16_hi(w01) + bf16_hi(w23);
        const uint32_t b0 = movmatrix_trans(w01);  // tokens 0..7
        const uint32_t b1 = movmatrix_trans(w23);  // tokens 8..15

        // ---- O^T += V^T . P^T
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint32_t a[4];
          ldmatrix_x4_trans(a, vaddr + (i >> 2) * kBoxBytes + voff[i & 3]);
          mma_bf16_16816(acc[i], a, b0, b1);
        }
        __syncwarp();

        // ---- refill this stage with the next tile of the run
        if (ix < hi) {
          fence_proxy_async_smem();
          issue(stage, next_entry);
          next_entry = load_entry();
        }
      }
      if (dead) break;

      // ---- the pair's part in this run is done
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l0 += __shfl_xor_sync(kFull, l0, o);
        l1 += __shfl_xor_sync(kFull, l1, o);
      }
      if (seg.x0 == seg.pstart && seg.x1 == seg.pend) {
        // whole: lane g even writes elements 16i + g, + 1, odd 16i + 7 + g, + 1
        const float inv0 = l0 > 0.f ? 1.f / l0 : 0.f, inv1 = l1 > 0.f ? 1.f / l1 : 0.f;
        const bool odd = g & 1;
        uint16_t* row = p.out + (static_cast<int64_t>(seg.seq) * p.Hq + seg.kvh * G + 2 * tq) *
                                    kHeadDim + (odd ? 7 + g : g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float inv = e == 0 ? inv0 : inv1;
            const float low8 = acc[i][e] * inv, high8 = acc[i][e + 2] * inv;
            const float got = __shfl_xor_sync(kFull, odd ? low8 : high8, 4);
            const uint32_t w = odd ? pack_bf16x2(got, high8) : pack_bf16x2(low8, got);
            if (2 * tq + e < G) *reinterpret_cast<uint32_t*>(row + e * kHeadDim + 16 * i) = w;
          }
        }
      } else {
        const int last = seg.x0 != lo;  // a run's first piece, or (not first) its last
        if (2 * tq < MH) {
          float* r0 = piece(warp, last, 2 * tq);
          float* r1 = r0 + kRecStride;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            r0[16 * i + g] = acc[i][0];
            r1[16 * i + g] = acc[i][1];
            r0[16 * i + g + 8] = acc[i][2];
            r1[16 * i + g + 8] = acc[i][3];
          }
          if (g == 0) {
            r0[128] = m0;
            r0[129] = l0;
            r1[128] = m1;
            r1[129] = l1;
          }
        }
        if (lane == 0) piece_pair[2 * warp + last] = seg.seq * Hkv + seg.kvh;
      }
      if (seg.x1 >= hi) break;
      seg = next_seg(seg);
    }
    if (dead) {
      // give the copies still in flight a bounded chance to land
      for (int k = consumed; k < issued; ++k)
        mbar_wait_bounded(&bars[k % S], static_cast<uint32_t>(k / S) & 1u);
    }
  }
  __syncthreads();

  // ---- join the pieces of each pair that warps of this CTA share: pieces in
  // warp order, lane j's is piece_pair[j] (2 W <= 32); consecutive ones of a pair
  // are a group, and head h of group g is task g G + h, dealt to the warps
  const int lane_pair = lane < 2 * W ? piece_pair[lane] : -1;
  const uint32_t taken = __ballot_sync(kFull, lane_pair >= 0);
  const uint32_t before = taken & ((1u << lane) - 1u);
  const int prev_pair = __shfl_sync(kFull, lane_pair, before != 0u ? 31 - __clz(before) : lane);
  const uint32_t starts =
      __ballot_sync(kFull, lane_pair >= 0 && (before == 0u || prev_pair != lane_pair));
  const int tasks = __popc(starts) * G;
  // (last group first: what a later CTA waits for goes out before a wait for earlier ones)
  for (int task = tasks - 1 - warp; task >= 0; task -= W) {
    const int grp = static_cast<uint32_t>(task) / static_cast<uint32_t>(G);
    const int hh = task - grp * G;
    uint32_t rest = starts;
    for (int k = 0; k < grp; ++k) rest &= rest - 1;
    const int n = __ffs(rest) - 1;  // pieces n .. end - 1 are this pair's (or empty)
    rest &= rest - 1;
    const int end = rest != 0u ? __ffs(rest) - 1 : 2 * W;
    const int pair = __shfl_sync(kFull, lane_pair, n);
    // lane j < end - n derives the weight of piece n + j (2 W <= 32 lanes)
    const int k = n + lane;
    const bool have = k < end && (taken >> k & 1u);
    const float* rk = piece(k < end ? k >> 1 : 0, k & 1, hh);
    const float mj = have ? rk[128] : -INFINITY, lj = have ? rk[129] : 0.f;
    float M = mj;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    // (a piece that saw scores of -inf or NaN alone has no maximum: its sum says)
    const float fj = lj == 0.f ? 0.f : fast_exp2(mj - M);
    float Ls = lj * fj;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) Ls += __shfl_xor_sync(kFull, Ls, o);
    const float wj = Ls != 0.f ? fj / Ls : 0.f;
    float4 o4 = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int e = n; e < end; ++e) {
      const float w = __shfl_sync(kFull, wj, e - n);
      if (!(taken >> e & 1u)) continue;
      const float4 v = *reinterpret_cast<const float4*>(piece(e >> 1, e & 1, hh) + lane * 4);
      o4.x = fmaf(w, v.x, o4.x);
      o4.y = fmaf(w, v.y, o4.y);
      o4.z = fmaf(w, v.z, o4.z);
      o4.w = fmaf(w, v.w, o4.w);
    }
    const float Mr = Ls != 0.f ? M : -INFINITY;
    // the CTAs cf .. cl that hold tiles of the pair
    TcSeg sg;
    sg.seq = static_cast<uint32_t>(pair) / static_cast<uint32_t>(Hkv);
    sg.kvh = pair - sg.seq * Hkv;
    const int64_t tiles = prefix[sg.seq + 1] - prefix[sg.seq];
    sg.pstart = static_cast<int64_t>(Hkv) * prefix[sg.seq] + sg.kvh * tiles;
    sg.pend = sg.pstart + tiles;
    sg.x0 = sg.pstart;
    sg.x1 = sg.pend;
    int cf = c, cl = c;
    if (sg.pstart < cta_run[0] || sg.pend > cta_run[1])
      tc_pair_ctas(sg, prefix, Hkv, p.seg_cost, V, P, &cf, &cl);
    const int qh = sg.kvh * G + hh;
    if (cf == cl) {
      tc_write_out(p, sg.seq, qh, lane, o4, Mr, Ls);
    } else if (cl != c) {
      tc_store_piece(p.rec + (static_cast<int64_t>(c) * kTcRecHeads + hh) * kRecStride, p.tag,
                     lane, o4, Mr, Ls);
    } else if (!tc_merge_earlier(p, sg.seq, qh, hh, cf, c, V, P, lane, o4, Mr, Ls) && lane == 0) {
      record_error(p.err, kErrTimeout);
    }
  }
}

namespace {

template <bool kContig, int W, int S, int MH>
cudaError_t launch_shape(const CUtensorMap& tk, const CUtensorMap& tv, const TcParams& p0,
                         int num_ctas, cudaStream_t stream) {
  using L = RunsSmem<W, S, MH>;
  static unsigned long long done_mask = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  auto kernel = decode_runs_kernel<kContig, W, S, MH>;
  if (!(__atomic_load_n(&done_mask, __ATOMIC_ACQUIRE) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal);
    if (e != cudaSuccess) return e;
    __atomic_fetch_or(&done_mask, bit, __ATOMIC_ACQ_REL);
  }
  const int chunk = tc_chunk_seqs(p0.max_context);
  for (int s0 = 0; s0 < p0.num_seqs; s0 += chunk) {
    TcParams p = p0;
    p.num_seqs = (p0.num_seqs - s0) < chunk ? (p0.num_seqs - s0) : chunk;
    p.q += static_cast<int64_t>(s0) * p.Hq * kHeadDim;
    p.out += static_cast<int64_t>(s0) * p.Hq * kHeadDim;
    p.ctx_lens += s0;
    if (p.sp.first_key != nullptr) p.sp.first_key += s0;
    if (kContig) p.req_ids += s0;
    else p.block_tables += static_cast<int64_t>(s0) * p.max_blocks;
    p.tag = next_launch_tag();  // every launch writes its piece records under a fresh tag
    e = launch_pdl_if(pdl_decode_enabled(), kernel, dim3(num_ctas), dim3(W * 32), L::kTotal,
                      stream, tk, tv, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_decode_runs(const CUtensorMap& tk, const CUtensorMap& tv, const TcParams& p_in,
                               bool contig, int num_ctas, cudaStream_t stream) {
  TcParams p = p_in;
  // The cost of a pair in tiles: 3, 4, 6 and 9 give 25.4, 25.1, 25.3 and 24.9 us
  // (64 ragged sequences, window 1024), 15.3, 15.5, 15.5 and 16.2 (window 256),
  // 15.3, 15.5, 16.1 and 16.9 (64 of 256).
  p.seg_cost = 4;
  if (p.G <= 4)
    return contig ? launch_shape<true, 12, 2, 4>(tk, tv, p, num_ctas, stream)
                  : launch_shape<false, 12, 2, 4>(tk, tv, p, num_ctas, stream);
  if (p.G <= kTcHeads)
    return contig ? launch_shape<true, 10, 2, 8>(tk, tv, p, num_ctas, stream)
                  : launch_shape<false, 10, 2, 8>(tk, tv, p, num_ctas, stream);
  return cudaErrorInvalidValue;
}

}  // namespace pkv
