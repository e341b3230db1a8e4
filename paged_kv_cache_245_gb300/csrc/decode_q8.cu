// decode_q8.cu -- decode attention over the 8-bit KV cache (q8.cuh), paged or
// contiguous: warp-level tensor-core math on 16-token tiles, each of which has
// one scale for K and one for V, and a persistent schedule balanced over every
// warp of the GPU.  sm_103a.
//
// For sequence i, query head h and KV head h / G:
//   out[i][h] = sum_j softmax_j(scale q . k_j) v_j,  k_j = kcode_j ks, v_j = vcode_j vs
// with ks and vs of the tile that holds j.  So
//   S = (q . kcode) (scale ks),   O += vs (P vcode)
// and the matrix products run on the codes themselves, which fp16 holds exactly
// (e4m3 by the conversion instruction; int8 as 1024 + 128 + code, put together
// from bytes, less 1152).  Queries enter as fp16 too: each row times a power of
// two that puts its largest element at 2^14 .. 2^15, exact for bf16 elements down
// to 2^-28 of that.  P, at most 1, is rounded to fp16 times 2^15 (off by 2^-11 of it down
// to 2^-29, by 2^-40 below); a tile's product is added to O in fp32 with its vs 2^-15.
//
// Schedule: that of decode_runs.cu -- the flattened list of tiles of every
// (sequence, KV head) pair cut evenly over the warps of the grid, pieces of a
// pair joined in shared memory within a CTA and through tagged records across.
//
// Data movement.  A tile is 16 rows x 128 bytes of K and as much of V, one TMA
// box each, 128-byte swizzled, into a per-warp ring of stages; the two scales
// come by cp.async and arrive on the same mbarrier.  A stage holds two tiles,
// which lanes 0 and 1 look up and ask for side by side, so that what is done once
// a stage (waits, the running maximum, the cursor) is done once for 32 positions.
//
// Math of a tile (one warp).  A lane takes two 16-byte chunks of K rows g and
// g + 8; which element of the head a k-slot of the product stands for is free, so
// word w of a lane's chunks is k-step w (elements 32 tq + 4 w ..) and Q's
// fragments are loaded in the same order.  V comes by ldmatrix.trans on pairs of
// codes: of elements 2g and 2g + 1 the lane gets keys 2tq and 2tq + 1, and rows g
// and g + 8 of the product stand for those two elements, so that the output's
// neighbours meet in one lane.
//
// What bounds it: HBM, past 8 us that the launch, the schedule (contexts, table, rows
// one after another) and the joins take.  128 sequences of 8000 to 8192 with 8 KV heads of
// 7 query heads (2.13 GB, e4m3) take 328 us, 6.5 TB/s or 0.96 of a plain copy; 64 ragged
// ones up to 8192 (157 MB) 33 us, 0.70; 32 of 100 to 4095 with 4 KV heads (36 MB) 16 us,
// 0.33; long contexts (int8, 4 query heads): 8 of 131072 (2.15 GB) 336 us, 0.94, 8 of
// 32768 90 us, one of 131072 55 us, of 32768 25 us.  Two tiles a stage took the first from
// 453 to 334 us.  Small batches are decode_q8_cluster.cu's.
//
// Chunks of few tokens (kChunks) are the same with 16 rows, (token, query head) pairs of
// up to 16 / G tokens, in two columns of products; each row masks the positions past its
// token.  64 chunks of 4 tokens after 2000 take 74 us for 39 us of reads: eight warps of
// 255 registers, two a scheduler, wait for their own results (issue slots 39 % busy).
#include "decode_launch.cuh"
#include "decode_tc.cuh"
#include "q8.cuh"
#include "q8_math.cuh"
#include "umma.cuh"

namespace pkv {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kTileCodes = 16 * kCodeRowBytes;  // 2 KiB
constexpr int kStageTiles = 2;                  // tiles of a stage, each K then V
constexpr int kStageQ8 = kStageTiles * 2 * kTileCodes;

struct DecodeQ8Params : TcParams {
  const float* k_scale;
  const float* v_scale;
  // Short chunks: sequence i of the schedule is token group i % groups of chunk i /
  // groups, group_tokens tokens, as 16 rows (token, query head) where decode has 8.
  const int32_t* cu_q;
  int32_t groups, group_tokens, max_q;
};

// W warps, S stages each; MH rows (query heads) of a KV head (4, 8; chunks: 16).
template <int W, int S, int MH>
struct Q8Smem {
  static constexpr int kPieceFloats = MH * kRecStride;  // o[128], m, l of each head
  static constexpr int kStagesOff = 0;                  // (a run's last piece goes over its stages)
  static constexpr int kBarsOff = W * S * kStageQ8;
  static constexpr int kScalesOff = kBarsOff + W * S * 8;        // (K, V) of each tile
  static constexpr int kFirstOff = kScalesOff + W * S * kStageTiles * 8;  // a run's first piece
  static constexpr int kRunOff = kFirstOff + W * kPieceFloats * 4;  // the CTA's tiles [lo, hi)
  static constexpr int kPairOff = kRunOff + 2 * 8;               // pairs of the pieces [W][2]
  static constexpr int kCtxOff = kPairOff + W * 2 * 4;
  static constexpr int kReqOff = kCtxOff + kTcMaxSeqs * 4;
  static constexpr int kRowOff = kReqOff + kTcMaxSeqs * 4;  // chunks: a group's first row of q
  static constexpr int kTokOff = kRowOff + (MH == 16 ? kTcMaxSeqs * 4 : 0);  // and its tokens
  static constexpr int kPrefixOff = kTokOff + (MH == 16 ? kTcMaxSeqs * 4 : 0);
  static constexpr int kTotal = kPrefixOff + (kTcMaxSeqs + 1) * 4 + 1024;  // + 1 KiB alignment
  static_assert(kTotal <= 232448, "shared memory per CTA exceeds 227 KiB");
  static_assert(kPieceFloats * 4 <= S * kStageQ8, "a piece fits a warp's stages");
  static_assert(kFirstOff % 16 == 0 && kRunOff % 8 == 0, "float4 records, 64-bit runs");
};

// The mbarrier counts one arrival more: when this thread's cp.async copies land.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

}  // namespace

template <bool kContig, bool kE4m3, bool kChunks, int W, int S, int MH>
__global__ void __launch_bounds__(W * 32, 1)
    decode_q8_kernel(const __grid_constant__ CUtensorMap tmk,
                     const __grid_constant__ CUtensorMap tmv,
                     const __grid_constant__ DecodeQ8Params p) {
  using L = Q8Smem<W, S, MH>;
  constexpr int NT = kChunks ? 2 : 1;  // tiles of 8 rows of queries
  static_assert(MH <= 8 * NT && kChunks == (MH == 16), "rows of the tiles");
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
  float2* scales = reinterpret_cast<float2*>(smem + L::kScalesOff) + warp * S * kStageTiles;
  int64_t* cta_run = reinterpret_cast<int64_t*>(smem + L::kRunOff);
  int32_t* piece_pair = reinterpret_cast<int32_t*>(smem + L::kPairOff);  // [W][first, last]
  int32_t* ctx_s = reinterpret_cast<int32_t*>(smem + L::kCtxOff);
  int32_t* req_s = reinterpret_cast<int32_t*>(smem + L::kReqOff);
  int32_t* row_s = reinterpret_cast<int32_t*>(smem + L::kRowOff);  // kChunks
  int32_t* tok_s = reinterpret_cast<int32_t*>(smem + L::kTokOff);
  int32_t* prefix = reinterpret_cast<int32_t*>(smem + L::kPrefixOff);
  // rows of sequence i, and its first row of q and out in units of Hq rows
  auto rows_of = [&](int i) -> int { return kChunks ? tok_s[i] * G : G; };
  auto token_of = [&](int i) -> int { return kChunks ? row_s[i] : i; };
  // the record of head h of a run's first (0) or last (1) piece
  auto piece = [&](int w, int last, int h) -> float* {
    unsigned char* base = last ? smem + L::kStagesOff + w * S * kStageQ8
                               : smem + L::kFirstOff + w * L::kPieceFloats * 4;
    return reinterpret_cast<float*>(base) + h * kRecStride;
  };

  if (lane == 0) {
    // the boxes', and each tile's scales'
    for (int s = 0; s < S; ++s) mbar_init(&bars[s], 1 + kStageTiles);
    fence_barrier_init();
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
    piece_pair[2 * warp] = piece_pair[2 * warp + 1] = -1;
  }
  // wait for the previous kernel in the stream before reading any input, then
  // let the next one get scheduled (no-ops without the launch attribute)
  grid_dependency_wait();
  grid_dependency_trigger();

  // ---- tile counts and their prefix over sequences
  for (int i = tid; i < B; i += W * 32) {
    if constexpr (kChunks) {
      // the keys that the group's last token sees
      const int seq = i / p.groups, t0 = (i - seq * p.groups) * p.group_tokens;
      const int q0 = p.cu_q[seq], n = p.cu_q[seq + 1] - q0;
      int ctx = p.ctx_lens[seq], req = kContig ? p.req_ids[seq] : 0;
      if (p.checked) {
        const int64_t cap = kContig ? p.bs : static_cast<int64_t>(p.max_blocks) * p.bs;
        const bool bad = n < 0 || n > p.max_q || ctx < n || ctx > cap;
        if ((bad || req < 0 || (kContig && req >= p.max_reqs)) && n != 0) {
          if (c == 0 && t0 == 0) record_error(p.err, bad ? kErrContext : kErrReqId);
          ctx = 0;  // the sequence is left unwritten
          req = 0;
        }
      }
      const int tokens = min(p.group_tokens, min(n, p.max_q) - t0);
      ctx_s[i] = ctx > 0 && tokens > 0 ? max(ctx - n + t0 + tokens, 0) : 0;
      row_s[i] = q0 + t0;
      tok_s[i] = tokens;
      if (kContig) req_s[i] = req;
    } else {
      const int ctx = tc_context(p, i, kContig, c == 0);
      ctx_s[i] = ctx;
      if (kContig) req_s[i] = ctx > 0 ? p.req_ids[i] : 0;
    }
  }
  __syncthreads();
  auto seq_tiles = [&](int i) -> int { return (ctx_s[i] + 15) >> 4; };
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

  // outputs of empty contexts are zeros (sequences c, c + P, ... of this CTA)
  for (int i = c; i < B && !kChunks; i += P) {
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

  const uint64_t policy = l2_policy_evict_first();
  unsigned char* stage0 = smem + L::kStagesOff + warp * S * kStageQ8;
  const int g = lane >> 2;   // accumulator row group
  const int tq = lane & 3;   // accumulator column pair

  // Elements 32 tq .. + 31 of query row r of a sequence (row 0's where it has fewer).
  auto q_row = [&](int seq, int kvh, int r) {
    int token = token_of(seq), head = r;
    if (r >= rows_of(seq)) head = 0;
    if (kChunks) {
      token += head / G;
      head %= G;
    }
    return p.q + (static_cast<int64_t>(token) * p.Hq + kvh * G + head) * kHeadDim + 32 * tq;
  };
  // the pair after `sg` (its tiles start at sg.pend < hi)
  auto next_seg = [&](const TcSeg& sg) -> TcSeg {
    int a = sg.seq;
    if (sg.kvh + 1 == Hkv)
      do ++a; while (prefix[a + 1] == prefix[a]);
    return tc_seg_at(sg.pend, hi, a, prefix, Hkv);
  };

  int issued = 0, consumed = 0;  // stages
  bool dead = false;
  if (lo < hi) {
    // ---- the issue cursor: tiles in .. of pair iseg, in_end of them in this run.
    // Lane l (0, 1) has the position of tile in + l: entry `blk` of the table, row
    // `off` of its block (contiguous: row off of the request).
    const uint32_t bs32 = static_cast<uint32_t>(p.bs);
    const uint32_t step_blk = 16 * kStageTiles / bs32, step_off = 16 * kStageTiles % bs32;
    TcSeg iseg = tc_seg_at(lo, hi, seq_lo, prefix, Hkv);
    int in = 0, in_end = 0;
    uint32_t blk = 0, off = 0;
    const int32_t* table = nullptr;  // of iseg's sequence
    int32_t entry = 0;  // of this lane's tile
    bool more = true;   // tiles are left to ask for
    auto look_up = [&]() {
      if (kContig) return;
      if (lane < kStageTiles && more && in + lane < in_end) entry = __ldg(table + blk);
    };
    auto at_seg = [&]() {
      in = static_cast<int>(iseg.x0 - iseg.pstart);
      in_end = static_cast<int>(iseg.x1 - iseg.pstart);
      // its query rows, which the pair's start waits for
#pragma unroll
      for (int y = 0; y < NT; ++y)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(q_row(iseg.seq, iseg.kvh, 8 * y + g)));
      const uint32_t pos = static_cast<uint32_t>(in + lane) * 16;
      if (kContig) {
        off = pos;
        entry = req_s[iseg.seq];
      } else {
        blk = pos / bs32;
        off = pos - blk * bs32;
        table = p.block_tables +
                static_cast<int64_t>(kChunks ? iseg.seq / p.groups : iseg.seq) * p.max_blocks;
      }
    };
    auto issue = [&](int stage) {
      if (lane < kStageTiles) {
        unsigned char* st = stage0 + stage * kStageQ8 + lane * 2 * kTileCodes;
        bool ok = in + lane < in_end;
        if (!kContig && p.checked && ok && (entry < 0 || entry >= p.num_blocks)) {
          record_error(p.err, kErrBlockId);
          ok = false;  // skip the copy: stale rows, undefined output, no fault
        }
        // (rows of the whole cache are fewer than 2^31)
        const uint32_t row = (static_cast<uint32_t>(entry) * static_cast<uint32_t>(Hkv) +
                              static_cast<uint32_t>(iseg.kvh)) * bs32 + off;
        const uint32_t tiles = __popc(__ballot_sync((1u << kStageTiles) - 1u, ok));
        if (lane == 0) mbar_arrive_expect_tx(&bars[stage], tiles * 2 * kTileCodes);
        __syncwarp((1u << kStageTiles) - 1u);
        if (ok) {
          const int32_t y = static_cast<int32_t>(row);
          tma_load_2d(st, &tmk, 0, y, &bars[stage], policy);
          tma_load_2d(st + kTileCodes, &tmv, 0, y, &bars[stage], policy);
          float2* sc = &scales[stage * kStageTiles + lane];
          cp_async_4(&sc->x, p.k_scale + (row >> 4));
          cp_async_4(&sc->y, p.v_scale + (row >> 4));
        }
        cp_async_arrive(&bars[stage]);
      }
      __syncwarp();
      ++issued;
      in += kStageTiles;
      off += step_off;
      blk += step_blk;
      if (!kContig && off >= bs32) {
        off -= bs32;
        ++blk;
      }
      if (in >= in_end) {
        more = iseg.x1 < hi;
        if (more) {
          iseg = next_seg(iseg);
          at_seg();
        }
      }
      look_up();
    };
    at_seg();
    look_up();
    if (more) issue(0);

    // ---- per-lane offsets inside a 128-byte-swizzled 16 x 128 B box
    // K: chunks 2 tq and 2 tq + 1 of row g (row g + 8: 1 KiB on)
    const uint32_t koff0 = g * 128 + (((2 * tq) ^ g) << 4);
    const uint32_t koff1 = g * 128 + (((2 * tq + 1) ^ g) << 4);
    // V: lanes 0-7 address keys 0-7 of chunk c, 8-15 keys 8-15, 16-31 chunk c + 1
    const int vrow = lane & 15, vch = lane >> 4;

    TcSeg seg = tc_seg_at(lo, hi, seq_lo, prefix, Hkv);
    while (true) {
      const int ctx = ctx_s[seg.seq];
      const int rows = rows_of(seg.seq);
      uint32_t qb[NT][8][2];
      float qs[NT][2];  // score units of rows 8 y + 2 tq and + 1
      int lim[NT][2];   // positions that they see (chunks)
#pragma unroll
      for (int y = 0; y < NT; ++y) {
        uint4 qn[4];
        const uint4* row = reinterpret_cast<const uint4*>(q_row(seg.seq, seg.kvh, 8 * y + g));
#pragma unroll
        for (int k = 0; k < 4; ++k)
          qn[k] = 8 * y + g < rows ? __ldg(row + k) : make_uint4(0u, 0u, 0u, 0u);
        const float down = queries_to_half(qn, qb[y]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          qs[y][e] = __shfl_sync(kFull, down, 8 * tq + 4 * e) * p.qscale;
          lim[y][e] = ctx;
          if (kChunks)
            lim[y][e] -= max(tok_s[seg.seq] - 1 - (8 * y + 2 * tq + e) / G, 0);
        }
      }
      // The run's other first stages only now: asked for at once by every warp, the first
      // stage of each came as late as the last (32 sequences of 1100 with 4 KV heads 17.1 ->
      // 16.1 us, 32 ragged ones with 8 27.0 -> 26.3).
      while (issued < S && more) issue(issued);
      // O^T of elements 16 i + 2 g (0) and + 1 (1): rows 8 y + 2 tq and + 1 as a pair
      uint64_t acc[NT][8][2];
      float m[NT][2], l[NT][2];
#pragma unroll
      for (int y = 0; y < NT; ++y) {
        m[y][0] = m[y][1] = -INFINITY;
        l[y][0] = l[y][1] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[y][i][0] = acc[y][i][1] = 0ull;
      }

      const int x_end = static_cast<int>(seg.x1 - seg.pstart);
      for (int x = static_cast<int>(seg.x0 - seg.pstart); x < x_end; x += kStageTiles) {
        const int stage = consumed % S;
        if (!__all_sync(kFull, mbar_wait_bounded(&bars[stage],
                                                 static_cast<uint32_t>(consumed / S) & 1u))) {
          dead = true;
          if (lane == 0) record_error(p.err, kErrTimeout);
          break;
        }
        ++consumed;
        unsigned char* st = stage0 + stage * kStageQ8;
        // rows of the stage that hold positions of the run's part of the pair
        const int nvalid = min(16 * min(kStageTiles, x_end - x), ctx - x * 16);
        const bool two = nvalid > 16;
        if (kE4m3 && (nvalid & 15) != 0) {  // rows past the context may hold NaN: 0 * NaN
          unsigned char* vt = st + kTileCodes + (two ? 2 * kTileCodes : 0);
          const int first = nvalid & 15;
          for (int idx = lane; idx < (16 - first) * 8; idx += 32)
            *reinterpret_cast<uint4*>(vt + first * 128 + idx * 16) = make_uint4(0u, 0u, 0u, 0u);
          __syncwarp();
        }

        // ---- S^T = K . Q^T; s[y][t]: scores of tokens g (0, 1) and g + 8 (2, 3) of
        // tile t, rows 8 y + 2 tq and + 1
        float s[NT][kStageTiles][4];
        float vs[kStageTiles];
#pragma unroll
        for (int t = 0; t < kStageTiles; ++t) {
          if (t > 0 && !two) {
#pragma unroll
            for (int y = 0; y < NT; ++y) s[y][t][0] = s[y][t][1] = s[y][t][2] = s[y][t][3] = -INFINITY;
            continue;
          }
          const float2 sc = scales[stage * kStageTiles + t];
          vs[t] = sc.y * kPDown;
          const unsigned char* kt = st + t * 2 * kTileCodes;
          float sa[NT][4], sb[NT][4];
#pragma unroll
          for (int y = 0; y < NT; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) sa[y][e] = sb[y][e] = 0.f;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const unsigned char* at = kt + (half ? koff1 : koff0);
            const uint4 r0 = *reinterpret_cast<const uint4*>(at);
            const uint4 r1 = *reinterpret_cast<const uint4*>(at + 1024);
            const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t a[4];
              halves_of<kE4m3>(w0[e], a[0], a[2]);
              halves_of<kE4m3>(w1[e], a[1], a[3]);
              const int ks = 4 * half + e;
#pragma unroll
              for (int y = 0; y < NT; ++y) {
                if (ks & 1) mma_f16_16816(sb[y], a, qb[y][ks][0], qb[y][ks][1]);
                else mma_f16_16816(sa[y], a, qb[y][ks][0], qb[y][ks][1]);
              }
            }
          }
#pragma unroll
          for (int y = 0; y < NT; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int at = g + 16 * t + (e >> 1) * 8;  // row of the stage
              const bool seen =
                  at < nvalid && (!kChunks || x * 16 + at < lim[y][e & 1]);
              s[y][t][e] = seen ? (sa[y][e] + sb[y][e]) * (qs[y][e & 1] * sc.x) : -INFINITY;
            }
        }

        // ---- online softmax, per row
        uint32_t pb[NT][kStageTiles][2];
#pragma unroll
        for (int y = 0; y < NT; ++y) {
          float mx0 = m[y][0], mx1 = m[y][1];
#pragma unroll
          for (int t = 0; t < kStageTiles; ++t) {
            mx0 = fmaxf(mx0, fmaxf(s[y][t][0], s[y][t][2]));
            mx1 = fmaxf(mx1, fmaxf(s[y][t][1], s[y][t][3]));
          }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(kFull, mx0, o));
            mx1 = fmaxf(mx1, __shfl_xor_sync(kFull, mx1, o));
          }
          if (mx0 > m[y][0] || mx1 > m[y][1]) {
            // (a maximum of -inf stays; 0 where it was that and no longer is)
            const float a0 = mx0 > m[y][0] ? fast_exp2(m[y][0] - mx0) : 1.f;
            const float a1 = mx1 > m[y][1] ? fast_exp2(m[y][1] - mx1) : 1.f;
            const uint64_t a2 = umma::f2_pack(__float_as_uint(a0), __float_as_uint(a1));
            l[y][0] *= a0;
            l[y][1] *= a1;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              acc[y][i][0] = umma::f2_mul(acc[y][i][0], a2);
              acc[y][i][1] = umma::f2_mul(acc[y][i][1], a2);
            }
            m[y][0] = mx0;
            m[y][1] = mx1;
          }
          // (chunks: a row may see nothing of a run's part of the pair)
          const float f0 = kChunks && m[y][0] == -INFINITY ? 0.f : m[y][0];
          const float f1 = kChunks && m[y][1] == -INFINITY ? 0.f : m[y][1];
#pragma unroll
          for (int t = 0; t < kStageTiles; ++t) {
            if (t > 0 && !two) break;
            const float p0 = fast_exp2(s[y][t][0] - f0), p2 = fast_exp2(s[y][t][2] - f0);
            const float p1 = fast_exp2(s[y][t][1] - f1), p3 = fast_exp2(s[y][t][3] - f1);
            l[y][0] += p0 + p2;
            l[y][1] += p1 + p3;
            // P^T as the B operand, rounded to fp16 once
            pb[y][t][0] = movmatrix_trans(probabilities_to_half2(p0, p1));  // tokens 0..7
            pb[y][t][1] = movmatrix_trans(probabilities_to_half2(p2, p3));  // tokens 8..15
          }
        }
        // ---- O^T += vs (V^T . P^T)
#pragma unroll
        for (int t = 0; t < kStageTiles; ++t) {
          if (t > 0 && !two) break;
          const uint64_t vs2 = umma::f2_pack(__float_as_uint(vs[t]), __float_as_uint(vs[t]));
          const uint32_t vaddr = smem_addr(st) + (2 * t + 1) * kTileCodes + vrow * 128;
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            uint32_t r[4];  // keys 0-7 and 8-15 of elements 16i .., then of 16(i + 1) ..
            ldmatrix_x4_trans(r, vaddr + (((i + vch) ^ (vrow & 7)) << 4));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t a[4];
              halves_across<kE4m3>(r[2 * k], a[0], a[1]);
              halves_across<kE4m3>(r[2 * k + 1], a[2], a[3]);
#pragma unroll
              for (int y = 0; y < NT; ++y) {
                float d[4];
                mma_f16_16816_zero(d, a, pb[y][t][0], pb[y][t][1]);
                acc[y][i + k][0] =
                    umma::f2_fma(umma::f2_pack(__float_as_uint(d[0]), __float_as_uint(d[1])), vs2,
                                 acc[y][i + k][0]);
                acc[y][i + k][1] =
                    umma::f2_fma(umma::f2_pack(__float_as_uint(d[2]), __float_as_uint(d[3])), vs2,
                                 acc[y][i + k][1]);
              }
            }
          }
        }
        __syncwarp();

        // ---- refill this stage with the next tiles of the run
        if (more) {
          fence_proxy_async_smem();
          issue(stage);
        }
      }
      if (dead) break;

      // ---- the pair's part in this run is done
#pragma unroll
      for (int y = 0; y < NT; ++y)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          l[y][0] += __shfl_xor_sync(kFull, l[y][0], o);
          l[y][1] += __shfl_xor_sync(kFull, l[y][1], o);
        }
      const bool whole = seg.x0 == seg.pstart && seg.x1 == seg.pend;
      const int last = seg.x0 != lo;  // a run's first piece, or (not first) its last
#pragma unroll
      for (int y = 0; y < NT; ++y)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 8 * y + 2 * tq + e;
          if (r >= rows) continue;
          if (whole) {
            const float inv = l[y][e] != 0.f ? 1.f / l[y][e] : 0.f;
            const int token = token_of(seg.seq) + (kChunks ? r / G : 0);
            uint16_t* row = p.out + (static_cast<int64_t>(token) * p.Hq + seg.kvh * G +
                                     (kChunks ? r % G : r)) * kHeadDim + 2 * g;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float x[2], z[2];
              umma::f2_unpack(acc[y][i][0], x[0], x[1]);
              umma::f2_unpack(acc[y][i][1], z[0], z[1]);
              *reinterpret_cast<uint32_t*>(row + 16 * i) = pack_bf16x2(x[e] * inv, z[e] * inv);
            }
          } else {
            float* rec = piece(warp, last, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float x[2], z[2];
              umma::f2_unpack(acc[y][i][0], x[0], x[1]);
              umma::f2_unpack(acc[y][i][1], z[0], z[1]);
              *reinterpret_cast<float2*>(rec + 16 * i + 2 * g) = make_float2(x[e], z[e]);
            }
            if (g == 0) {
              rec[128] = m[y][e];
              rec[129] = l[y][e];
            }
          }
        }
      if (!whole && lane == 0) piece_pair[2 * warp + last] = seg.seq * Hkv + seg.kvh;
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
  const int heads = kChunks ? p.group_tokens * G : G;  // rows of a pair at most
  const int tasks = __popc(starts) * heads;
  // (last group first: what a later CTA waits for goes out before a wait for earlier ones)
  for (int task = tasks - 1 - warp; task >= 0; task -= W) {
    const int grp = static_cast<uint32_t>(task) / static_cast<uint32_t>(heads);
    const int hh = task - grp * heads;
    uint32_t rest = starts;
    for (int k = 0; k < grp; ++k) rest &= rest - 1;
    const int n = __ffs(rest) - 1;  // pieces n .. end - 1 are this pair's (or empty)
    rest &= rest - 1;
    const int end = rest != 0u ? __ffs(rest) - 1 : 2 * W;
    const int pair = __shfl_sync(kFull, lane_pair, n);
    if (kChunks && hh >= rows_of(static_cast<uint32_t>(pair) / static_cast<uint32_t>(Hkv))) continue;
    // lane j < end - n derives the weight of piece n + j (2 W <= 32 lanes)
    const int k = n + lane;
    const bool have = k < end && (taken >> k & 1u);
    const float* rk = piece(k < end ? k >> 1 : 0, k & 1, hh);
    const float mj = have ? rk[128] : -INFINITY, lj = have ? rk[129] : 0.f;
    float M = mj;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
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
    const int token = token_of(sg.seq) + (kChunks ? hh / G : 0);
    const int qh = sg.kvh * G + (kChunks ? hh % G : hh);
    if (cf == cl) {
      tc_write_out(p, token, qh, lane, o4, Mr, Ls);
    } else if (cl != c) {
      tc_store_piece(p.rec + (static_cast<int64_t>(c) * kTcRecHeads + hh) * kRecStride, p.tag,
                     lane, o4, Mr, Ls);
    } else if (!tc_merge_earlier(p, token, qh, hh, cf, c, V, P, lane, o4, Mr, Ls) && lane == 0) {
      record_error(p.err, kErrTimeout);
    }
  }
}

namespace {

template <bool kContig, bool kE4m3, bool kChunks, int W, int S, int MH>
cudaError_t launch_shape(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeQ8Params& p0,
                         int num_ctas, cudaStream_t stream) {
  using L = Q8Smem<W, S, MH>;
  static unsigned long long done_mask = 0;
  auto kernel = decode_q8_kernel<kContig, kE4m3, kChunks, W, S, MH>;
  cudaError_t e = ensure_smem_limit(kernel, L::kTotal, &done_mask);
  if (e != cudaSuccess) return e;
  // (of chunks, whole ones: their groups are the schedule's sequences)
  const int groups = kChunks ? p0.groups : 1;
  const int chunk = tc_chunk_seqs(p0.max_context) / groups * groups;
  for (int s0 = 0; s0 < p0.num_seqs; s0 += chunk) {
    DecodeQ8Params p = p0;
    const int first = s0 / groups;  // sequence of the call
    p.num_seqs = (p0.num_seqs - s0) < chunk ? (p0.num_seqs - s0) : chunk;
    if (kChunks) {
      p.cu_q += first;
    } else {
      p.q += static_cast<int64_t>(s0) * p.Hq * kHeadDim;
      p.out += static_cast<int64_t>(s0) * p.Hq * kHeadDim;
    }
    p.ctx_lens += first;
    if (kContig) p.req_ids += first;
    else p.block_tables += static_cast<int64_t>(first) * p.max_blocks;
    p.tag = next_launch_tag();  // every launch writes its piece records under a fresh tag
    e = launch_pdl_if(pdl_decode_enabled(), kernel, dim3(num_ctas), dim3(W * 32), L::kTotal,
                      stream, tk, tv, p);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <bool kContig, bool kE4m3>
cudaError_t launch_heads(const CUtensorMap& tk, const CUtensorMap& tv, const DecodeQ8Params& p,
                         int num_ctas, cudaStream_t stream) {
  if (p.cu_q != nullptr)
    return launch_shape<kContig, kE4m3, true, 8, 2, 16>(tk, tv, p, num_ctas, stream);
  return p.G <= 4 ? launch_shape<kContig, kE4m3, false, 12, 2, 4>(tk, tv, p, num_ctas, stream)
                  : launch_shape<kContig, kE4m3, false, 10, 2, 8>(tk, tv, p, num_ctas, stream);
}

// Codes [rows][128] as a 2-D tensor; boxes of 16 rows, 128-byte swizzle.
bool encode_codes(CUtensorMap* map, const void* base, int64_t rows) {
  auto enc = tensor_map_encoder();
  if (enc == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kCodeRowBytes), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kCodeRowBytes)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kCodeRowBytes), 16u};
  const cuuint32_t estr[2] = {1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Tokens that 16 rows hold.
static int chunk_group_tokens(int G) { return 16 / G; }

// Chunks of one group of 16 rows; of two where they hold 1.5 groups' tokens on average
// at most (drafts of 2 to 8 tokens: the second group of the shorter ones is empty).
// More than 8 rows of few pairs spend their time in the join.  8 KV heads of 4 query
// heads, int8, us a call, this kernel / the tiles of prefill: 600 x 4 tokens after 200
// 111 / 182, 64 x 4 after 2000 73.6 / 106, 16 x 4 28.4 / 38.0, 4 x 4 20.5 / 21.0, 16 drafts
// 32.8 / 37.8; 64 x 8 (two full groups) 132 / 106; 1 x 2 16.9 / 19.5, 2 x 4 21.6 / 20.3,
// after 8000 27.7 / 24.3.
bool chunks_by_runs(int num_tokens, int num_seqs, int max_q, int Hkv, int G, int max_context) {
  const int group = chunk_group_tokens(G);
  const int groups = (max_q + group - 1) / group;
  if (groups > 1 && (groups > 2 || 2ll * num_tokens > 3ll * group * num_seqs)) return false;
  if (max_q * G > 8 && static_cast<int64_t>(num_seqs) * Hkv < 32) return false;
  return tc_chunk_seqs(max_context) >= groups;  // (a launch takes whole chunks)
}

TcStatus launch_decode_q8(const AttentionQ8Params& a, bool e4m3, bool contig, int num_ctas,
                          void* workspace, cudaStream_t stream, cudaError_t* cuda_err) {
  *cuda_err = cudaSuccess;
  const int64_t rows = a.num_blocks * a.Hkv * a.bs;
  alignas(64) CUtensorMap tk;
  alignas(64) CUtensorMap tv;
  if (!encode_codes(&tk, a.k_codes, rows) || !encode_codes(&tv, a.v_codes, rows))
    return TcStatus::kEncodeFailed;
  DecodeQ8Params p = {};
  p.q = a.q;
  p.out = a.out;
  p.ctx_lens = a.ctx_lens;
  p.block_tables = contig ? nullptr : a.tables;
  p.req_ids = contig ? a.tables : nullptr;
  p.rec = static_cast<uint64_t*>(workspace);
  p.seg_cost = 4;
  p.bs = a.bs;
  p.num_blocks = a.num_blocks;
  p.max_blocks = a.max_blocks;
  p.max_reqs = static_cast<int32_t>(a.num_blocks);
  p.num_seqs = a.num_seqs;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.G;
  p.max_context = a.max_context;
  p.qscale = a.qscale;
  p.checked = a.checked;
  p.err = a.err;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  if (a.cu_q != nullptr) {
    p.cu_q = a.cu_q;
    p.group_tokens = chunk_group_tokens(a.G);
    p.groups = (a.max_q + p.group_tokens - 1) / p.group_tokens;
    p.num_seqs = a.num_seqs * p.groups;
    p.max_q = a.max_q;
  }
  if (contig)
    *cuda_err = e4m3 ? launch_heads<true, true>(tk, tv, p, num_ctas, stream)
                     : launch_heads<true, false>(tk, tv, p, num_ctas, stream);
  else
    *cuda_err = e4m3 ? launch_heads<false, true>(tk, tv, p, num_ctas, stream)
                     : launch_heads<false, false>(tk, tv, p, num_ctas, stream);
  return *cuda_err == cudaSuccess ? TcStatus::kOk : TcStatus::kCudaError;
}

}  // namespace pkv
