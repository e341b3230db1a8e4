// prefill_scored.cu -- prefill attention with capped, biased and masked scores
// (score.cuh) over a paged KV cache, on the fifth-generation tensor cores.
//
// For row (token, query head) r of a chunk and the keys j it sees (one
// interval of positions lo .. hi): O_r = sum_j softmax_j(score(q_r . k_j)) v_j.
//
// Work items are those of the plain kernel (prefill.cu): two row tiles of 128
// rows (whole tokens of one KV head's group), one KV head, one sequence.  An
// item's key tiles start at the first position any of its rows sees (rounded
// down to a box), so a window's or a document's cost is its own.
//
// Schedule.  What an item costs depends on its masks and on its sequence's
// length, and in a ragged batch most (row tile, sequence) pairs have no rows.
// Up to kListMax pairs each CTA (one an SM) sorts them by key tiles, and the
// grid has one CTA an item: a running CTA takes the place of one that has not
// started (cluster launch control), so that the next heaviest item goes to
// whoever is free.  Longer lists, and those of one round, are dealt to one CTA
// an SM in rounds of alternating direction, latest rows first, which a ragged
// batch leaves uneven.  Rounds / on demand, 32 / 8 heads, capped: 15 chunks of
// 260 to 1040 tokens 97.8 / 84.9 us, 3 of 518 to 2072 82.4 / 59.8, 24 of 50 to
// 150 24.6 / 20.6; 6 chunks of 56 heads under every mask 117 / 103; even
// batches pay the sort: 8 x 2048 uncapped 247 / 250.
//
// Few items (a short chunk after a long context): a cluster of 2 to 16 CTAs
// shares an item's key tiles, as many as the device holds for all items at
// once, and joins its parts through distributed shared memory (join_parts).
// The join takes 5 us, a key tile 1.8 (one row tile) to 2.2 us: items of fewer
// than kJoinTiles are the first CTA's alone.  32 / 8 heads, one CTA / a cluster
// an item: 64 tokens after 8000 129 / 30 us, 512 after 8000 136 / 81, 2 x 256
// after 2000 to 4000 70 / 46, 4 x 1 after 996 21.1 / 13.9.  Kernels of their own:
// in one, the code of the join cost 2 x 8192 tokens 256 -> 262 us.
//
// Roles, tensor memory and the order of products are the plain kernel's:
//
//   warps 0-3  softmax and output of row tile 0   warps 4-7  of row tile 1
//   warp 8     the K/V tiles of 128 keys by TMA into a 2-stage ring
//   warp 9     tensor-memory owner and MMA issuer (one thread)
//   warp 10    the item list and the Q rows, by TMA into two rotating slots
//
// What bounds it, as the plain kernel, is the chain of a row tile's S, softmax,
// P and P V product (the two row tiles take turns on the tensor cores).  Tried
// and slower: two warps per 32 rows, each on half the keys (+3 %); P in shared
// memory, so that S is free once it is in registers (+15 %: each hand-over
// waits for the proxy fence, and both softmax warpgroups run in step).  32 / 8
// heads, 8 chunks of 2048: masks alone 254 us (1083 TFLOP/s), capped 273 (1007),
// with slopes 273, capped with slopes 335, any score 509; contiguous 2 x 8192
// under a window of 1024: 258 us (996 TFLOP/s).  The plain kernel takes 238 us for
// the first: what its softmax does not do (masks, the cap, the check of the output
// rows) is the rest, and two exposed loads of S a tile.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>

#include "cluster.cuh"
#include "pkv_device.cuh"
#include "prefill.cuh"
#include "prefill_scored.cuh"
#include "umma.cuh"

namespace pkv {

using namespace umma;

namespace {

constexpr int kStages = 2;
constexpr int kQSlots = 2;                            // Q tiles in rotation
constexpr int kOffK = kQSlots * kOpBytes;             // after the Q slots
constexpr int kStageBytes = 2 * kOpBytes;             // K then V
constexpr int kOffOut = kOffK + kStages * kStageBytes;  // output staging, 4 KiB per softmax warp
constexpr int kTilesBytes = kOffOut + 8 * 4096;       // 224 KiB
constexpr int kOffResponse = kTilesBytes + 480;       // 16 bytes, after barriers and item ring
constexpr int kOffList = kTilesBytes + 512;
constexpr int kListMax = 704;                         // sorted (row tile, sequence) pairs
constexpr int kListScan = 2816;                       // candidates looked through for them
constexpr int kSmemBytes = kOffList + kListMax * 2 + 1024;  // + alignment
static_assert(kSmemBytes <= 232448, "shared memory per CTA exceeds 227 KiB");
constexpr int kThreads = 352;
constexpr int kRingUsers = 10;                        // readers: softmax, K/V and MMA warps

// One work item as warp 10 publishes it; ntiles == 0 ends the list.  Its key
// tiles start at position k0 (a multiple of run_rows); no row of it sees a
// position before klo (INT_MAX: none sees any).
// With `joined` the item is a part of the cluster's: its O and sums stay for the join.
struct Item {
  int32_t seq, kvh, row0, rows, base, ntiles, q0, ctx, k0, klo, joined;
};

// Asks for a CTA of this grid that has not started: its index comes to `to`
// (16 bytes of shared memory, counted on bar) in its place, or a refusal.
__device__ __forceinline__ void take_block(void* to, uint64_t* bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], "
      "[%1];" ::"r"(smem_addr(to)),
      "r"(smem_addr(bar))
      : "memory");
}

// The answer: the CTA's blockIdx.x, or -1 (no further request may be made).
__device__ __forceinline__ int taken_block(const void* from) {
  int x = -1;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 r, [%1];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, r;\n\t}"
      : "+r"(x)
      : "r"(smem_addr(from))
      : "memory");
  return x;
}

// What a cluster's CTAs share of the item they have in parts: in the output
// staging, which a part does not use.
struct Join {
  float2 sums[2 * kRowTile];  // (m, l) of every row of this CTA's part
  Item item;                  // the whole item
};
constexpr int kOffJoin = kOffOut + 8192;  // (past the keys of the sort)
constexpr int kJoinTiles = 6;             // fewer key tiles are not split
static_assert(8192 >= (kListMax + 4) * 4 && kOffJoin + sizeof(Join) <= kTilesBytes, "join");

// Row `row` of an item.
__device__ __forceinline__ ScoredRow score_row(const PrefillParams& p, const Item& it, int row) {
  ScoredRow r;
  r.valid = true;
  const int tok = row / p.G;
  const int head = it.kvh * p.G + row - tok * p.G;
  const int pos = it.base + tok;
  r.qrow = (static_cast<int64_t>(it.q0) + tok) * p.Hq + head;
  int lo, hi;
  visible_keys(p.sp, pos, p.sp.first_key != nullptr ? __ldg(p.sp.first_key + it.q0 + tok) : 0,
               p.sp.prefix != nullptr ? __ldg(p.sp.prefix + it.seq) : 0, it.ctx, lo, hi);
  r.lo = lo <= hi ? lo - it.k0 : INT_MAX;
  r.hi = lo <= hi ? hi - it.k0 : -1;
  r.pos = pos - it.k0;
  r.slope2 = p.sp.slopes != nullptr ? slope_log2(p.sp.slopes, head) : 0.f;
  return r;
}

__device__ __forceinline__ KvRows kv_rows(const PrefillParams& p, const Item& it) {
  KvRows kv;
  kv.k = p.k;
  kv.v = p.v;
  kv.table = p.block_tables + static_cast<int64_t>(it.seq) * p.max_blocks;
  kv.bs = p.bs;
  kv.num_blocks = p.num_blocks;
  kv.Hkv = p.Hkv;
  kv.kvh = it.kvh;
  kv.checked = p.checked;
  kv.err = p.err;
  kv.err_code = p.err_code;
  return kv;
}

// Puts the rows of the warp right that are not finite, their output being on its way
// (repair_rows).  l: the row's sum of probabilities.  A row whose sum is NaN sees a
// NaN score, and is NaN by the formula.
__device__ __noinline__ void repair_item(const PrefillParams& p, const Item& it, float l,
                                         uint32_t o_tm) {
  const int lane = threadIdx.x & 31, lr = threadIdx.x & (kRowTile - 1);
  const int row = it.row0 + (threadIdx.x >> 7) * p.tile_rows + lr;
  const bool valid = lr < p.tile_rows && row < it.rows;
  const ScoredRow r = score_row(p, it, valid ? row : it.rows - 1);
  if (lane == 0) bulk_wait_done();  // the tensor stores of these rows come first
  __syncwarp();
  const Columns bad = bad_columns(o_tm);
  const bool flagged = valid && l == l && (bad.w[0] | bad.w[1] | bad.w[2] | bad.w[3]) != 0u;
  repair_rows(p, kv_rows(p, it), flagged, bad, r, it.k0, lane);
}

// Sums the CTAs' parts of rows rank, rank + kN, .. of an item: a warp a row, 16
// loads in flight.
template <int kN>
__device__ __forceinline__ void sum_rows(const PrefillParams& p, const Item& it, const Join& join,
                                         unsigned char* smem, int rank, int row_tiles) {
  constexpr int kRows = 16 / kN, kWarps = kThreads / 32, kShare = kRowTile / kN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i0 = warp; i0 < row_tiles * kShare; i0 += kWarps * kRows) {
    float4 x[kRows][kN];
    int row[kRows];  // of the item's rows, or -1
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int i = i0 + u * kWarps;
      const int t = i / kShare, lr = (i - t * kShare) * kN + rank;
      row[u] = it.row0 + t * p.tile_rows + lr;
      if (i >= row_tiles * kShare || lr >= p.tile_rows || row[u] >= it.rows) row[u] = -1;
      const unsigned char* at =
          smem + kOffK + (row[u] < 0 ? 0 : t * 65536 + lr * 512 + ((lane ^ (lr & 31)) << 4));
#pragma unroll
      for (int k = 0; k < kN; ++k)
        x[u][k] = row[u] < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : ld_cluster_f4(in_cta(at, k));
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (row[u] < 0) continue;
      float4 o = x[u][0];
#pragma unroll
      for (int k = 1; k < kN; ++k) {
        o.x += x[u][k].x;
        o.y += x[u][k].y;
        o.z += x[u][k].z;
        o.w += x[u][k].w;
      }
      const int tok = row[u] / p.G;
      const int64_t qrow =
          (static_cast<int64_t>(it.q0) + tok) * p.Hq + it.kvh * p.G + row[u] - tok * p.G;
      *reinterpret_cast<uint2*>(p.out + qrow * kHeadDim + 4 * lane) =
          make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
      const float z = 0.f * o.x + 0.f * o.y + 0.f * o.z + 0.f * o.w;  // 0, or NaN
      if (__any_sync(kFull, z != 0.f)) {
        // (a sum that is NaN: a NaN score that the row sees)
        const int i = i0 + u * kWarps, t = i / kShare;
        const float2* sums = &join.sums[t * kRowTile + (i - t * kShare) * kN + rank];
        const float l = lane < kN ? ld_cluster_f2(in_cta(sums, lane)).y : 0.f;
        if (__any_sync(kFull, l != l)) continue;
        Columns bad;
        bad.w[0] = __ballot_sync(kFull, !(fabsf(o.x) < INFINITY));
        bad.w[1] = __ballot_sync(kFull, !(fabsf(o.y) < INFINITY));
        bad.w[2] = __ballot_sync(kFull, !(fabsf(o.z) < INFINITY));
        bad.w[3] = __ballot_sync(kFull, !(fabsf(o.w) < INFINITY));
        const ScoredRow r = score_row(p, it, row[u]);
        __syncwarp();  // the row is written
        repair_rows(p, kv_rows(p, it), lane == 0, bad, r, it.k0, lane);
      }
    }
  }
}

// The parts of a cluster's item, joined through distributed shared memory:
//   O = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k.
// Every CTA scales its O into its K/V stages, idle by then, and sums its share
// of the rows over the CTAs (pushed to the CTA that sums them, 16 bytes a lane,
// the rows took 2 us longer).  Every CTA comes to each barrier whatever its
// item: what goes before them waits a bounded time.
static __device__ __noinline__ void join_parts(const PrefillParams& p, unsigned char* smem,
                                               uint32_t tmem, const ScoredBars& B,
                                               const Join& join, int rank) {
  constexpr int kMost = 16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int TR = p.tile_rows, n = p.split;
  __syncwarp();
  cluster_sync();
  const bool on = __all_sync(
      kFull, lane >= n || ld_cluster_s32(in_cta(&B.joined, lane < n ? lane : 0)) != 0);
  const Item it = join.item;
  const int row_tiles = it.rows > it.row0 + TR ? 2 : 1;
  if (on && warp < 4 * row_tiles) {
    tc_fence_after();
    const int t = warp >> 2, lr = tid & (kRowTile - 1);
    const uint32_t o_tm = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 256 + t * 128;
    const float2* at = &join.sums[t * kRowTile + lr];
    float2 x[kMost];
#pragma unroll
    for (int k = 0; k < kMost; ++k)
      x[k] = k < n ? ld_cluster_f2(in_cta(at, k)) : make_float2(-INFINITY, 0.f);
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int k = 0; k < kMost; ++k)
      if (x[k].y != 0.f) M = fmaxf(M, x[k].x);
#pragma unroll
    for (int k = 0; k < kMost; ++k)
      if (x[k].y != 0.f) L = fmaf(x[k].y, fast_exp2(x[k].x - M), L);
    const bool any = at->y != 0.f;  // (else O is 0 or was never written)
    const float w = any ? fast_exp2(at->x - M) / L : 0.f;
    unsigned char* to = smem + kOffK + t * 65536 + lr * 512;
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      uint32_t a[32], b[32];
      tmem_ld32(a, o_tm + 64 * h);
      tmem_ld32(b, o_tm + 64 * h + 32);
      tmem_wait_ld(a);
      tmem_ready(b);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t* o = i < 8 ? a + 4 * i : b + 4 * (i - 8);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (any)
          v = make_float4(__uint_as_float(o[0]) * w, __uint_as_float(o[1]) * w,
                          __uint_as_float(o[2]) * w, __uint_as_float(o[3]) * w);
        *reinterpret_cast<float4*>(to + (((16 * h + i) ^ lane) << 4)) = v;
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync();
  if (on) {
    if (n == 2) sum_rows<2>(p, it, join, smem, rank, row_tiles);
    else if (n == 4) sum_rows<4>(p, it, join, smem, rank, row_tiles);
    else if (n == 8) sum_rows<8>(p, it, join, smem, rank, row_tiles);
    else sum_rows<16>(p, it, join, smem, rank, row_tiles);
  }
  __syncwarp();
  cluster_sync();  // no CTA leaves while another reads its shared memory
}

// A Q tile's slot in the rotation and the phase of that slot's barriers.
struct QCursor {
  int slot;
  uint32_t phase;
  __device__ QCursor next(int nslots) const {
    QCursor c = *this;
    if (++c.slot == nslots) {
      c.slot = 0;
      c.phase ^= 1u;
    }
    return c;
  }
};

static_assert(sizeof(ScoredBars) <= 256 && 256 + kRing * sizeof(Item) <= 480,
              "barriers and item ring");

}  // namespace

// kMode: a PrefillMode.  kSplit: clusters of p.split CTAs, an item each.
template <int kMode, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_scored_kernel(const __grid_constant__ CUtensorMap tmk,
                          const __grid_constant__ CUtensorMap tmv,
                          const __grid_constant__ CUtensorMap tmq,
                          const __grid_constant__ CUtensorMap tmo,
                          const __grid_constant__ PrefillParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  ScoredBars& B = *reinterpret_cast<ScoredBars*>(smem + kTilesBytes);
  volatile int* abort = &B.abort;
  Item* ring = reinterpret_cast<Item*>(smem + kTilesBytes + 256);  // [kRing]

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int G = p.G;
  const int TR = p.tile_rows;  // rows of a row tile: whole tokens, (128 / G) G
  auto q_off = [](int slot) { return slot * kOpBytes; };

  grid_dependency_wait();
  grid_dependency_trigger();

  // Read descriptor n of the ring (every lane of the calling warp); false
  // when a wait gave up.  The warp's lane 0 then frees its claim on the slot.
  auto read_item = [&](int n, Item& it) -> bool {
    const int slot = n & (kRing - 1);
    if (!__all_sync(kFull, wait_role(&B.ifull[slot], (n / kRing) & 1, abort, p)))
      return false;
    it = ring[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&B.iempty[slot]);
    return true;
  };

  // The first key (from k0) of the j-th key tile an item takes.  With a bias the
  // last come first: the nearest keys set the running maximum, and O is not
  // rescaled at every tile on the way to them.
  auto tile_key = [](const Item& it, int j) -> int {
    constexpr bool kLastFirst = kMode == kPrefillBiased || kMode == kPrefillCappedBiased;
    return (kLastFirst ? it.ntiles - 1 - j : j) * kKeys;
  };
  // Rows and positions of row tile pair rt of a sequence; false where its rows
  // lie past the chunk or, checked, the sequence is left unwritten.
  const int R = (p.max_q * G + 2 * TR - 1) / (2 * TR);
  auto describe = [&](int rt, int seq, int kvh, Item& it) -> bool {
    it.seq = seq;
    it.kvh = kvh;
    it.q0 = p.cu_q[seq];
    const int Lq = p.cu_q[seq + 1] - it.q0;
    it.ctx = p.ctx_lens[seq];
    if (p.checked) {
      const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.bs;
      if (Lq < 0 || Lq > p.max_q || it.ctx < Lq || it.ctx > cap) {
        if (rt == 0 && kvh == 0) record_error(p.err, kErrContext);
        return false;
      }
    }
    it.rows = Lq * G;
    it.row0 = rt * 2 * TR;
    it.base = it.ctx - Lq;  // position of the chunk's first token
    // (before the first position: only when ctx < Lq, caught in checked mode)
    const int last = min(it.row0 + 2 * TR, it.rows) - 1;
    return it.row0 < it.rows && it.base + last / G + 1 > 0;
  };
  Join& join = *reinterpret_cast<Join*>(smem + kOffJoin);
  const int rank = kSplit ? static_cast<int>(cluster_rank()) : 0;
  if (kSplit) {
    if (tid < 2 * kRowTile) join.sums[tid] = make_float2(-INFINITY, 0.f);
    if (tid == 0) B.joined = 0;
  }
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + kOffOut);  // (before any output)
  uint16_t* list = reinterpret_cast<uint16_t*>(smem + kOffList);
  if (p.list) {
    for (int i = tid; i < kListMax + 4; i += kThreads) keys[i] = 0u;
    if (tid == 0) B.pairs = 0;
  }

  // Setup: barriers (warp 8) and the tensor memory (warp 9).
  if (warp == 8) {
    if (lane == 0) {
      for (int s = 0; s < 2; ++s) {
        mbar_init(&B.kfull[s], 1);
        mbar_init(&B.vfull[s], 1);
        mbar_init(&B.kempty[s], 1);
        mbar_init(&B.vempty[s], 1);
        mbar_init(&B.sfull[s], 1);
        mbar_init(&B.pfull[s], 4);   // one arrival per softmax warp
        mbar_init(&B.ofull[s], 1);
        mbar_init(&B.qfull[s], 32);  // every lane of the Q warp
        mbar_init(&B.qempty[s], 1);
      }
      for (int s = 0; s < kRing; ++s) {
        mbar_init(&B.ifull[s], 1);
        mbar_init(&B.iempty[s], kRingUsers);
      }
      mbar_init(&B.drain, 1);
      mbar_init(&B.taken, 1);
      *abort = 0;
      fence_barrier_init();
      prefetch_tensormap(&tmk);
      prefetch_tensormap(&tmv);
      prefetch_tensormap(&tmq);
      if (p.out_tma) prefetch_tensormap(&tmo);
    }
  } else if (warp == 10 && TR < kRowTile) {
    // rows TR .. 127 of every Q slot are padding that no copy writes: zero
    for (int slot = 0; slot < kQSlots; ++slot)
      for (int x = lane; x < (kRowTile - TR) * 16; x += 32)
        *reinterpret_cast<uint4*>(smem + q_off(slot) + q_chunk_offset(TR + (x >> 4), x & 15)) =
            make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  } else if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(&B.tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B.tmem;
  const uint32_t smem_base = smem_addr(smem);

  if (p.list) {
    // The (row tile, sequence) pairs that have rows, by descending key tiles
    // (of the first and last token's positions; ties: latest rows first): the
    // same list in every CTA.
    for (int c = tid; c < R * p.num_seqs; c += kThreads) {
      const int rt = c / p.num_seqs;
      Item it;
      if (!describe(rt, c - rt * p.num_seqs, 0, it)) continue;
      const int t0 = it.row0 / G, t1 = (min(it.row0 + 2 * TR, it.rows) - 1) / G;
      const int prefix = p.sp.prefix != nullptr ? p.sp.prefix[it.seq] : 0;
      const int* fk = p.sp.first_key != nullptr ? p.sp.first_key + it.q0 : nullptr;
      int lo, hi, lo1, hi1;
      visible_keys(p.sp, it.base + t0, fk ? fk[t0] : 0, prefix, it.ctx, lo, hi);
      visible_keys(p.sp, it.base + t1, fk ? fk[t1] : 0, prefix, it.ctx, lo1, hi1);
      const int tiles = hi1 >= lo ? min((hi1 - lo) / kKeys + 1, 65535) : 1;
      const int at = atomicAdd(&B.pairs, 1);
      if (at < kListMax) keys[at] = static_cast<uint32_t>(tiles) << 16 | static_cast<uint32_t>(c);
    }
    __syncthreads();
    const int n = min(B.pairs, kListMax);
    for (int i = tid; i < n; i += kThreads) {
      const uint32_t key = keys[i];
      int rank = 0;
      for (int j = 0; j < n; j += 4) {
        const uint4 k = *reinterpret_cast<const uint4*>(keys + j);
        rank += (k.x > key) + (k.y > key) + (k.z > key) + (k.w > key);
      }
      list[rank] = static_cast<uint16_t>(key);
    }
    __syncthreads();
  }

  if (warp == 8) {
    // ================= K/V producer =================
    // Every row tile of a sequence and KV head reads the same K/V tiles: keep
    // them in L2 for the items after.
    const uint64_t policy = l2_policy_evict_last();
    const int run = p.run_rows;    // rows per box (16 .. 128, divides 128 and bs)
    const int runs = kKeys / run;  // boxes per tile and tensor (<= 8)
    const int prun = lane & 15;    // lanes 0-15 copy K of run prun, lanes 16-31 V
    // block-table entry of run prun of tile j of `it` (-1: outside the visible positions or rejected)
    auto entry = [&](const Item& it, int j) -> int32_t {
      const int kpos = it.k0 + tile_key(it, j) + prun * run;
      int32_t e = -1;
      if (prun < runs && kpos < it.ctx && kpos + run > it.klo) {
        e = p.block_tables[static_cast<int64_t>(it.seq) * p.max_blocks + kpos / p.bs];
        if (p.checked && (e < 0 || e >= p.num_blocks)) {
          record_error(p.err, p.err_code);
          e = -1;  // skip the copy: stale rows, undefined output, no fault
        }
      }
      return e;
    };
    int g = 0;             // tiles (of all items) whose K and V were both issued
    bool kv_half = false;  // tile g has its K issued, not its V
    int nread = 0;
    Item cur;
    bool ok = read_item(nread++, cur);
    int32_t e = ok && cur.ntiles > 0 ? entry(cur, 0) : -1;  // entries of the next tile to issue
    while (ok && cur.ntiles > 0) {
      Item nx = cur;
      for (int j = 0; j < cur.ntiles; ++j) {
        const int s = g & 1;
        const uint32_t loaded = __popc(__ballot_sync(kFull, lane < 16 && e >= 0));
        const int off = (cur.k0 + tile_key(cur, j) + prun * run) % p.bs;
        const int32_t grp =
            e >= 0 ? static_cast<int32_t>(cache_row(e, cur.kvh, p.Hkv, p.bs, off) >> 3) : 0;
        unsigned char* dst = smem + kOffK + s * kStageBytes + prun * run * kRowBytes;
        // K first: its stage frees once both S products of tile g - 2 are done
        if (g >= kStages && !__all_sync(kFull, wait_role(&B.kempty[s], ((g >> 1) - 1) & 1, abort, p))) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&B.kfull[s], loaded * run * kRowBytes);
        __syncwarp();
        if (lane < 16 && e >= 0) tma_load_4d(dst, &tmk, grp, &B.kfull[s], policy);
        // then V, whose stage frees after both P V products of tile g - 2
        if (g >= kStages && !__all_sync(kFull, wait_role(&B.vempty[s], ((g >> 1) - 1) & 1, abort, p))) {
          kv_half = true;
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&B.vfull[s], loaded * run * kRowBytes);
        __syncwarp();
        if (lane >= 16 && e >= 0) tma_load_4d(dst + kOpBytes, &tmv, grp, &B.vfull[s], policy);
        ++g;
        // the next tile's entries load while this one lands
        if (j + 1 < cur.ntiles) {
          e = entry(cur, j + 1);
        } else {
          ok = read_item(nread++, nx);
          e = ok && nx.ntiles > 0 ? entry(nx, 0) : -1;
        }
      }
      cur = nx;
    }
    if (*abort && lane == 0) {
      // let the copies in flight land before the CTA's shared memory is released
      for (int j = max(0, g - kStages); j < g; ++j) {
        mbar_wait_bounded(&B.kfull[j & 1], (j >> 1) & 1);
        mbar_wait_bounded(&B.vfull[j & 1], (j >> 1) & 1);
      }
      if (kv_half) mbar_wait_bounded(&B.kfull[g & 1], (g >> 1) & 1);
    }
  } else if (warp == 10) {
    // ================= item list and Q rows =================
    // Q tile n (row tile 0 of an item, then row tile 1 if it has rows) goes to
    // slot n % 2 once the last S product reading tile n - 2 completed.
    const uint64_t qpolicy = l2_policy_evict_first();  // every Q row is read once
    int published = 0;
    uint32_t nq = 0;      // Q tiles loaded
    QCursor qc = {0, 0};  // slot of Q tile nq and its phase
    uint32_t last_phase = 0;  // bit s: phase of the last load into slot s
    bool ok = true;
    auto publish = [&](const Item& it) -> bool {
      const int slot = published & (kRing - 1);
      if (published >= kRing &&
          !__all_sync(kFull, wait_role(&B.iempty[slot], ((published / kRing) - 1) & 1, abort, p)))
        return false;
      if (lane == 0) {
        ring[slot] = it;
        mbar_arrive(&B.ifull[slot]);
      }
      __syncwarp();
      ++published;
      return true;
    };
    // Publishes an item and brings its Q rows; false when a wait gave up.
    auto serve = [&](Item it) -> bool {
      const int last_row = min(it.row0 + 2 * TR, it.rows) - 1;
      // the interval of positions that some token of the item sees
      const int prefix = p.sp.prefix != nullptr ? p.sp.prefix[it.seq] : 0;
      int low = INT_MAX, high = -1;
      for (int tok = it.row0 / G + lane; tok <= last_row / G; tok += 32) {
        int lo, hi;
        visible_keys(p.sp, it.base + tok,
                     p.sp.first_key != nullptr ? p.sp.first_key[it.q0 + tok] : 0, prefix,
                     it.ctx, lo, hi);
        if (lo <= hi) {
          low = min(low, lo);
          high = max(high, hi);
        }
      }
      it.klo = __reduce_min_sync(kFull, low);
      int kend = __reduce_max_sync(kFull, high) + 1;
      it.k0 = it.klo < kend ? it.klo / p.run_rows * p.run_rows : 0;
      kend = max(kend - it.k0, 1);  // an item that sees nothing is one tile, all masked
      it.ntiles = (kend + kKeys - 1) / kKeys;
      if (kSplit) {
        it.joined = it.ntiles >= kJoinTiles;
        if (it.joined) {
          if (lane == 0) {
            join.item = it;
            B.joined = 1;
          }
          __syncwarp();
          const int from = it.ntiles * rank / p.split;
          it.ntiles = it.ntiles * (rank + 1) / p.split - from;
          it.k0 += from * kKeys;
        } else if (rank > 0) {
          it.ntiles = 0;
        }
        if (it.ntiles == 0) return true;
      }
      if (!publish(it)) return false;
      const int nt = it.rows > it.row0 + TR ? 2 : 1;
      for (int t = 0; t < nt; ++t, ++nq, qc = qc.next(kQSlots)) {
        const int qs = qc.slot;
        if (nq >= static_cast<uint32_t>(kQSlots) &&
            !__all_sync(kFull, wait_role(&B.qempty[qs], qc.phase ^ 1u, abort, p)))
          return false;
        last_phase = (last_phase & ~(1u << qs)) | (qc.phase << qs);
        unsigned char* dst = smem + q_off(qs);
        // the tile is TR / G whole tokens, each column half one box of
        // (tokens, G heads, 64 columns); rows past the chunk bring the next
        // tokens' rows (or zeros past the tensor) and are never written out
        const int tok0 = it.q0 + (it.row0 + t * TR) / G;
        if (lane == 0) {
          // two column halves of TR rows x 128 bytes
          mbar_arrive_expect_tx(&B.qfull[qs], static_cast<uint32_t>(TR) * kRowBytes);
          tma_load_4d_at(dst, &tmq, 0, 0, it.kvh * G, tok0, &B.qfull[qs], qpolicy);
          tma_load_4d_at(dst + kHalfBytes, &tmq, 0, 1, it.kvh * G, tok0, &B.qfull[qs], qpolicy);
        } else {
          mbar_arrive(&B.qfull[qs]);
        }
      }
      return true;
    };
    if (p.list || kSplit) {
      // Item i is KV head i % Hkv of pair i / Hkv of the list, and CTA i's own
      // until another takes it.  A CTA takes its next item when it starts one
      // (the K/V producer runs ahead into it): heaviest first, to whoever is
      // there next.  (A cluster has one item.)
      uint32_t phase = 0;
      const int n = p.list ? min(B.pairs, kListMax) : R * p.num_seqs;
      for (int i = kSplit ? blockIdx.x / p.split : blockIdx.x; i >= 0;) {
        const int at = i / p.Hkv;
        if (at < n) {
          const int c = p.list ? list[at] : at, rt = c / p.num_seqs;
          Item it = {};
          ok = !describe(rt, c - rt * p.num_seqs, i - at * p.Hkv, it) || serve(it);
          if (!ok) break;
        }
        if (kSplit) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&B.taken, 16);
          take_block(smem + kOffResponse, &B.taken);
        }
        __syncwarp();
        if (!__all_sync(kFull, mbar_wait_bounded(&B.taken, phase))) {
          if (lane == 0) {
            *abort = 1;
            record_error(p.err, kErrTimeout);
          }
          ok = false;
          break;
        }
        phase ^= 1u;
        i = taken_block(smem + kOffResponse);
        fence_proxy_async_smem();  // read before the next answer comes in
        __syncwarp();
      }
    } else {
      // Items in order of index: row tile (latest first), then sequence, then
      // KV head.  Round k deals items k P .. k P + P - 1 to the P CTAs,
      // forwards in even rounds and backwards in odd ones; 32 rounds at a time,
      // one a lane, so that items whose rows lie past their chunk cost one latency.
      const int P = gridDim.x;
      const int per = p.num_seqs * p.Hkv;
      const int total = R * per;
      for (int64_t k0 = 0; ok && k0 * P < total; k0 += 32) {
        const int64_t k = k0 + lane;
        const int64_t slot = k * P + ((k & 1) ? P - 1 - static_cast<int>(blockIdx.x)
                                              : static_cast<int>(blockIdx.x));
        Item mine = {};
        bool there = slot < total;
        if (there) {
          const int idx = static_cast<int>(slot);
          const int rem = idx - (idx / per) * per;
          const int seq = rem / p.Hkv;
          there = describe(R - 1 - idx / per, seq, rem - seq * p.Hkv, mine);
        }
        for (uint32_t left = __ballot_sync(kFull, there); ok && left != 0u; left &= left - 1) {
          const int src = __ffs(left) - 1;
          Item it;
          it.seq = __shfl_sync(kFull, mine.seq, src);
          it.kvh = __shfl_sync(kFull, mine.kvh, src);
          it.q0 = __shfl_sync(kFull, mine.q0, src);
          it.ctx = __shfl_sync(kFull, mine.ctx, src);
          it.rows = __shfl_sync(kFull, mine.rows, src);
          it.row0 = __shfl_sync(kFull, mine.row0, src);
          it.base = __shfl_sync(kFull, mine.base, src);
          ok = serve(it);
        }
      }
    }
    if (ok) {
      Item end = {};  // ntiles 0: the end of this CTA's list
      publish(end);
    }
    if (*abort && lane == 0) {
      // let the Q copies in flight land before the shared memory is released
      for (int qs = 0; qs < kQSlots && static_cast<uint32_t>(qs) < nq; ++qs)
        mbar_wait_bounded(&B.qfull[qs], (last_phase >> qs) & 1u);
    }
  } else if (warp == 9) {
    // ================= MMA issuer: lane 0 alone =================
    // One thread issues every product, waits on single-lane barrier checks
    // and never votes or reconverges with the other lanes inside the loop.
    if (lane == 0) {
    auto issue_s = [&](int t, int qs, int stage) {  // S_t = Q K^T
      const uint32_t q_addr = smem_base + q_off(qs);
      const uint32_t k_addr = smem_base + kOffK + stage * kStageBytes;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t koff = (kk & 3) * 32;
        umma_ss(tmem + t * 128, smem_desc(q_addr + (kk >> 2) * kHalfBytes + koff, 16, 1024),
                smem_desc(k_addr + (kk >> 2) * 1024 + koff, 16, 2048), kIdescS, kk > 0);
      }
    };
    auto issue_pv = [&](int t, int stage, bool acc) {  // O_t (+)= P_t V
      const uint32_t v_addr = smem_base + kOffK + stage * kStageBytes + kOpBytes;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        umma_ts(tmem + 256 + t * 128, tmem + t * 128 + kk * 8,
                smem_desc(v_addr + kk * 4096, 1024, 2048), kIdescPV, (acc || kk > 0));
    };
    auto waitb = [&](uint64_t* b, uint32_t parity) -> bool {
      return wait_role(b, parity, abort, p);
    };
    auto read_item1 = [&](int n, Item& it) -> bool {
      const int slot = n & (kRing - 1);
      if (!wait_role(&B.ifull[slot], (n / kRing) & 1, abort, p)) return false;
      it = ring[slot];
      mbar_arrive(&B.iempty[slot]);
      return true;
    };
    auto has_two = [TR](const Item& it) { return it.rows > it.row0 + TR; };
    // S products of an item's first tile, global tile g, its Q tiles at qa, qb
    auto first_s = [&](const Item& it, QCursor qa, QCursor qb, int g) -> bool {
      if (!waitb(&B.kfull[g & 1], (g >> 1) & 1) || !waitb(&B.qfull[qa.slot], qa.phase))
        return false;
      tc_fence_after();
      {
        issue_s(0, qa.slot, g & 1);
        umma_commit(&B.sfull[0]);
        if (it.ntiles == 1) umma_commit(&B.qempty[qa.slot]);
      }
      if (has_two(it)) {
        if (!waitb(&B.qfull[qb.slot], qb.phase)) return false;
        tc_fence_after();
        {
          issue_s(1, qb.slot, g & 1);
          umma_commit(&B.sfull[1]);
          if (it.ntiles == 1) umma_commit(&B.qempty[qb.slot]);
        }
      }
      umma_commit(&B.kempty[g & 1]);  // both S products of tile g issued
      return true;
    };
    int nread = 0;
    Item cur;
    bool ok = read_item1(nread++, cur);
    QCursor q0 = {0, 0};        // cur's Q tiles: row tile 0 at q0, row tile 1 at q1
    QCursor q1 = q0.next(kQSlots);
    int g = 0;                  // tile index over all items (ring stage g & 1)
    uint32_t np0 = 0, np1 = 0;  // P hand-overs taken per row tile
    if (ok && cur.ntiles > 0) ok = first_s(cur, q0, q1, g);
    // Tile g, (cur, j): within an item PV_0(j) S_0(j+1) | PV_1(j) S_1(j+1);
    // at an item's last tile both P V products go first, then the next
    // item's first S products, so the current item never waits on the next.
    int j = 0;
    while (ok && cur.ntiles > 0) {
      const int s = g & 1;
      const bool two = has_two(cur);
      const bool last = j == cur.ntiles - 1;
      const bool qlast = j + 1 == cur.ntiles - 1;  // S of tile j + 1 reads cur's Q last
      ok = waitb(&B.vfull[s], (g >> 1) & 1);
      if (!ok) break;
      ok = waitb(&B.pfull[0], np0 & 1);
      ++np0;
      if (ok && !last) ok = waitb(&B.kfull[s ^ 1], ((g + 1) >> 1) & 1);
      if (!ok) break;
      tc_fence_after();
      {
        issue_pv(0, s, j > 0);
        if (last) umma_commit(&B.ofull[0]);
        if (!two) umma_commit(&B.vempty[s]);
        if (!last) {
          issue_s(0, q0.slot, s ^ 1);
          umma_commit(&B.sfull[0]);
          if (qlast) umma_commit(&B.qempty[q0.slot]);
          if (!two) umma_commit(&B.kempty[s ^ 1]);
        }
      }
      if (two) {
        ok = waitb(&B.pfull[1], np1 & 1);
        ++np1;
        if (!ok) break;
        tc_fence_after();
        {
          issue_pv(1, s, j > 0);
          if (last) umma_commit(&B.ofull[1]);
          umma_commit(&B.vempty[s]);  // the producer reuses the stage
          if (!last) {
            issue_s(1, q1.slot, s ^ 1);
            umma_commit(&B.sfull[1]);
            if (qlast) umma_commit(&B.qempty[q1.slot]);
            umma_commit(&B.kempty[s ^ 1]);
          }
        }
      }
      ++g;
      if (last) {
        Item nx;
        ok = read_item1(nread++, nx);
        if (!ok) break;
        q0 = two ? q1.next(kQSlots) : q1;  // the next item's Q tiles follow cur's
        q1 = q0.next(kQSlots);
        cur = nx;
        j = 0;
        if (cur.ntiles > 0) ok = first_s(cur, q0, q1, g);
      } else {
        ++j;
      }
    }
      // every MMA issued has completed before the tensor memory is released
      umma_commit(&B.drain);
      mbar_wait_bounded(&B.drain, 0);
    }
    __syncwarp();
  } else {
    // ================= scored softmax (prefill_scored.cuh) =================
    const int t = warp >> 2;                      // row tile
    const int lr = tid & (kRowTile - 1);          // row in the tile = tensor-memory lane
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + t * 128;
    const uint32_t o_tm = tmem + lane_base + 256 + t * 128;
    // descriptor n stays in the ring until this warp is done with it
    auto wait_item = [&](int n) -> bool {
      return __all_sync(kFull, wait_role(&B.ifull[n & (kRing - 1)], (n / kRing) & 1, abort, p));
    };
    auto has_rows = [&](const Item& it) { return t == 0 || it.rows > it.row0 + TR; };
    auto row_of = [&](const Item& it) -> ScoredRow {
      const int row = it.row0 + t * TR + lr;  // row of the chunk
      const bool valid = lr < TR && row < it.rows;
      ScoredRow r = score_row(p, it, valid ? row : it.rows - 1);  // padding mirrors the last row
      r.valid = valid;
      return r;
    };
    uint32_t ns = 0, no = 0;  // S tiles and items this row tile took
    const CappedRegs cap_regs = capped_regs<kMode>(p);
    bool ok = wait_item(0);
    ScoredRow row;
    if (ok && ring[0].ntiles != 0) row = row_of(ring[0]);
    for (int n = 0; ok; ++n) {
      const Item& it = ring[n & (kRing - 1)];
      if (it.ntiles == 0) break;
      const bool mine = has_rows(it);
      SoftState st = {-INFINITY, 0.f};
      for (int j = 0; mine && j < it.ntiles; ++j) {
        ok = __all_sync(kFull, wait_role(&B.sfull[t], ns & 1, abort, p));
        ++ns;
        if (!ok) break;
        tc_fence_after();
        scored_tile<kMode>(p, cap_regs, row, s_tm, o_tm, tile_key(it, j), j == 0, st);
        // V rows that no row sees (stale or foreign bytes) must not meet a
        // zero probability: zeroed once the tile has landed, before P is
        // handed over
        const int k0 = it.k0 + tile_key(it, j);
        if (t == 0 && (it.klo > k0 || it.ctx < k0 + kKeys)) {
          const int z0 = it.klo > k0 ? min(it.klo - k0, kKeys) : 0;
          const int z1 = max(min(it.ctx - k0, kKeys), z0);
          const uint32_t g = ns - 1;  // row tile 0 takes every key tile
          ok = __all_sync(kFull, wait_role(&B.vfull[g & 1], (g >> 1) & 1, abort, p));
          if (!ok) break;
          unsigned char* vt = smem + kOffK + (g & 1) * kStageBytes + kOpBytes;
#pragma unroll 1
          for (int idx = lr; idx < (z0 + kKeys - z1) * 16; idx += kRowTile) {
            const int r = idx >> 4;
            *reinterpret_cast<uint4*>(vt + kv_chunk_offset(r < z0 ? r : z1 + r - z0, idx & 15)) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.pfull[t]);
      }
      if (!ok) break;
      // the next item's row: its loads land while this item's last product runs
      ok = wait_item(n + 1);
      if (!ok) break;
      ScoredRow next_row = row;
      if (ring[(n + 1) & (kRing - 1)].ntiles != 0) next_row = row_of(ring[(n + 1) & (kRing - 1)]);
      if (kSplit && mine && it.joined) {
        ok = __all_sync(kFull, wait_role(&B.ofull[t], no & 1, abort, p));
        ++no;
        if (!ok) break;
        // (under a fixed offset every part has the same)
        join.sums[t * kRowTile + lr] = make_float2(kMode == kPrefillCapped ? 0.f : st.m, st.l);
      } else if (mine) {
        // the item's output rows; the next item's first P V product overwrites
        // O_t only after these warps hand over its first P
        ok = __all_sync(kFull, wait_role(&B.ofull[t], no & 1, abort, p));
        ++no;
        if (!ok) break;
        tc_fence_after();
        const float inv = st.l > 0.f ? 1.f / st.l : 0.f;
        const int wrow0 = it.row0 + t * TR + 32 * (warp & 3);  // this warp's first row
        // G divides 32 and every row of the warp is in the chunk: its 32 rows
        // are 32 / G whole tokens, stored by tensor stores
        const bool whole = p.out_tma && 32 * (warp & 3) + 32 <= TR && wrow0 + 32 <= it.rows;
        unsigned char* stg = smem + kOffOut + warp * 4096;
        // (the row's place again: not kept in registers through the tiles)
        const int own = it.row0 + t * TR + lr;
        const bool valid = lr < TR && own < it.rows;
        const int tok = own / G;
        uint4* dst = reinterpret_cast<uint4*>(
            p.out + ((static_cast<int64_t>(it.q0) + tok) * p.Hq + it.kvh * G + own - tok * G) * kHeadDim);
        uint64_t z = 0ull;  // (0, 0) while every element is finite
        // (a loop: this code runs once an item, out of a cold instruction cache)
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t a[32], b[32];
          tmem_ld32(a, o_tm + 64 * h);
          tmem_ld32(b, o_tm + 64 * h + 32);
          tmem_wait_ld(a);
          tmem_ready(b);
          add_finite(z, a);
          add_finite(z, b);
          if (whole) store_half_tma(&tmo, stg, lane, inv, a, b, h, it.kvh * G, it.q0 + wrow0 / G);
          else if (valid) store_half(dst + 8 * h, inv, a, b, p.out_v8);
        }
        // A row that is not finite may have met a NaN or an infinity that it does
        // not see (0 times either is NaN): repair_rows.  (One whose sum is NaN
        // sees a NaN score, and is NaN by the formula.)
        const bool repair = valid && !is_zero(z) && st.l == st.l;
        if (__any_sync(kFull, repair)) repair_item(p, it, st.l, o_tm);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.iempty[n & (kRing - 1)]);
      row = next_row;
    }
    if (lane == 0) bulk_wait_done();  // the warp's tensor stores completed
  }

  tc_fence_before();
  __syncthreads();
  if (kSplit) join_parts(p, smem, tmem, B, join, rank);
  if (warp == 9) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

namespace {

// One CTA per SM (the shared memory admits no second): SMs of a device, and
// clusters of 2, 4, 8 and 16 CTAs that it holds at once.
struct Room {
  std::atomic<int> sms;
  int clusters[4];
};

template <int kMode>
cudaError_t launch_mode(const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tq,
                        const CUtensorMap& to, const PrefillParams& p, cudaStream_t stream) {
  if (p.tile_rows <= 0 || p.tile_rows > kRowTile || p.tile_rows % p.G != 0)
    return cudaErrorInvalidValue;
  auto kernel = prefill_scored_kernel<kMode, false>, split = prefill_scored_kernel<kMode, true>;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  cfg.attrs = attr;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;

  static Room rooms[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64) return cudaErrorInvalidDevice;
  Room& room = rooms[dev];
  if (room.sms.load(std::memory_order_acquire) == 0) {
    static std::mutex once;
    std::lock_guard<std::mutex> lock(once);
    if (room.sms.load() == 0) {
      int n = 0;
      for (auto f : {kernel, split})
        if (e == cudaSuccess)
          e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(split, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return e;
      for (int i = 0; i < 4; ++i) {
        attr[0].val.clusterDim.x = 2u << i;
        cfg.gridDim = dim3(2u << i);
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&room.clusters[i], split, &cfg) != cudaSuccess) {
          room.clusters[i] = 0;  // no clusters of this size
          cudaGetLastError();
        }
      }
      room.sms.store(n, std::memory_order_release);
    }
  }
  const int n = room.sms.load(std::memory_order_acquire);

  const int64_t row_tiles =
      (static_cast<int64_t>(p.max_q) * p.G + 2 * p.tile_rows - 1) / (2 * p.tile_rows);
  const int64_t items = row_tiles * p.Hkv * p.num_seqs;
  if (items <= 0) return cudaSuccess;
  if (items > INT32_MAX) return cudaErrorInvalidValue;
  const int64_t bound = static_cast<int64_t>(p.num_tokens) * p.G / (2 * p.tile_rows) + p.num_seqs;
  const int64_t pairs = bound < row_tiles * p.num_seqs ? bound : row_tiles * p.num_seqs;
  const bool listable = pairs <= kListMax && row_tiles * p.num_seqs <= kListScan;
  PrefillParams pl = p;
  pl.split = 1;
  // Waits outlast rows computed again: 32 a warp, one after another, at 4 positions in
  // 0.8 us (6.4 us a position: 50000 of them 0.32 s), after a look through V (16
  // positions in 1 us).  A role may wait for two such items in a row; the limit allows
  // for 2.5 times that.
  pl.wait_ns = kWaitLimitNs + 32768ull * static_cast<unsigned long long>(p.max_blocks) * p.bs;
  // few items: the largest cluster an item that the device holds for all of them
  // at once, and whose parts the key tiles (at most) are enough for
  int64_t span = static_cast<int64_t>(p.max_blocks) * p.bs;
  if (p.sp.window > 0) span = std::min<int64_t>(span, int64_t{p.sp.window} + 2 * p.tile_rows / p.G);
  const int64_t most = span / kKeys + 1;
  for (int i = 3; i >= 0 && pl.split == 1; --i)
    if ((listable ? pairs * p.Hkv : items) <= room.clusters[i] && most >= kJoinTiles &&
        most > (1 << i))
      pl.split = 2 << i;
  int64_t grid;
  if (pl.split > 1) {
    pl.list = listable && items > room.clusters[__builtin_ctz(pl.split) - 1];
    grid = (pl.list ? pairs * p.Hkv : items) * pl.split;
  } else {
    // on demand over a grid of one CTA an item, or in rounds over one CTA an SM
    pl.list = listable && pairs * p.Hkv > n;
    grid = pl.list ? pairs * p.Hkv : std::min<int64_t>(items, n);
  }
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  int attrs = 0;
  if (pl.split > 1) attr[attrs++].val.clusterDim.x = static_cast<unsigned>(pl.split);
  if (pdl_enabled()) {
    attr[attrs] = {};
    attr[attrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[attrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.numAttrs = static_cast<unsigned>(attrs);
  return cudaLaunchKernelEx(&cfg, pl.split > 1 ? split : kernel, tk, tv, tq, to, pl);
}

}  // namespace

namespace {

uint64_t pair_of(float x) {
  uint32_t b;
  std::memcpy(&b, &x, sizeof b);
  return (static_cast<uint64_t>(b) << 32) | b;
}

// The polynomial of a cap, where a raw product at the cap (cap / scale) has an
// eighth power that neither overflows nor underflows in fp32 (else s_max is
// negative: no product is in range).  Returns whether the capped kernels serve
// the cap: one whose range fits the fixed offset.
bool capped_constants(const PrefillParams& p, CappedScore* c) {
  const ScoreParams& sp = p.sp;
  std::memset(c, 0, sizeof *c);
  if (!(sp.cap2 > 0.f)) return false;
  const float r = p.qscale * sp.inv_cap2;  // a raw product's share of the cap
  const bool poly = std::fabs(r) >= 1.220703125e-4f && std::fabs(r) <= 8192.f;  // 2^-13 .. 2^13
  const float fit[5] = {0.99999309f, -0.33298065f, 0.13036811f, -0.04481755f, 0.00903642f};
  float power = p.qscale;
  for (int i = 0; poly && i < 5; ++i) {
    c->c[i] = pair_of(fit[i] * power);
    power *= r * r;
  }
  c->s_max = poly ? std::fabs(1.f / r) : -1.f;
  if (!poly || sp.cap2 > 75.f) return false;
  // the offset m: the lowest score (-cap) keeps 2^-100
  const float m = sp.cap2 <= 50.f ? sp.cap2 : 100.f - sp.cap2;
  c->neg_m2 = pair_of(-m);
  // P at +cap; 2^18 (64 scores, 2^-12) times P at -cap
  const float edge = 0.76159416f * sp.cap2;  // tanh(1)
  c->p_high = std::exp2(edge - m);
  c->p_low = std::exp2(18.f - edge - m);
  c->exp_k = p.qscale * sp.cap_k;
  c->neg_2cap = -2.f * sp.cap2;
  c->cap_m = sp.cap2 - m;
  return true;
}

}  // namespace

cudaError_t launch_prefill_scored(const CUtensorMap& tk, const CUtensorMap& tv,
                                  const CUtensorMap& tq, const CUtensorMap& to,
                                  const PrefillParams& p_in, cudaStream_t stream) {
  PrefillParams p = p_in;
  // (a negative scale: the largest product is the lowest score, any-score kernel)
  if (p.sp.cap2 == 0.f && p.qscale >= 0.f)
    return p.sp.slopes == nullptr ? launch_mode<kPrefillMasked>(tk, tv, tq, to, p, stream)
                                  : launch_mode<kPrefillBiased>(tk, tv, tq, to, p, stream);
  if (capped_constants(p, &p.cap))
    return p.sp.slopes == nullptr
               ? launch_mode<kPrefillCapped>(tk, tv, tq, to, p, stream)
               : launch_mode<kPrefillCappedBiased>(tk, tv, tq, to, p, stream);
  return launch_mode<kPrefillGeneral>(tk, tv, tq, to, p, stream);
}

}  // namespace pkv
