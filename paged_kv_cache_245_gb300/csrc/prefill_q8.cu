// prefill_q8.cu -- causal prefill attention over the 8-bit KV cache (q8.cuh) on the
// fifth-generation tensor cores.
//
// Work items, tensor memory and the order of products are those of the plain
// kernel (prefill.cu): two row tiles of 128 (token, query head) rows of one KV head
// and sequence, key tiles of 128 positions, S_t and O_t in tensor memory.  What is
// added turns codes into operands:
//
//   warps 0-3    softmax and output of row tile 0   warps 4-7  of row tile 1
//   warp 8       tensor-memory owner and MMA issuer
//   warp 9       the item list and the Q rows
//   warp 10      codes of K and V (16 KiB a tile each) by bulk copies into one slot
//                each, and the tile's 16 scales by cp.async
//   warps 12-19  codes -> bf16 into the two stages of K and V operands
//
// The operands hold the codes themselves, which bf16 holds exactly (int8 and e4m3
// have at most 8 significant bits): a key's scale is uniform over 16 columns of S
// and enters the softmax's own multiplication, and a value's enters the exponent,
// so that P is rounded to bf16 with it -- the one rounding that the plain kernel has
// too, and bf16's range holds any scale.  With ks, vs the scales of key j's group:
//   s_j = (q . kcode_j) (scale ks),  P_j vs = 2^(s_j log2 e - m + log2 vs),
//   O += (P_j vs) vcode_j,           l += (sum over a group of P_j vs) / vs.
//
// Schedule.  Many items: dealt to the CTAs (one an SM) in rounds of alternating
// direction, sorted by cost where the list is short enough for each CTA to sort, else
// latest rows first.  Few items (a host bound of kSplitItems an SM): the
// flattened list of all items' key tiles is cut evenly over the CTAs, an item
// counting as kItemCost tiles more; an item that is cut leaves its pieces' (O, m, l)
// in the workspace, and a second kernel joins them:
//   O = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k.
//
// What bounds it: of a key tile's 3690 cycles (two row tiles, 8192 positions) the
// products take 2500, and the rest is a row tile's chain of S, softmax (2130 cycles), P
// and P V, since S and O of two row tiles fill the tensor memory; an item's start and end
// cost some 4 us more.  8 x 2048 tokens, 32 / 8 heads: int8 264 us, e4m3 260 (1060
// TFLOP/s, 0.55 of the library's rate), 4 x 8192 1624 and 1608 us (1368, 0.71); the bf16
// kernel 240 and 1529.  512 tokens after 8000 (floor 36) 70 us, after 100000 (436) 595;
// 64 after 8000 (4.4) 31.  The converters' proxy fence costs int8 1 % of the first.
#include <climits>

#include "decode_launch.cuh"
#include "pkv_device.cuh"
#include "prefill.cuh"
#include "q8.cuh"
#include "q8_math.cuh"
#include "umma.cuh"

namespace pkv {

using namespace umma;

namespace {

constexpr int kStages = 2;
constexpr int kQSlots = 2;                            // Q tiles in rotation
constexpr int kOffK = kQSlots * kOpBytes;             // after the Q slots
constexpr int kStageBytes = 2 * kOpBytes;             // K then V
constexpr int kCodeTile = kKeys * kCodeRowBytes;      // 16 KiB
constexpr int kOffCodes = kOffK + kStages * kStageBytes;  // a tile's codes of K, then of V
constexpr int kTilesBytes = kOffCodes + 2 * kCodeTile;  // 224 KiB
constexpr int kScaleRing = 8;                         // tiles whose scales are kept
// One pass over a tile is taken up to this sum of P, and of P vs: fp32 (and bf16, whose
// range is the same) then holds the sums over all tiles, and 448 times as much in O.
constexpr float kOnePassSum = 7.9228163e28f;  // 2^96
constexpr int kScaleFloats = 24;                      // of 8 groups: ks, log2 vs, 1 / vs
constexpr int kConvert0 = 12, kConverters = 8;        // converter warps
constexpr int kOffScales = kTilesBytes + 512;
constexpr int kSmemBytes = kOffScales + kScaleRing * kScaleFloats * 4 + 1024;  // + alignment
static_assert(kSmemBytes <= 232448, "shared memory per CTA exceeds 227 KiB");
constexpr int kProducer = 10;                         // the code producer
static_assert(kProducer == 10 && kConvert0 == 12, "warps 0-7 are the softmax's, 8 and 9 the next two");
constexpr int kThreads = 32 * (kConvert0 + kConverters);
// Registers a thread of the warpgroups, from the launch's.  The softmax's rows of S want
// many, the others do with less.  One warpgroup of converters was busy all the time (3800
// cycles of a key tile's 4270 in int8, 3150 of 3680 in e4m3) and a second one costs the
// softmax 8 registers: 8 x 2048 int8 282 -> 266 us, 4 x 8192 1822 -> 1611.
constexpr int kRegsLaunch = 96, kRegsSoftmax = 168, kRegsRoles = 64, kRegsConvert = 40;
static_assert(256 * kRegsSoftmax + 128 * kRegsRoles + 32 * kConverters * kRegsConvert <=
                      kThreads * kRegsLaunch && kThreads * kRegsLaunch <= 65536,
              "the launch's registers");
constexpr int kRingUsers = 10 + kConverters;  // readers: softmax, MMA, producer, converters
constexpr int kRing = 4;                              // item descriptors in flight
constexpr int kSplitItems = 4;               // items an SM up to which they are cut
constexpr int kSplitPairs = 1024;            // (sequence, row tiles) pairs up to which they are cut
constexpr int kSortPairs = 512;              // such pairs up to which whole items are sorted
constexpr int kItemCost = 2;                 // what an item costs, in key tiles
constexpr int kLeastUnits = 6;               // a CTA's share is at least this
constexpr int kPieceRow = 136;               // floats of a piece's row: o[128], m, l

// One work item, or a piece of one, as the item warp publishes it: key tiles t0 ..
// t0 + ntiles - 1 (ntiles 0 ends the list); part: the record that its sums go to, or
// -1 (the whole item).
struct PItem {
  int32_t seq, kvh, row0, rows, base, ntiles, q0, ctx, t0, part;
};

// What a CTA leaves for the join: the item whose first tiles are its last (rows 0:
// none), and whether its first tiles continue an earlier CTA's item (1), and end it
// (2).
struct PieceDesc {
  int32_t q0, kvh, row0, rows, continues, pad[3];
};

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

// The mbarriers after the tiles.
struct PBars {
  uint64_t* cfull;      // [2] a tile's codes and scales of K, its codes of V landed
  uint64_t* cempty;     // [2] the converters hold them in registers
  uint64_t* kfull;      // [2] K of a stage written (one arrival per converter warp)
  uint64_t* vfull;      // [2] V of a stage written
  uint64_t* kempty;     // [2] both S products reading a stage's K completed
  uint64_t* vempty;     // [2] both P V products reading a stage's V completed
  uint64_t* sfull;      // [2] S_t of the next key tile (and PV_t before it) done
  uint64_t* pfull;      // [2] P_t written (one arrival per warp)
  uint64_t* ofull;      // [2] an item's last PV_t completed
  uint64_t* qfull;      // [2] a Q slot written (every lane of the item warp arrives)
  uint64_t* qempty;     // [2] the last S product reading a Q slot completed
  uint64_t* ifull;      // [4] an item descriptor published
  uint64_t* iempty;     // [4] every reader took its copy
  uint64_t* drain;      // the MMA warp's final wait
};

// One lane of the warp (every lane calls).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r));
  return r != 0u;
}

// 64 consecutive columns of this warp's 32 lanes, loaded and waited for in one
// statement: until the wait the registers are not to be touched, and what the compiler
// puts between a load and a wait of their own (a copy of the first is enough) would.
__device__ __forceinline__ void tmem_ld64(uint32_t (&a)[32], uint32_t (&b)[32], uint32_t taddr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
      "%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,"
      "%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63"
      "}, [%64];\n\ttcgen05.wait::ld.sync.aligned;"
      : PKV_R32(PKV_OUT, a), PKV_R32(PKV_OUT, b)
      : "r"(taddr)
      : "memory");
}

// Four bytes of shared memory from global memory, or zeros.
__device__ __forceinline__ void cp_async_4_or_zero(void* dst, const void* src, bool copy) {
  const int n = copy ? 4 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src),
               "r"(n)
               : "memory");
}

// Shared memory that is written anew after this warp's arrival on an mbarrier: read by
// statements that the compiler places no later than where they stand.  What follows them
// is __syncwarp and lane 0's arrival, which releases the reads of the whole warp to a
// thread that waits for it and writes; a writer through the async proxy needs a proxy
// fence between the reads and the arrival too.
__device__ __forceinline__ uint4 ld_shared_v4(const void* p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(smem_addr(p))
               : "memory");
  return v;
}
__device__ __forceinline__ PItem ld_item(const PItem* p) {
  static_assert(sizeof(PItem) == 40, "five pairs of words");
  int32_t w[10];
#pragma unroll
  for (int i = 0; i < 5; ++i)
    asm volatile("ld.shared.v2.s32 {%0,%1}, [%2];"
                 : "=r"(w[2 * i]), "=r"(w[2 * i + 1])
                 : "r"(smem_addr(p) + 8 * i)
                 : "memory");
  return PItem{w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7], w[8], w[9]};
}

// Sixteen codes (a chunk of a row) as bf16, exact.
template <bool kE4m3>
__device__ __forceinline__ void codes_to_bf16(const uint4& c, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kE4m3) {
      // by fp16, which keeps NaN
      const uint32_t h[2] = {e4m3x2_to_half2(w[i]), e4m3x2_to_half2(w[i] >> 16)};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x, y;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\t"
            "cvt.f32.f16 %1, h;\n\t}" : "=f"(x), "=f"(y) : "r"(h[k]));
        o[2 * i + k] = pack_bf16x2(x, y);
      }
    } else {
      // y: the byte u = code + 128 as the low byte of 128's bits, which is 128 + u below
      // 128 and 2 u from there (the step doubles).  Less 256, and less half of what is
      // then positive, that is the code; exact, and all but the byte's placing on the
      // multiply-add pipe (the softmax keeps the other one busy).
      const uint32_t u = w[i] ^ 0x80808080u;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t y = __byte_perm(u, 0x43434343u, k == 0 ? 0x4140u : 0x4342u);
        uint32_t d, r;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(y), "r"(0x3f803f80u), "r"(0xc380c380u));
        asm("fma.rn.relu.bf16x2 %0, %1, %2, %3;"
            : "=r"(r) : "r"(y), "r"(0x3f003f00u), "r"(0xc300c300u));
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(o[2 * i + k]) : "r"(r), "r"(0xbf80bf80u), "r"(d));
      }
    }
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

}  // namespace

// What the kernel reads beside the plain one's parameters.
struct PrefillQ8Params : PrefillParams {
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const float* k_scale;
  const float* v_scale;
  PieceDesc* desc;      // [CTAs] and
  float* rec;           // [CTAs][2][rec_rows][kPieceRow]: items are cut; null: they are not
  int32_t rec_rows;     // rows of an item at most
  int32_t sorted;       // pairs (row tiles, sequence) to sort, or 0
};

// The larger one, or NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_q8_kernel(const __grid_constant__ CUtensorMap tmq,
                      const __grid_constant__ PrefillQ8Params p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
  uint64_t* bar0 = reinterpret_cast<uint64_t*>(smem + kTilesBytes);
  PBars B;
  B.kfull = bar0;
  B.vfull = bar0 + 2;
  B.kempty = bar0 + 4;
  B.vempty = bar0 + 6;
  B.sfull = bar0 + 8;
  B.pfull = bar0 + 10;
  B.ofull = bar0 + 12;
  B.cfull = bar0 + 14;
  B.cempty = bar0 + 16;
  B.qfull = bar0 + 18;
  B.qempty = B.qfull + kQSlots;
  B.ifull = B.qempty + kQSlots;
  B.iempty = B.ifull + kRing;
  B.drain = B.iempty + kRing;
  constexpr int kNumBars = 19 + 2 * kQSlots + 2 * kRing;
  static_assert(kNumBars * 8 + 8 <= 320 && 320 + kRing * sizeof(PItem) <= 512,
                "barriers, tensor-memory address and abort flag; item ring");
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar0 + kNumBars);
  volatile int* abort = reinterpret_cast<volatile int*>(bar0 + kNumBars) + 1;
  PItem* ring = reinterpret_cast<PItem*>(smem + kTilesBytes + 320);  // [kRing]
  float* scales = reinterpret_cast<float*>(smem + kOffScales);       // [kScaleRing][kScaleFloats]

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
  auto read_item = [&](int n, PItem& it) -> bool {
    const int slot = n & (kRing - 1);
    if (!__all_sync(kFull, wait_or_abort(&B.ifull[slot], (n / kRing) & 1, abort, p.err)))
      return false;
    it = ld_item(&ring[slot]);
    __syncwarp();
    if (lane == 0) mbar_arrive(&B.iempty[slot]);
    return true;
  };

  // Row tiles rt of a sequence (any KV head); false if there are none.
  auto describe = [&](int rt, int seq, bool report, PItem& it) -> bool {
    it.seq = seq;
    it.kvh = 0;
    it.t0 = 0;
    it.part = -1;
    it.q0 = p.cu_q[seq];
    const int Lq = p.cu_q[seq + 1] - it.q0;
    it.ctx = p.ctx_lens[seq];
    if (p.checked) {
      const int64_t cap = static_cast<int64_t>(p.max_blocks) * p.bs;
      if (Lq < 0 || Lq > p.max_q || it.ctx < Lq || it.ctx > cap) {
        if (report) record_error(p.err, kErrContext);
        return false;  // the sequence is left unwritten
      }
    }
    // (the workspace holds records for chunks of the call's bound: what a longer one has past
    // it is left unwritten, whether its item is cut or not)
    it.rows = min(Lq, p.max_q) * G;
    it.row0 = rt * 2 * TR;
    if (it.row0 >= it.rows) return false;  // past the chunk
    it.base = it.ctx - Lq;                 // position of the chunk's first token
    const int last_row = min(it.row0 + 2 * TR, it.rows) - 1;
    const int kend = it.base + last_row / G + 1;  // keys the item needs
    it.ntiles = (kend + kKeys - 1) / kKeys;
    return kend > 0;  // (not only when ctx < Lq, caught in checked mode)
  };
  // Setup: barriers, the Q slots' padding, the tensor memory.
  if (warp == kProducer) {
    if (lane == 0) {
      for (int s = 0; s < 2; ++s) {
        mbar_init(&B.cfull[s], s == 0 ? 1 + 32 : 1);  // the copies; K: and the lanes' scales
        mbar_init(&B.cempty[s], kConverters);
        mbar_init(&B.kfull[s], kConverters);
        mbar_init(&B.vfull[s], kConverters);
        mbar_init(&B.kempty[s], 1);
        mbar_init(&B.vempty[s], 1);
        mbar_init(&B.sfull[s], 1);
        mbar_init(&B.pfull[s], 4);  // one arrival per softmax warp
        mbar_init(&B.ofull[s], 1);
      }
      for (int s = 0; s < kQSlots; ++s) {
        mbar_init(&B.qfull[s], 32);  // every lane of the item warp
        mbar_init(&B.qempty[s], 1);
      }
      for (int s = 0; s < kRing; ++s) {
        mbar_init(&B.ifull[s], 1);
        mbar_init(&B.iempty[s], kRingUsers);
      }
      mbar_init(B.drain, 1);
      *abort = 0;
      fence_barrier_init();
      prefetch_tensormap(&tmq);
    }
  } else if (warp == 9 && TR < kRowTile) {
    // rows TR .. 127 of every Q slot are padding that no copy writes: zero
    for (int slot = 0; slot < kQSlots; ++slot)
      for (int x = lane; x < (kRowTile - TR) * 16; x += 32)
        *reinterpret_cast<uint4*>(smem + q_off(slot) + q_chunk_offset(TR + (x >> 4), x & 15)) =
            make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  } else if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // Pairs (row tiles, sequence) by what their items cost, dearest first: list[n] is the
  // n-th one's index.  In the operand stages, which nothing writes before the item warp
  // has read its part of the list.
  int32_t* key = reinterpret_cast<int32_t*>(smem + kOffK);
  int32_t* list = key + kSortPairs;
  if (p.sorted > 0) {
    for (int c = tid; c < kSortPairs; c += kThreads) {
      PItem it;
      const bool there = c < p.sorted && describe(c / p.num_seqs, c % p.num_seqs, blockIdx.x == 0 && c < p.num_seqs, it);
      // (a tile of two row tiles costs 2 to 1.2 of one with one; an item some 3 us more)
      key[c] = there ? it.ntiles * (it.rows > it.row0 + TR ? 5 : 3) + 8 : 0;
      list[c] = -1;
    }
    __syncthreads();
    for (int c = tid; c < p.sorted; c += kThreads) {
      const int mine = key[c];
      int rank = 0;
      for (int x = 0; x < p.sorted; x += 4) {
        const int4 k = *reinterpret_cast<const int4*>(key + x);
        rank += (k.x > mine || (k.x == mine && x < c)) + (k.y > mine || (k.y == mine && x + 1 < c)) +
                (k.z > mine || (k.z == mine && x + 2 < c)) + (k.w > mine || (k.w == mine && x + 3 < c));
      }
      if (mine > 0) list[rank] = c;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t smem_base = smem_addr(smem);

  // The converters: codes -> operands.  A thread takes 16 codes of rows row0, row0 +
  // kRowStep, ..  The eight lanes of a quarter warp take chunks 0-3 of one row and 4-7 of
  // the next (or the other way), whose loads and swizzled stores meet different banks.
  auto convert = [&]() {
    constexpr int kRowStep = 4 * kConverters;
    static_assert(4 * kRowStep == kKeys, "four rows a thread");
    const int row0 = (warp - kConvert0) * 4 + ((lane >> 4) << 1) + ((lane >> 2) & 1);
    const int ch = (lane & 3) + (((lane >> 2) ^ (lane >> 3)) & 1) * 4;  // chunk of 16 codes
    int g = 0;  // tiles of all items
    int nread = 0;
    bool ok = true;
    while (ok) {
      PItem it;
      if (!read_item(nread++, it) || it.ntiles == 0) break;
      for (int j = 0; j < it.ntiles && ok; ++j, ++g) {
        const int s = g & 1;
        const int left = it.ctx - (it.t0 + j) * kKeys;  // rows of the tile that hold positions
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {  // K, then V
          ok = __all_sync(kFull, wait_or_abort(&B.cfull[kv], g & 1, abort, p.err));
          if (!ok) break;
          const unsigned char* from = smem + kOffCodes + kv * kCodeTile + row0 * 128 + ch * 16;
          uint64_t* empty = kv == 0 ? B.kempty : B.vempty;
          unsigned char* to = smem + kOffK + s * kStageBytes + kv * kOpBytes;
          uint4 c[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) c[i] = ld_shared_v4(from + i * kRowStep * 128);
          // The next codes come by bulk copies, through the async proxy, and nothing has used
          // these values yet: only a proxy fence of the lanes that read keeps the copies
          // behind their reads (an arrival alone does not: without more the next codes now
          // and then came in first).
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&B.cempty[kv]);
          if (kv == 0 && warp == kConvert0 && lane < 8) {
            // a scale below 2^-100 is that of zeros, whose P only enters the sum
            float* sct = scales + (g & (kScaleRing - 1)) * kScaleFloats + 8 + lane;
            const float vs = *sct < kScaleTiny ? kScaleTiny : *sct;
            sct[0] = log2f(vs);
            sct[8] = 1.f / vs;
          }
          if (g >= kStages &&
              !__all_sync(kFull, wait_or_abort(&empty[s], ((g >> 1) - 1) & 1, abort, p.err))) {
            ok = false;
            break;
          }
          if (kv == 1 && left < kKeys) {  // values past the context: 0 x whatever stands there
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (row0 + kRowStep * i >= left) c[i] = make_uint4(0u, 0u, 0u, 0u);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 lo, hi;
            codes_to_bf16<kE4m3>(c[i], lo, hi);
            const int r = row0 + kRowStep * i;
            *reinterpret_cast<uint4*>(to + kv_chunk_offset(r, 2 * ch)) = lo;
            *reinterpret_cast<uint4*>(to + kv_chunk_offset(r, 2 * ch + 1)) = hi;
          }
          fence_proxy_async_smem();  // the products read them through the async proxy
          __syncwarp();
          if (lane == 0) mbar_arrive(kv == 0 ? &B.kfull[s] : &B.vfull[s]);
        }
      }
    }
  };

  if (warp >= kConvert0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
    // ================= converters: codes -> operands =================
    convert();
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRoles));
    if (warp == kProducer) {
      // ================= code producer =================
      // Every row tile of a sequence and KV head reads the same tiles: keep them in
      // L2 for the items after.
      const uint64_t policy = l2_policy_evict_last();
      const int run = p.run_rows;    // rows per copy (16 .. 128, divides 128 and bs)
      const int runs = kKeys / run;  // copies per tile and tensor (<= 8)
      const int prun = lane & 15;    // lanes 0-15 copy K of run prun, lanes 16-31 V
      const int kv = lane >> 4;
      const uint32_t bs = static_cast<uint32_t>(p.bs);
      // The run's row of the cache in tile j of `it` (-1: past the context, or a bad table
      // entry: the copy is skipped, stale rows, undefined output, no fault).  (Prefetched
      // to L2 a tile ahead, everything got slower: 8 x 2048 281 -> 298 us.)
      auto row_of = [&](const PItem& it, int j) -> int64_t {
        const int kpos = (it.t0 + j) * kKeys + prun * run;
        if (prun >= runs || kpos >= it.ctx) return -1;
        const uint32_t at = static_cast<uint32_t>(kpos) / bs;
        const int32_t e = p.block_tables[static_cast<int64_t>(it.seq) * p.max_blocks + at];
        if (p.checked && (e < 0 || e >= p.num_blocks)) {
          record_error(p.err, p.err_code);
          return -1;
        }
        return cache_row(e, it.kvh, p.Hkv, bs, static_cast<uint32_t>(kpos) - at * bs);
      };
      int g = 0;             // tiles (of all items) whose K and V were both asked for
      bool half = false;     // K of tile g was asked for, not its V
      int nread = 0;
      PItem cur;
      bool ok = read_item(nread++, cur);
      int64_t row = ok && cur.ntiles > 0 ? row_of(cur, 0) : -1;  // of the next tile
      while (ok && cur.ntiles > 0) {
        PItem nx = cur;
        for (int j = 0; j < cur.ntiles; ++j) {
          const int kpos = (cur.t0 + j) * kKeys + prun * run;
          const uint32_t loaded = __popc(__ballot_sync(kFull, lane < 16 && row >= 0));
          float* sc = scales + (g & (kScaleRing - 1)) * kScaleFloats + kv * 8;
  #pragma unroll 1
          for (int x = 0; x < 2; ++x) {  // K, then V, each when its slot is read
            if (g > 0 && !__all_sync(kFull, wait_or_abort(&B.cempty[x], (g - 1) & 1, abort, p.err))) {
              half = x == 1;
              ok = false;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&B.cfull[x], loaded * run * kCodeRowBytes);
            __syncwarp();
            if (kv == x && row >= 0)
              bulk_copy_g2s(smem + kOffCodes + x * kCodeTile + prun * run * kCodeRowBytes,
                            (x == 0 ? p.k_codes : p.v_codes) + row * kCodeRowBytes,
                            static_cast<uint32_t>(run * kCodeRowBytes), &B.cfull[x], policy);
            if (x == 0) {
              // the scales of the run's groups, V's with K's (the softmax of S takes both);
              // 0 past the context, where P is 0.  The slot's last readers are done: the
              // converters hold K of tile g - 1, so that of tile g - 2 is written, the S of
              // tile g - 4 that freed its stage is complete, and P of tile g - 5 was handed
              // over before.
              if (prun < runs) {
                const float* from =
                    (kv == 0 ? p.k_scale : p.v_scale) + (row >= 0 ? row / kGroupRows : 0);
                for (int i = 0; i < run / kGroupRows; ++i)
                  cp_async_4_or_zero(sc + prun * (run / kGroupRows) + i, from + (row >= 0 ? i : 0),
                                     row >= 0 && kpos + i * kGroupRows < cur.ctx);
              }
              asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                               smem_addr(&B.cfull[0]))
                           : "memory");
            }
            __syncwarp();
          }
          if (!ok) break;
          ++g;
          // the next tile is looked up while this one lands
          if (j + 1 < cur.ntiles) {
            row = row_of(cur, j + 1);
          } else {
            ok = read_item(nread++, nx);
            row = ok && nx.ntiles > 0 ? row_of(nx, 0) : -1;
          }
        }
        cur = nx;
      }
      if (*abort && lane == 0) {
        // let the copies in flight land before the CTA's shared memory is released
        if (g > 0) {
          if (!half) mbar_wait_bounded(&B.cfull[0], (g - 1) & 1);
          mbar_wait_bounded(&B.cfull[1], (g - 1) & 1);
        }
        if (half) mbar_wait_bounded(&B.cfull[0], g & 1);
      }
    } else if (warp == 9) {
      // ================= item list and Q rows =================
      // Q tile n (row tile 0 of an item, then row tile 1 if it has rows) goes to slot
      // n % 2 once the last S product reading tile n - 2 completed.
      const int P = gridDim.x;
      const int R = (p.max_q * G + 2 * TR - 1) / (2 * TR);
      const uint64_t qpolicy = l2_policy_evict_first();  // every Q row is read once
      int published = 0;
      uint32_t nq = 0;      // Q tiles loaded
      QCursor qc = {0, 0};  // slot of Q tile nq and its phase
      uint32_t last_phase = 0;  // bit s: phase of the last load into slot s
      bool ok = true;
      auto publish = [&](const PItem& it) -> bool {
        const int slot = published & (kRing - 1);
        if (published >= kRing &&
            !__all_sync(kFull, wait_or_abort(&B.iempty[slot], ((published / kRing) - 1) & 1,
                                             abort, p.err)))
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
      auto serve = [&](const PItem& it) -> bool {
        if (!publish(it)) return false;
        const int nt = it.rows > it.row0 + TR ? 2 : 1;
        for (int t = 0; t < nt; ++t, ++nq, qc = qc.next(kQSlots)) {
          const int qs = qc.slot;
          if (nq >= static_cast<uint32_t>(kQSlots) &&
              !__all_sync(kFull, wait_or_abort(&B.qempty[qs], qc.phase ^ 1u, abort, p.err)))
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
      // the item of lane src
      auto of_lane = [&](const PItem& mine, int src) -> PItem {
        PItem it;
        it.seq = __shfl_sync(kFull, mine.seq, src);
        it.kvh = __shfl_sync(kFull, mine.kvh, src);
        it.row0 = __shfl_sync(kFull, mine.row0, src);
        it.rows = __shfl_sync(kFull, mine.rows, src);
        it.base = __shfl_sync(kFull, mine.base, src);
        it.ntiles = __shfl_sync(kFull, mine.ntiles, src);
        it.q0 = __shfl_sync(kFull, mine.q0, src);
        it.ctx = __shfl_sync(kFull, mine.ctx, src);
        it.t0 = 0;
        it.part = -1;
        return it;
      };
      if (p.rec != nullptr) {
        // Pairs c = (sequence c / R, row tiles c % R) in order, 32 at a time, one a
        // lane; a pair's items (its KV heads) of kItemCost + ntiles units each.  A CTA's
        // units [u0, u1) hold a run of key tiles; those of an item that it has not
        // whole are a piece.
        const int pairs = R * p.num_seqs;
        auto pair_of_lane = [&](int c0, bool report, PItem& it) -> int64_t {
          const int c = c0 + lane;
          it = PItem{};
          if (c >= pairs || !describe(c % R, c / R, report && c % R == 0, it)) return 0;
          return static_cast<int64_t>(p.Hkv) * (kItemCost + it.ntiles);
        };
        PItem mine;
        int64_t V = 0, units = 0;
        for (int c0 = 0; c0 < pairs; c0 += 32) {
          units = pair_of_lane(c0, blockIdx.x == 0, mine);
          int64_t sum = units;
  #pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
          V += sum;
        }
        const int64_t shares = max(static_cast<int64_t>(1), min(static_cast<int64_t>(P), V / kLeastUnits));
        const int64_t me = blockIdx.x;
        const int64_t u0 = me < shares ? me * V / shares : V;
        const int64_t u1 = me < shares ? (me + 1) * V / shares : V;
        PieceDesc desc = {};
        int64_t at = 0;
        for (int c0 = 0; ok && c0 < pairs && at < u1; c0 += 32) {
          if (pairs > 32) units = pair_of_lane(c0, false, mine);
          int64_t end = units;
  #pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(kFull, end, o);
            if (lane >= o) end += v;
          }
          const int64_t begin = at + end - units;
          for (uint32_t hit = __ballot_sync(kFull, units > 0 && begin < u1 && begin + units > u0);
               ok && hit != 0u; hit &= hit - 1) {
            const int src = __ffs(hit) - 1;
            PItem it = of_lane(mine, src);
            const int64_t b = __shfl_sync(kFull, begin, src);
            const int n = it.ntiles, span = kItemCost + n;
            for (int h = u0 > b ? static_cast<int>((u0 - b) / span) : 0; ok && h < p.Hkv; ++h) {
              const int64_t first = b + static_cast<int64_t>(h) * span + kItemCost;  // unit of tile 0
              if (first >= u1) break;
              const int from = u0 > first ? static_cast<int>(u0 - first) : 0;
              const int to = u1 - first < n ? static_cast<int>(u1 - first) : n;
              if (from >= to) continue;
              it.kvh = h;
              it.t0 = from;
              it.ntiles = to - from;
              it.part = -1;
              if (to - from < n) {
                it.part = 2 * blockIdx.x + (from == 0 ? 1 : 0);
                if (from == 0) {
                  desc.q0 = it.q0;
                  desc.kvh = h;
                  desc.row0 = it.row0;
                  desc.rows = min(it.rows - it.row0, 2 * TR);
                } else {
                  desc.continues = to == n ? 2 : 1;
                }
              }
              ok = serve(it);
            }
          }
          at += __shfl_sync(kFull, end, 31);
        }
        if (lane == 0) p.desc[blockIdx.x] = desc;
      } else {
        // Items in order: pairs as sorted, or row tile (latest first), then sequence; then
        // KV head.  Round k deals items k P .. k P + P - 1 to the P CTAs, forwards in even
        // rounds and backwards in odd ones; 32 rounds at a time, one a lane, so that items
        // whose rows lie past their chunk cost one latency (a sorted list has no more).
        const int total = R * p.num_seqs * p.Hkv;
        for (int64_t k0 = 0; ok && k0 * P < total; k0 += 32) {
          const int64_t k = k0 + lane;
          const int64_t slot = k * P + ((k & 1) ? P - 1 - static_cast<int>(blockIdx.x)
                                                : static_cast<int>(blockIdx.x));
          PItem mine = {};
          bool there = slot < total;
          if (there) {
            const int idx = static_cast<int>(slot), at = idx / p.Hkv;
            const int c = p.sorted > 0 ? (at < p.sorted ? list[at] : -1)
                                       : (R - 1 - at / p.num_seqs) * p.num_seqs + at % p.num_seqs;
            there = c >= 0 && describe(c / p.num_seqs, c % p.num_seqs,
                                       p.sorted == 0 && c < p.num_seqs && idx == at * p.Hkv, mine);
            mine.kvh = idx - at * p.Hkv;
          }
          for (uint32_t left = __ballot_sync(kFull, there); ok && left != 0u; left &= left - 1)
            ok = serve(of_lane(mine, __ffs(left) - 1));
        }
      }
      if (ok) {
        PItem end = {};  // ntiles 0: the end of this CTA's list
        publish(end);
      }
      if (*abort && lane == 0) {
        // let the Q copies in flight land before the shared memory is released
        for (int qs = 0; qs < kQSlots && static_cast<uint32_t>(qs) < nq; ++qs)
          mbar_wait_bounded(&B.qfull[qs], (last_phase >> qs) & 1u);
      }
    } else if (warp == 8) {
      // ================= MMA issuer =================
      // The whole warp walks the tiles on warp-uniform values, so that descriptors stay
      // in uniform registers; one elected lane issues.
      const uint32_t tm = __shfl_sync(kFull, tmem, 0);
      const uint32_t base = __shfl_sync(kFull, smem_base, 0);
      // the low words of the operands' descriptors (smem_desc): address, leading offset
      const uint32_t q_lo = (((base + q_off(0)) & 0x3FFFFu) >> 4) | ((16u >> 4) << 16);
      const uint32_t k_lo = (((base + kOffK) & 0x3FFFFu) >> 4) | ((16u >> 4) << 16);
      const uint32_t v_lo = (((base + kOffK + kOpBytes) & 0x3FFFFu) >> 4) | ((1024u >> 4) << 16);
      constexpr uint32_t kHiQ = (1024u >> 4) | (1u << 14) | (2u << 29);  // stride, mode
      constexpr uint32_t kHiKV = (2048u >> 4) | (1u << 14) | (2u << 29);
      auto desc = [](uint32_t lo, uint32_t hi) -> uint64_t {
        return (static_cast<uint64_t>(hi) << 32) | lo;
      };
      auto issue_s = [&](int t, int qs, int stage) {  // S_t = Q K^T
        const uint32_t q = q_lo + qs * (kOpBytes >> 4), k = k_lo + stage * (kStageBytes >> 4);
  #pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_ss(tm + t * 128, desc(q + (kk >> 2) * (kHalfBytes >> 4) + (kk & 3) * 2, kHiQ),
                  desc(k + (kk >> 2) * (1024 >> 4) + (kk & 3) * 2, kHiKV), kIdescS, kk > 0);
      };
      auto issue_pv = [&](int t, int stage, bool acc) {  // O_t (+)= P_t V
        const uint32_t v = v_lo + stage * (kStageBytes >> 4);
  #pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_ts(tm + 256 + t * 128, tm + t * 128 + kk * 8, desc(v + kk * (4096 >> 4), kHiKV),
                  kIdescPV, (acc || kk > 0));
      };
      auto waitb = [&](uint64_t* b, uint32_t parity) -> bool {
        return __all_sync(kFull, wait_or_abort(b, parity, abort, p.err));
      };
      // what the products need of an item: its key tiles (0: the end), a second row tile
      int ntiles = 0;
      bool two = false;
      auto next_item = [&](int n) -> bool {
        PItem it;
        if (!read_item(n, it)) return false;
        ntiles = __shfl_sync(kFull, it.ntiles, 0);
        two = __shfl_sync(kFull, it.rows - it.row0, 0) > TR;
        return true;
      };
      // S products of the item's first tile, global tile g, its Q tiles at qa, qb
      auto first_s = [&](QCursor qa, QCursor qb, int g) -> bool {
        if (!waitb(&B.kfull[g & 1], (g >> 1) & 1) || !waitb(&B.qfull[qa.slot], qa.phase))
          return false;
        tc_fence_after();
        if (elect_one()) {
          issue_s(0, qa.slot, g & 1);
          umma_commit(&B.sfull[0]);
          if (ntiles == 1) umma_commit(&B.qempty[qa.slot]);
          if (!two) umma_commit(&B.kempty[g & 1]);
        }
        __syncwarp();
        if (two) {
          if (!waitb(&B.qfull[qb.slot], qb.phase)) return false;
          tc_fence_after();
          if (elect_one()) {
            issue_s(1, qb.slot, g & 1);
            umma_commit(&B.sfull[1]);
            if (ntiles == 1) umma_commit(&B.qempty[qb.slot]);
            umma_commit(&B.kempty[g & 1]);  // both S products of tile g issued
          }
          __syncwarp();
        }
        return true;
      };
      int nread = 0;
      bool ok = next_item(nread++);
      QCursor q0 = {0, 0};        // the item's Q tiles: row tile 0 at q0, row tile 1 at q1
      QCursor q1 = q0.next(kQSlots);
      int g = 0;                  // tile index over all items (ring stage g & 1)
      uint32_t np0 = 0, np1 = 0;  // P hand-overs taken per row tile
      if (ok && ntiles > 0) ok = first_s(q0, q1, g);
      // Tile g, tile j of the item: within an item PV_0(j) S_0(j+1) | PV_1(j) S_1(j+1);
      // at an item's last tile both P V products go first, then the next item's first S
      // products, so the current item never waits on the next.
      int j = 0;
      while (ok && ntiles > 0) {
        const int s = g & 1;
        const bool last = j == ntiles - 1;
        const bool qlast = j + 1 == ntiles - 1;  // S of tile j + 1 reads the item's Q last
        ok = waitb(&B.vfull[s], (g >> 1) & 1) && waitb(&B.pfull[0], np0 & 1);
        ++np0;
        if (ok && !last) ok = waitb(&B.kfull[s ^ 1], ((g + 1) >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
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
        __syncwarp();
        if (two) {
          ok = waitb(&B.pfull[1], np1 & 1);
          ++np1;
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            issue_pv(1, s, j > 0);
            if (last) umma_commit(&B.ofull[1]);
            umma_commit(&B.vempty[s]);  // the converters reuse the stage
            if (!last) {
              issue_s(1, q1.slot, s ^ 1);
              umma_commit(&B.sfull[1]);
              if (qlast) umma_commit(&B.qempty[q1.slot]);
              umma_commit(&B.kempty[s ^ 1]);
            }
          }
          __syncwarp();
        }
        ++g;
        if (last) {
          const bool had_two = two;
          ok = next_item(nread++);
          if (!ok) break;
          q0 = had_two ? q1.next(kQSlots) : q1;  // the next item's Q tiles follow
          q1 = q0.next(kQSlots);
          j = 0;
          if (ntiles > 0) ok = first_s(q0, q1, g);
        } else {
          ++j;
        }
      }
      // every product issued has completed before the tensor memory is released (one
      // lane has issued them all: elect.sync gives the same lane each time)
      if (elect_one()) {
        umma_commit(B.drain);
        mbar_wait_bounded(B.drain, 0);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ================= softmax warpgroups (warps 0-7) =================
    const int t = warp >> 2;                      // row tile
    const int lr = tid & (kRowTile - 1);          // row in the tile = tensor-memory lane
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + t * 128;
    const uint32_t o_tm = tmem + lane_base + 256 + t * 128;
    const bool negative = p.qscale < 0.f;
    const float sc = fabsf(p.qscale);
    uint32_t ns = 0, no = 0;  // S tiles and items this row tile took
    int g = 0;                // tiles of all items, this one's first
    bool ok = true;
    for (int n = 0; ok; ++n) {
      PItem it;
      if (!read_item(n, it) || it.ntiles == 0) break;
      const int g0 = g;
      g += it.ntiles;
      if (t == 1 && it.rows <= it.row0 + TR) continue;  // row tile 1 holds no rows
      const int r = it.row0 + t * TR + lr;  // row of the chunk
      const bool valid = lr < TR && r < it.rows;
      const int rr = valid ? r : it.rows - 1;     // padding rows mirror the last row
      const int tok = rr / G;
      const int head = it.kvh * G + rr % G;
      const int pos = it.base + tok;
      const int64_t qrow = (static_cast<int64_t>(it.q0) + tok) * p.Hq + head;
      float m_used = -INFINITY;  // the maximum P is taken against (scaled logits)
      float l = 0.f;
      for (int j = 0; j < it.ntiles; ++j) {
        ok = __all_sync(kFull, wait_or_abort(&B.sfull[t], ns & 1, abort, p.err));
        ++ns;
        if (!ok) break;
        tc_fence_after();
        const int k0 = (it.t0 + j) * kKeys;
        // columns of the tile that this row sees, and that all / any of the warp's do
        const int seen = min(max(pos - k0 + 1, 0), kKeys);
        const int all = __reduce_min_sync(kFull, seen), any = __reduce_max_sync(kFull, seen);
        // plain: nothing is masked, and the largest of 16 columns is the largest product
        const bool plain = all == kKeys && !negative;
        // the tile's scales, of 16 columns each: ks, log2 vs, 1 / vs
        const float* sct = scales + ((g0 + j) & (kScaleRing - 1)) * kScaleFloats;
        // Else S takes the sign of the softmax's factor and -inf for the columns that the
        // row does not see, and what follows is the same; no factor is 0, so that -inf
        // stays that.
        auto factors = [&](int h, float (&ks)[4]) {
          const float4 k4 = *reinterpret_cast<const float4*>(sct + 4 * h);
          ks[0] = max_nan(k4.x * sc, 1.17549435e-38f);
          ks[1] = max_nan(k4.y * sc, 1.17549435e-38f);
          ks[2] = max_nan(k4.z * sc, 1.17549435e-38f);
          ks[3] = max_nan(k4.w * sc, 1.17549435e-38f);
        };
        // columns 64 h .. 64 h + 31 (a) and + 32 .. + 63 (b) of S, with its sign and mask
        auto load_half = [&](int h, uint32_t (&a)[32], uint32_t (&b)[32]) {
          tmem_ld64(a, b, s_tm + 64 * h);
          if (negative) {
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              a[c] ^= 0x80000000u;
              b[c] ^= 0x80000000u;
            }
          }
          if (all < 64 * h + 64) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              if (all >= 64 * h + 16 * q + 16) continue;
              uint32_t* x = q < 2 ? a + 16 * q : b + 16 * (q - 2);
#pragma unroll
              for (int c = 0; c < 16; ++c) x[c] = 64 * h + 16 * q + c < seen ? x[c] : 0xff800000u;
            }
          }
        };
        // P vs = 2^(s * scale - m + log2 vs) as bf16 pairs, and the sum of P, which is that
        // of a group divided by its vs, to `sum` (as it is to `values`)
        auto powers = [&](int h, const uint32_t (&a)[32], const uint32_t (&b)[32], float m,
                          uint32_t (&pk)[32], float& sum, float& values) {
          float ks[4];
          factors(h, ks);
          const float4 lv4 = *reinterpret_cast<const float4*>(sct + 8 + 4 * h);
          const float lv[4] = {lv4.x - m, lv4.y - m, lv4.z - m, lv4.w - m};
          uint64_t ls2[4];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const uint32_t u0 = c < 16 ? a[2 * c] : b[2 * c - 32];
            const uint32_t u1 = c < 16 ? a[2 * c + 1] : b[2 * c - 31];
            const uint32_t kq = __float_as_uint(ks[c >> 3]), lq = __float_as_uint(lv[c >> 3]);
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(u0, u1), f2_pack(kq, kq), f2_pack(lq, lq)), x0, x1);
            const float e0 = fast_exp2(x0), e1 = fast_exp2(x1);
            const uint64_t e2 = f2_pack(__float_as_uint(e0), __float_as_uint(e1));
            ls2[c >> 3] = (c & 7) == 0 ? e2 : f2_add(ls2[c >> 3], e2);
            pk[c] = pack_bf16x2(e0, e1);
          }
          const float4 iv4 = *reinterpret_cast<const float4*>(sct + 16 + 4 * h);
          const float iv[4] = {iv4.x, iv4.y, iv4.z, iv4.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float l0, l1;
            f2_unpack(ls2[q], l0, l1);
            sum = fmaf(l0 + l1, iv[q], sum);
            values += l0 + l1;
          }
        };
        // One pass over S against a maximum of the tiles before, 0 at first: P is what it
        // would be against the tile's own, times a power of two, which O and l have too.
        // That stands where the sums stay in range, and, of the first tile, reach the 1
        // that they have against their maximum (so that no more of P underflows than
        // there).  S is left alone until then.
        bool done = false;
        if (plain) {
          const float m = j > 0 ? m_used : 0.f;
          float sum = 0.f, values = 0.f;
          uint32_t p0[32], p1[32];
          {
            uint32_t a[32], b[32];
            tmem_ld64(a, b, s_tm);
            powers(0, a, b, m, p0, sum, values);
          }
          {
            uint32_t a[32], b[32];
            tmem_ld64(a, b, s_tm + 64);
            powers(1, a, b, m, p1, sum, values);
          }
          // (not NaN; whatever a padding row holds is not asked)
          done = __all_sync(kFull, !valid || (sum <= kOnePassSum && values <= kOnePassSum &&
                                              (j > 0 || sum >= 1.f)));
          if (done) {
            tmem_st32(s_tm, p0);
            tmem_st32(s_tm + 32, p1);
            l += sum;
            m_used = m;
          }
        }
        if (!done) {
          // pass 1: the row maximum of the scaled, masked logits
          float tmax = -INFINITY;
#pragma unroll 1
          for (int h = 0; h < 2 && any > 64 * h; ++h) {
            uint32_t a[32], b[32];
            load_half(h, a, b);
            float ks[4];
            factors(h, ks);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t* x = q < 2 ? a + 16 * q : b + 16 * (q - 2);
              float u = __uint_as_float(x[0]), v = __uint_as_float(x[1]);
#pragma unroll
              for (int c = 2; c < 14; c += 4) {
                u = fmax3(u, __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
                v = fmax3(v, __uint_as_float(x[c + 2]), __uint_as_float(x[c + 3]));
              }
              u = fmax3(u, __uint_as_float(x[14]), __uint_as_float(x[15]));
              tmax = fmaxf(tmax, fmaxf(u, v) * ks[q]);
            }
          }
          const float m_new = fmaxf(m_used, tmax);
          if (j == 0) {
            m_used = m_new;  // finite, but in a piece that the row sees nothing of
          } else {
            // (a maximum that the one pass took may be far below this one; that it stays
            // is bounded by the values' scales)
            const float4 v0 = *reinterpret_cast<const float4*>(sct + 8);
            const float4 v1 = *reinterpret_cast<const float4*>(sct + 12);
            const float far = fmaxf(fmax3(fmax3(v0.x, v0.y, v0.z), v0.w, v1.x), fmax3(v1.y, v1.z, v1.w));
            const bool grow = m_new > m_used + (far <= 40.f ? 40.f : kRescaleLog2);
            if (__any_sync(kFull, grow)) {
              const float alpha = grow ? fast_exp2(m_used - m_new) : 1.f;
              if (grow) {
                l *= alpha;
                m_used = m_new;
              }
#pragma unroll
              for (int c0 = 0; c0 < kHeadDim; c0 += 64) {
                uint32_t w[32], w2[32];
                tmem_ld64(w, w2, o_tm + c0);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                  w[c] = __float_as_uint(__uint_as_float(w[c]) * alpha);
                  w2[c] = __float_as_uint(__uint_as_float(w2[c]) * alpha);
                }
                tmem_st32(o_tm + c0, w);
                tmem_st32(o_tm + c0 + 32, w2);
              }
            }
          }
          // pass 2: P, over the columns already read
          float values = 0.f;  // (unused)
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[32];
            if (any > 64 * h) {
              uint32_t a[32], b[32];
              load_half(h, a, b);
              powers(h, a, b, m_used == -INFINITY ? 0.f : m_used, pk, l, values);
            } else {  // no row of the warp sees a key of this half
#pragma unroll
              for (int c = 0; c < 32; ++c) pk[c] = 0u;
            }
            tmem_st32(s_tm + 32 * h, pk);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.pfull[t]);
      }
      if (!ok) break;
      ok = __all_sync(kFull, wait_or_abort(&B.ofull[t], no & 1, abort, p.err));
      ++no;
      if (!ok) break;
      // the item's output rows, or a piece's sums; the next item's first P V product
      // overwrites O_t only after these warps hand over its first P
      tc_fence_after();
      if (it.part < 0) {
        const float inv = l != 0.f ? 1.f / l : 0.f;
        uint4* dst = reinterpret_cast<uint4*>(p.out + qrow * kHeadDim);
#pragma unroll 1
        for (int c0 = 0; c0 < kHeadDim; c0 += 64) {
          uint32_t w[32], w2[32];
          tmem_ld64(w, w2, o_tm + c0);
          if (valid) {
            uint4 o[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const uint32_t* x = q < 4 ? w + 8 * q : w2 + 8 * (q - 4);
              o[q].x = pack_bf16x2(__uint_as_float(x[0]) * inv, __uint_as_float(x[1]) * inv);
              o[q].y = pack_bf16x2(__uint_as_float(x[2]) * inv, __uint_as_float(x[3]) * inv);
              o[q].z = pack_bf16x2(__uint_as_float(x[4]) * inv, __uint_as_float(x[5]) * inv);
              o[q].w = pack_bf16x2(__uint_as_float(x[6]) * inv, __uint_as_float(x[7]) * inv);
            }
            if (p.out_v8) {  // out 32-byte aligned: whole 32-byte sectors
#pragma unroll
              for (int q = 0; q < 8; q += 2) st_global_v8(dst + c0 / 8 + q, o[q], o[q + 1]);
            } else {
#pragma unroll
              for (int q = 0; q < 8; ++q) dst[c0 / 8 + q] = o[q];
            }
          }
        }
      } else {
        float* rec = p.rec + (static_cast<int64_t>(it.part) * p.rec_rows + t * TR + lr) * kPieceRow;
#pragma unroll 1
        for (int c0 = 0; c0 < kHeadDim; c0 += 64) {
          uint32_t w[32], w2[32];
          tmem_ld64(w, w2, o_tm + c0);
          if (valid) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const uint32_t* x = q < 4 ? w + 8 * q : w2 + 8 * (q - 4);
              st_global_v8(rec + c0 + 8 * q, make_uint4(x[0], x[1], x[2], x[3]),
                           make_uint4(x[4], x[5], x[6], x[7]));
            }
          }
        }
        if (valid) {
          rec[128] = m_used;
          rec[129] = l;
        }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
  }
}

namespace {

// Joins the pieces of the item that CTA blockIdx.x began and did not end: a warp a
// row, rows dealt to the warps of grid y.
__global__ void __launch_bounds__(256) prefill_q8_join_kernel(const __grid_constant__ PrefillQ8Params p,
                                                              int ctas) {
  grid_dependency_trigger();
  grid_dependency_wait();
  const PieceDesc d = p.desc[blockIdx.x];
  const int lane = threadIdx.x & 31;
  if (d.rows <= static_cast<int>(blockIdx.y) * 8) return;
  // the CTA of the item's last piece: the first after this one that does not go on
  int last = blockIdx.x + 1;
  for (bool found = false; !found; last += 32) {
    const int c = last + lane;
    const uint32_t ends = __ballot_sync(kFull, c >= ctas - 1 || p.desc[c].continues != 1);
    found = ends != 0u;
    if (found) last += __ffs(ends) - 1 - 32;
  }
  const int64_t stride = static_cast<int64_t>(2) * p.rec_rows * kPieceRow;  // CTA to CTA
  const int n = last - static_cast<int>(blockIdx.x) + 1;  // pieces
  for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < d.rows; r += gridDim.y * 8) {
    // piece k's row: record 1 of this CTA, then record 0 of the next ones
    const float* base = p.rec + blockIdx.x * stride + static_cast<int64_t>(r) * kPieceRow;
    auto row_of = [&](int k) {
      return base + (k == 0 ? static_cast<int64_t>(p.rec_rows) * kPieceRow : k * stride);
    };
    float M = -INFINITY;
    for (int k = lane; k < n; k += 32) {
      const float2 ml = *reinterpret_cast<const float2*>(row_of(k) + 128);
      if (ml.y != 0.f) M = fmaxf(M, ml.x);  // (0: the row sees nothing of the piece)
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    float L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const float2 ml = *reinterpret_cast<const float2*>(row_of(k) + 128);
      const float4 v = *reinterpret_cast<const float4*>(row_of(k) + 4 * lane);
      const float w = ml.y != 0.f ? fast_exp2(ml.x - M) : 0.f;
      L = fmaf(w, ml.y, L);
      o.x = fmaf(w, v.x, o.x);
      o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    const int tok = (d.row0 + r) / p.G;
    const int64_t qrow = (static_cast<int64_t>(d.q0) + tok) * p.Hq + d.kvh * p.G + d.row0 + r - tok * p.G;
    *reinterpret_cast<uint2*>(p.out + qrow * kHeadDim + 4 * lane) =
        make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  }
}

template <bool kE4m3>
cudaError_t launch(const CUtensorMap& tq, const PrefillQ8Params& p, int grid, cudaStream_t stream) {
  static unsigned long long done_mask = 0;
  auto kernel = prefill_q8_kernel<kE4m3>;
  const cudaError_t e = ensure_smem_limit(kernel, kSmemBytes, &done_mask);
  if (e != cudaSuccess) return e;
  return launch_pdl_if(pdl_decode_enabled(), kernel, dim3(static_cast<unsigned>(grid)),
                       dim3(kThreads), kSmemBytes, stream, tq, p);
}

int64_t row_tile_pairs(int64_t max_q, int G, int tile_rows) {
  return (max_q * G + 2 * tile_rows - 1) / (2 * tile_rows);
}

// Rows of a piece's record; 0: items are not cut.
int split_rows(int num_tokens, int num_seqs, int max_q, int Hkv, int G, int sms) {
  const int tile_rows = (kRowTile / G) * G;
  const int64_t R = row_tile_pairs(max_q, G, tile_rows);
  const int64_t most = static_cast<int64_t>(num_tokens) * G / (2 * tile_rows) + num_seqs;
  const int64_t pairs = R * num_seqs;
  if (pairs > kSplitPairs || (most < pairs ? most : pairs) * Hkv > static_cast<int64_t>(kSplitItems) * sms)
    return 0;
  const int64_t rows = static_cast<int64_t>(max_q) * G;
  return static_cast<int>(rows < 2 * tile_rows ? rows : 2 * tile_rows);
}

size_t desc_bytes(int sms) { return static_cast<size_t>(sms) * sizeof(PieceDesc); }

}  // namespace

size_t prefill_q8_workspace(int num_tokens, int num_seqs, int max_q, int Hkv, int G, int sms) {
  const int rows = split_rows(num_tokens, num_seqs, max_q < num_tokens ? max_q : num_tokens, Hkv, G, sms);
  if (rows == 0) return 0;
  return desc_bytes(sms) + static_cast<size_t>(sms) * 2 * rows * kPieceRow * sizeof(float);
}

TcStatus launch_prefill_q8(const AttentionQ8Params& a, bool e4m3, bool contig, int num_tokens, int sms,
                           void* workspace, cudaStream_t stream, cudaError_t* cuda_err) {
  *cuda_err = cudaSuccess;
  PrefillQ8Params p = {};
  p.q = a.q;
  p.out = a.out;
  p.cu_q = a.cu_q;
  p.ctx_lens = a.ctx_lens;
  p.block_tables = a.tables;
  p.bs = a.bs;
  p.num_blocks = a.num_blocks;
  p.max_blocks = a.max_blocks;
  p.num_seqs = a.num_seqs;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.G;
  p.max_q = a.max_q;
  // rows a copy: those of a block that a tile holds whole (contiguous: a group, so
  // that no row past the last group with positions is read)
  int run = 128;
  while (a.bs % run != 0) run >>= 1;
  p.run_rows = contig ? kGroupRows : run;
  p.tile_rows = (kRowTile / a.G) * a.G;
  p.qscale = a.qscale;
  p.out_v8 = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 ? 1 : 0;
  p.checked = a.checked;
  p.err = a.err;
  p.err_code = a.err_code;
  p.k_codes = a.k_codes;
  p.v_codes = a.v_codes;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  alignas(64) CUtensorMap tq;
  if (!encode_prefill_rows(&tq, a.q, num_tokens, a.Hq, a.G, p.tile_rows))
    return TcStatus::kEncodeFailed;
  const int64_t items = row_tile_pairs(p.max_q, p.G, p.tile_rows) * p.Hkv * p.num_seqs;
  if (items > INT32_MAX) {
    *cuda_err = cudaErrorInvalidValue;
    return TcStatus::kCudaError;
  }
  int grid = static_cast<int>(items < sms ? items : sms);
  p.rec_rows = split_rows(num_tokens, p.num_seqs, p.max_q, p.Hkv, p.G, sms);
  if (p.rec_rows > 0) {
    grid = sms;
    p.desc = static_cast<PieceDesc*>(workspace);
    p.rec = reinterpret_cast<float*>(static_cast<unsigned char*>(workspace) + desc_bytes(sms));
  }
  // (the item warp holds 32 rounds, one a lane)
  if (p.rec_rows == 0 && items > sms && items / p.Hkv <= kSortPairs && items <= 32 * static_cast<int64_t>(sms))
    p.sorted = static_cast<int32_t>(items / p.Hkv);
  *cuda_err = e4m3 ? launch<true>(tq, p, grid, stream) : launch<false>(tq, p, grid, stream);
  if (*cuda_err == cudaSuccess && p.rec_rows > 0)
    *cuda_err = launch_pdl_if(pdl_decode_enabled(), prefill_q8_join_kernel,
                              dim3(static_cast<unsigned>(grid), static_cast<unsigned>((p.rec_rows + 7) / 8)),
                              dim3(256), 0, stream, p, grid);
  return *cuda_err == cudaSuccess ? TcStatus::kOk : TcStatus::kCudaError;
}

}  // namespace pkv
