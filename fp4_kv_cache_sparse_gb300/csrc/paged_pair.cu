// paged_pair.cu -- attention over a paged FP4 cache for sequences that share
// prefixes, where many query rows see the same tokens (the rows of a group over its
// prefix, those of a sequence over its own tokens): 128 rows at a time on a pair of SMs.
//
// The mathematics is that of paged.cu (S^T = K Q^T, P^T = 2^(scale (S - m)),
// O^T += V^T P^T, one pass with a lazy running maximum); the split is not.  There
// one SM decodes every record for 64 rows, and shared memory is what bounds it:
// V is written and read at 128 KB a tile whatever the rows.  Here a 2-CTA cluster
// issues products over both SMs (cta_group::2): an item is 256 tokens, of which
// each CTA decodes K for its own 128 (its lanes of S^T) and V for its own 256 dims
// (its lanes of O^T), and holds Q and P of its own 64 rows (half of the B operands).
// So a record is decoded once as key and once as value for 128 rows, and the
// accesses of shared memory per row and token are under half of paged.cu's.
//
// What the CTAs exchange: P^T of the other's rows (16 KB an item, by remote
// stores), a vote per item whether some row's maximum has grown past its slack
// (both CTAs hold the same running maximum of all 128 rows, as O^T adds up the
// tokens of both), the new maxima when it has, row sums at a unit's end.
//
// What bounds it is the chain of an item, some 8000 cycles: V goes into two slots a
// block, so each waits for its product before it is written again, 2000 cycles a
// page; and the P of the other CTA's rows is there 3000 to 4000 after it is
// written.  Nothing is full: instruction issue 54 %, tensor cores 46 %, shared memory 55 %.
// 64 sequences x 128 heads over one prefix of 16k tokens take 267 us, 284
// GFLOP at 1.06 PFLOP/s or 53 % of measured (paged.cu's form: 354).
// A vote that passes costs an item some 3000 cycles, as the last product and both
// CTAs have to be waited for.  So the pages that are selected for a query
// token stay with paged.cu: 64 x 128 heads over 64 pages each take 82 us here
// and 93 there when scores are flat, but 130 and 113 when many heads have a page
// of their own that towers above the others, which is what is selected.
//
// One CTA, 28 warps: softmax (16, thread = token x 32 rows), K decode (4), V
// decode (4), loader; in the first CTA the score issuer and two value issuers.
#include <cstdint>

#include "mla_device.cuh"
#include "mla_internal.h"
#include "mla_tensor.cuh"
#include "shared_units.cuh"

namespace mla {

namespace {

constexpr int NR = 128, kMine = 64;  // rows of a unit, of a CTA
constexpr int kStep = 256;           // tokens of an item
constexpr int kUnitCost = 2;         // what a unit's Q and epilogue take, in items
constexpr int kMergeCost = 3;
constexpr float kSlack = 10.f;       // as in paged.cu
constexpr float kPBias = 5.f;
constexpr float kNoMax = -3.0e38f;
constexpr uint64_t kWaitNs = 2000000000ull;

constexpr int kSoftmaxWarps = 16, kKWarp0 = 16, kVWarp0 = 20, kLoadWarp = 24, kScoreWarp = 25, kValueWarp0 = 26;
constexpr int kThreads = 28 * 32, kSoftmaxThreads = kSoftmaxWarps * 32;
// Registers by warpgroups: a softmax thread sums 32 rows.
constexpr int kSoftmaxRegs = 88, kOtherRegs = 56;
constexpr int kDecodeRegs = 48, kLaunchRegs = 72;
static_assert(4 * kSoftmaxRegs + kOtherRegs + 2 * kDecodeRegs <= 7 * kLaunchRegs, "registers of the launch");
constexpr int kInfoRing = 8;

struct Unit {  // (the loader reads it word by word)
  int b;            // sequence, or -1 - group of a prefix
  int row0, nrows;  // first row (of the batch), rows
  int first;        // position of the sequence's first query token
  int p_lo, p_hi;   // positions of the first and the last row's query token
  int tiles;        // items; a unit that sees nothing still writes its rows, a prefix without tokens is none (0)
};

constexpr int kUnitWords = 7;
static_assert(sizeof(Unit) == 4 * kUnitWords, "units");
// What the loader tells the other warps of an item, in words: tokens of its four
// pages (a byte each), flags, tile, unit, and when the piece closes and the run goes
// on the Unit that comes next.
constexpr int kItemBytes = 48;
enum : int {
  kOpens = 1,      // first item of a piece
  kCloses = 2,     // last item of a piece
  kFromStart = 4,  // the piece begins with its unit
  kToEnd = 8,      // the piece ends with its unit
  kWhole = 16      // every row sees every token
};

struct L {
  // A page in shared memory: this CTA's half of its rows' data bytes (128-byte
  // swizzle) and the 32 scale bytes a row (32-byte swizzle); of the CTA's own
  // pages, which are keys too, the other half lies in a ring of its own.
  static constexpr int kHalf = kPage * 128, kEntry = kHalf + kPage * 32;
  static constexpr int kOwn = 5, kOther = 2, kForeign = 2;
  static constexpr int kVTokens = 32, kVUnit = kVTokens * 256, kVSlots = 2;  // of a block of 128 dims
  static constexpr int kKDims = 64, kKSlots = 4;
  static constexpr int kQOff = 0;
  static constexpr int kPOff = kQOff + kMine * kD * 2;
  static constexpr int kVOff = kPOff + kStep * kMine * 2;
  static constexpr int kOwnOff = kVOff + 2 * kVSlots * kVUnit;
  static constexpr int kOtherOff = kOwnOff + kOwn * kEntry;
  static constexpr int kForeignOff = kOtherOff + kOther * kHalf;
  static constexpr int kBarOff = kForeignOff + kForeign * kEntry;
  static constexpr int bOwnFull = 0, bOwnFree = bOwnFull + kOwn, bOtherFull = bOwnFree + kOwn,
                       bOtherFree = bOtherFull + kOther, bForeignFull = bOtherFree + kOther,
                       bForeignFree = bForeignFull + kForeign, bKFull = bForeignFree + kForeign,
                       bKFree = bKFull + kKSlots, bVFull = bKFree + kKSlots, bVFree = bVFull + 2 * kVSlots,
                       bSFull = bVFree + 2 * kVSlots, bSFree = bSFull + 1, bPFull = bSFree + 1, bPFree = bPFull + 2,
                       bQFull = bPFree + 2, bOFree = bQFull + 1, bQRaw = bOFree + 1, bUnit = bQRaw + 1,
                       bVote = bUnit + 1, bXchg = bVote + 2, bDrain = bXchg + 1, bInfo = bDrain + 1,
                       kNumBars = bInfo + kInfoRing;
  static constexpr int kColOff = (kBarOff + kNumBars * 8 + 15) & ~15;
  // A float (int) for each row: minus the running maximum of the unscaled scores; minus the largest score that P has
  // room for under it; the factor of the last rescale; 1 / sum; the scale, of this unit and the next in turn; both
  // CTAs' maxima and sums; the last position that the row sees; the maxima or sums of the four lane quadrants.
  static constexpr int kMinusMOff = kColOff, kMinusMostOff = kMinusMOff + NR * 4, kAlphaOff = kMinusMostOff + NR * 4,
                       kLinvOff = kAlphaOff + NR * 4, kScaleOff = kLinvOff + NR * 4, kXMaxOff = kScaleOff + 2 * NR * 4,
                       kXSumOff = kXMaxOff + 2 * NR * 4, kHiOff = kXSumOff + 2 * NR * 4, kRedOff = kHiOff + NR * 4;
  static constexpr int kInfoOff = kRedOff + 4 * NR * 4;
  static constexpr int kMiscOff = kInfoOff + kInfoRing * kItemBytes;
  static constexpr int kUnitOff = kMiscOff + 336;
  static constexpr int kEnd = kMiscOff + 400;
  static constexpr int kAlloc = kEnd + 1024;
  static_assert(kAlloc <= 232448, "shared memory of one CTA");
  __device__ static int arrivals(int i) {
    if (i >= bOwnFree && i < bOtherFull) return 2 + 4;      // K warps of the page's quadrants, V warps
    if (i >= bOtherFree && i < bForeignFull) return 2;
    if (i >= bForeignFree && i < bKFull) return 4;
    if (i >= bKFull && i < bKFree) return 2 * 4;            // both CTAs
    if (i >= bVFull && i < bVFree) return 2;                // both CTAs
    if (i == bSFree || i == bQFull || i == bOFree || i == bUnit || i == bVote || i == bVote + 1)
      return 2 * kSoftmaxWarps;
    // Half of P, the tokens of two lane quadrants: eight warps of each CTA, whichever CTA their rows' P goes to.
    if (i == bPFull || i == bPFull + 1) return kSoftmaxWarps;
    if (i == bPFree || i == bPFree + 1) return 2;              // both value issuers
    if (i == bXchg) return 2 * 4;
    if (i == bDrain) return 3;
    return 1;
  }
  // Tensor memory columns: O^T blocks, S^T, K quarters.
  static constexpr int cO = 0, cS = 2 * NR, cK = 3 * NR;
  static_assert(cK + kKSlots * (kKDims / 2) == 512, "tensor memory");
};

// The pages of an item in the order in which they go into O^T, the CTAs' in turn: page 0 and 2 carry the P of
// both CTAs' first two lane quadrants, so one half of P is written while the product reads the other.
__device__ __forceinline__ int page_at_step(int at) { return ((at & 1) << 1) | (at >> 1); }

// ------------------------------------------------------------------ geometry

__device__ __forceinline__ Unit unit_of(const SharedParams& p, int groups, int u, bool& bad, int num_groups) {
  Unit t;
  if (u >= p.batch * groups) {
    const PrefixUnit at = prefix_unit_at<NR>(p, u - p.batch * groups, num_groups);
    bad = at.bad;
    t.b = -1 - at.group;
    t.row0 = at.row0;
    t.nrows = at.nrows;
    t.first = t.p_lo = t.p_hi = at.len - 1;
    t.tiles = (at.len + kStep - 1) / kStep;
    return t;
  }
  t.b = u / groups;
  const int row = (u - t.b * groups) * NR;  // of the sequence
  t.row0 = t.b * p.rows + row;
  t.nrows = min(NR, p.rows - row);
  const int len = load_i32(p.seq_lens + t.b);
  bad = len < 0 || len > p.max_pages * kPage;
  t.first = (bad ? 0 : len) - p.s;
  t.p_lo = t.first + row / p.h;
  t.p_hi = t.first + (row + t.nrows - 1) / p.h;
  t.tiles = max((t.p_hi + 1 + kStep - 1) / kStep, 1);
  return t;
}

// ------------------------------------------------------------------ the pair's wrappers

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A shared-memory address of this CTA as that of CTA `rank`'s.
__device__ __forceinline__ uint32_t in_cta(uint32_t local, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}
// Arrivals on a barrier by its cluster address, by what they hand over:
// arrive_at, tensor memory alone, which the tcgen05 fences on both sides order around an arrival of any kind;
// hand_at, what the warp has read or written in its own CTA's shared memory (behind a proxy fence where the tensor
// cores read it), by a fence that is of that memory only;
// release_at, what it has stored in the other CTA's: it waits until those writes are performed there, some 1000 cycles.
__device__ __forceinline__ void arrive_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void hand_at(uint32_t bar) {
  asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
  arrive_at(bar);
}
__device__ __forceinline__ void release_at(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void store_at(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void store_at4(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Generic writes to either CTA's shared memory before the tensor cores' reads.
__device__ __forceinline__ void fence_proxy_async_cluster() {
  asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");
}

__device__ __forceinline__ void expect_tx_at(uint32_t bar, uint32_t bytes) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void tma_load_at(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
template <bool kCluster>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (kCluster)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  return ok != 0;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float lds_f(uint32_t a) { return __uint_as_float(lds32(a)); }
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) {
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void sts_f(uint32_t a, float v) { sts32(a, __float_as_uint(v)); }
__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  const uint4 v = lds128(a);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
// mbar_wait_warp by 32-bit addresses; kCluster: for barriers that the other CTA arrives on.  (A softmax thread
// has no register to spare for generic pointers.)
template <bool kCluster>
__device__ __forceinline__ void wait_at(uint32_t bar, uint32_t parity, uint32_t abort_at, int32_t* d_error) {
  uint32_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 1; !try_wait<kCluster>(bar, parity); ++i) {
    if ((i & 63) == 0) {
      uint32_t t;  // (the low half turns over after 4 s)
      asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
      if (t0 == 0) t0 = t;
      const bool late = t - t0 > static_cast<uint32_t>(kWaitNs);
      if (late || lds32(abort_at) != 0) {
        sts32(abort_at, 1);
        if (late && d_error) atomicOr(d_error, MLA_DEVERR_TIMEOUT);
        break;
      }
    }
  }
  __syncwarp();
}

// mbar_drain by a 32-bit address: it heeds no abort flag, but has a bound of its own.
__device__ __forceinline__ void drain_at(uint32_t bar, uint32_t parity, int32_t* d_error, uint64_t limit_ns) {
  const uint64_t t0 = global_timer_ns();
  while (!try_wait<true>(bar, parity)) {
    if (global_timer_ns() - t0 > limit_ns) {
      if (d_error) atomicOr(d_error, MLA_DEVERR_TIMEOUT);
      break;
    }
  }
}
__device__ __forceinline__ void store_unit(uint32_t a, const Unit& u) {
  sts32(a, u.b);
  sts32(a + 4, u.row0);
  sts32(a + 8, u.nrows);
  sts32(a + 12, u.first);
  sts32(a + 16, u.p_lo);
  sts32(a + 20, u.p_hi);
  sts32(a + 24, u.tiles);
}

__device__ __forceinline__ void mma2_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                        uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma2_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                        uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %2};\n\t"
      "mov.b64 b, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrives on this barrier of both CTAs once the products so far are complete.
__device__ __forceinline__ void commit_both(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\t"
      "mov.u16 m, 3;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          bar)
      : "memory");
}
__device__ __forceinline__ void tmem2_alloc(uint32_t* slot_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot_smem)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem2_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// ------------------------------------------------------------------ the kernel

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    paged_pair_kernel(const SharedParams p, const int groups, const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ CUtensorMap data_map, const __grid_constant__ CUtensorMap scale_map) {
  constexpr int NC = 32, HC = 8;  // rows of a softmax thread, of which it works on so many at a time
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  // This part's run: first unit, its item that the run begins with, items; the
  // cost of every run; the phase of the last copy of Q asked for.
  int* cut = reinterpret_cast<int*>(smem + L::kMiscOff + 8);
  uint32_t* votes = reinterpret_cast<uint32_t*>(smem + L::kMiscOff + 32);  // [2]
  int* warp_sum = reinterpret_cast<int*>(smem + L::kMiscOff + 48);                            // [warps]
  int* warp_most = reinterpret_cast<int*>(smem + L::kMiscOff + 176);                          // [warps]
  Unit* first_unit = reinterpret_cast<Unit*>(smem + L::kMiscOff + 304);  // the run's first
  Unit* now = reinterpret_cast<Unit*>(smem + L::kUnitOff);  // where the loader is; 32 bytes on, what comes next

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const uint32_t c = cluster_rank();
  const int part = blockIdx.x >> 1, parts = gridDim.x >> 1;

  if (tid < L::kNumBars) mbar_init(&bars[tid], L::arrivals(tid));
  if (tid == 0) {
    *abort_flag = 0;
    votes[0] = votes[1] = 0;
    cut[2] = 0;
    cut[4] = 0;
  }
  if (tid < L::kNumBars) {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == kValueWarp0) tmem2_alloc(tmem_slot, 512);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const uint32_t sm = smem_u32(smem);
  const auto bar = [&](int i) { return sm + L::kBarOff + i * 8; };
  const auto wait = [&](int i, uint32_t parity) { wait_at<false>(bar(i), parity, sm + L::kMiscOff + 4, p.d_error); };
  const auto wait2 = [&](int i, uint32_t parity) { wait_at<true>(bar(i), parity, sm + L::kMiscOff + 4, p.d_error); };
  const auto item_word = [&](uint32_t n, int k) {
    return static_cast<int>(lds32(sm + L::kInfoOff + (n % kInfoRing) * kItemBytes + k * 4));
  };
  const auto lead = [&](int i) { return in_cta(bar(i), 0); };  // a barrier of the first CTA

  const int num_groups = groups_in_order(p, tid, kThreads, blockIdx.x == 0), units = p.units;
  const auto unit_at = [&](int u, bool& bad) { return unit_of(p, groups, u, bad, num_groups); };

  // This CTA's half of a unit's Q arrives by TMA as bf16, K-major with 128-byte swizzle ...
  const auto request_q = [&](int row0) {
    expect_tx_at(bar(L::bQRaw), kMine * kD * 2);
#pragma unroll 1
    for (int k = 0; k < 8; ++k)
      tma_load_at(sm + L::kQOff + k * (kMine * 128), &q_map, k * 64, row0 + static_cast<int>(cluster_rank()) * kMine,
                  bar(L::bQRaw));
  };

  // The cut, as in paged.cu: units' costs, this part's run, and the unit it begins in.
  const int per = (units + kThreads - 1) / kThreads;
  const int u_a = min(units, tid * per), u_b = min(units, u_a + per);
  const auto cost_of = [](const Unit& t) { return t.tiles == 0 ? 0 : t.tiles + kUnitCost; };
  int mine = 0, most = 0;
  for (int u = u_a; u < u_b; ++u) {
    bool bad;
    const int cost = cost_of(unit_at(u, bad));
    mine += cost;
    most = max(most, cost);
    if (bad && blockIdx.x == 0 && p.d_error) atomicOr(p.d_error, MLA_DEVERR_BAD_LENGTH);
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (lane == 31) warp_sum[warp] = incl, warp_most[warp] = most;
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // the other CTA's barriers are there
  tc_fence_after();
  {
    const bool is_warp = lane < kThreads / 32;
    const int sum = is_warp ? warp_sum[lane] : 0;
    const int total = __reduce_add_sync(0xFFFFFFFFu, sum), before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sum : 0);
    most = __reduce_max_sync(0xFFFFFFFFu, is_warp ? warp_most[lane] : 0);
    const int share = (total + parts - 1) / parts;
    const bool whole = units <= parts && most <= share + kMergeCost;
    const int64_t from = static_cast<int64_t>(part) * share;
    const int g0 = static_cast<int>(min(from, static_cast<int64_t>(total)));
    const int g1 = static_cast<int>(min(from + share, static_cast<int64_t>(total)));
    const int excl = before + incl - mine;
    if (whole ? u_a <= part && part < u_b : g0 < g1 && excl <= g0 && g0 < excl + mine) {
      // Units up to the run's first one, then those that it goes on with.
      int at = excl, count = 0, row0 = 0;
      bool found = false;
      for (int u = whole ? part : u_a;; ++u) {
        bool bad;
        const Unit unit = unit_at(u, bad);
        const int cost = cost_of(unit);
        if (!found && !whole && at + cost <= g0) {
          at += cost;
          continue;
        }
        if (!found) {
          const int k = whole ? 0 : max(g0 - at - kUnitCost, 0);
          *first_unit = unit;
          *now = unit;
          cut[0] = u;
          cut[1] = k;
          cut[3] = share;
          row0 = unit.row0;
          count = -k;
          found = true;
          if (whole) {
            count = unit.tiles;
            break;
          }
        }
        count += max(min(at + kUnitCost + unit.tiles, g1) - (at + kUnitCost), 0);
        at += cost;
        if (at + kUnitCost >= g1) break;
      }
      count = max(count, 0);
      cut[2] = count;
      if (count > 0) request_q(row0);
    }
  }
  __syncthreads();

  // (Each role reads what it needs of all this again: a register that lives through
  // every role is one that the decode warps have not.)
  const auto run_items = [&] { return lds32(sm + L::kMiscOff + 16); };
  const auto tmem_base = [&] { return lds32(sm + L::kMiscOff); };
  if (run_items() == 0) {
    // Nothing for this pair.
  } else if (warp >= kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    const uint32_t items = run_items(), tmem = tmem_base(), c = cluster_rank();
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------------- loader
      // It alone walks the units; the others read what it found.  (The unit itself stays
      // in shared memory, for registers.)
      const uint32_t unit = sm + L::kUnitOff;
      const auto of_unit = [&](int field) { return static_cast<int>(lds32(unit + field * 4)); };
      enum { kB = 0, kRow0 = 1, kRows = 2, kLo = 4, kHi = 5, kTiles = 6 };
      int u = static_cast<int>(lds32(sm + L::kMiscOff + 8)), k = static_cast<int>(lds32(sm + L::kMiscOff + 12));
      bool mid = k > 0;  // the run begins inside its first unit
      uint32_t asked = 0, asked_foreign = 0;  // items whose pages were asked for
      int last_row = -1;  // this lane's page of the last item
      const auto page_at = [&](uint32_t dst, uint32_t full, int first_row) {  // this CTA's half and the scales
        expect_tx_at(full, first_row >= 0 ? L::kEntry : 0);
        if (first_row >= 0) {
          tma_load_at(dst, &data_map, static_cast<int>(c) * 128, first_row, full);
          tma_load_at(dst + L::kHalf, &scale_map, 256, first_row, full);
        }
      };
      const auto foreign = [&](uint32_t n, int first_row) {
        const bool ask = !__any_sync(0xFFFFFFFFu, lds32(sm + L::kMiscOff + 4) != 0);
        if (ask) ++asked_foreign;
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
          const uint32_t no = 2 * n + j, slot = no % L::kForeign;
          wait(L::bForeignFree + slot, ((no / L::kForeign) & 1) ^ 1);
          if (lane == static_cast<int>(c ^ 1) * 2 + j && ask)
            page_at(sm + L::kForeignOff + slot * L::kEntry, bar(L::bForeignFull + slot), first_row);
        }
      };
#pragma unroll 1
      for (uint32_t n = 0; n < items; ++n) {
        // Lane j < 4 looks after page j: 0 and 1 are the first CTA's own.
        int tokens = 0, first_row = -1;  // (-1: nothing of the page)
        bool bad = false;
        if (lane < 4) {
          const int pos = k * kStep + lane * kPage, end = of_unit(kHi) + 1, b = of_unit(kB);
          if (pos < end) {
            const int32_t* row = p.block_table + static_cast<int64_t>(b) * p.max_pages;
            if (b < 0) row = p.prefix_table + static_cast<int64_t>(-1 - b) * p.max_prefix_pages;
            const int page = load_i32(row + k * 4 + lane);
            if (page >= 0 && page < p.num_pages) {
              tokens = min(kPage, end - pos);
              first_row = page * kPage;
            } else {
              bad = true;
            }
          }
        }
        if (bad && c == 0 && p.d_error) atomicOr(p.d_error, MLA_DEVERR_BAD_INDEX);
        uint32_t counts = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) counts |= static_cast<uint32_t>(__shfl_sync(0xFFFFFFFFu, tokens, j)) << (8 * j);
        const int tiles = of_unit(kTiles);
        int flags = 0;
        if (counts == 0x40404040u && k * kStep + kStep - 1 <= of_unit(kLo)) flags |= kWhole;
        if (n == 0 || k == 0) flags |= kOpens;
        if (n + 1 == items || k + 1 == tiles) flags |= kCloses;
        if (!mid) flags |= kFromStart;
        if (k + 1 == tiles) flags |= kToEnd;
        int next_u = u;
        if (k + 1 == tiles && n + 1 < items) {
          // The next unit that has items (there is one, as items are left).
          Unit next;
          bool bad_len;
          do next = unit_at(++next_u, bad_len);
          while (next_u + 1 < units && next.tiles == 0);
          if (lane == 0) store_unit(unit + 32, next);
        }
        // After a wait that gave up nothing more is asked for.
        const bool ask = !__any_sync(0xFFFFFFFFu, lds32(sm + L::kMiscOff + 4) != 0);
        if (ask) ++asked;
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
          const uint32_t no = 2 * n + j, own = no % L::kOwn, oth = no % L::kOther;
          wait(L::bOwnFree + own, ((no / L::kOwn) & 1) ^ 1);
          if (j == 0 && lane == 0) {
            const uint32_t it = sm + L::kInfoOff + (n % kInfoRing) * kItemBytes;
            sts32(it, counts);
            sts32(it + 4, flags);
            sts32(it + 8, k);
            sts32(it + 12, u);
#pragma unroll 1
            for (int f = 0; f < kUnitWords; ++f) sts32(it + 16 + f * 4, lds32(unit + 32 + f * 4));
            arrive(bar(L::bInfo + n % kInfoRing));
          }
          wait(L::bOtherFree + oth, ((no / L::kOther) & 1) ^ 1);
          if (lane == static_cast<int>(c) * 2 + j && ask) {
            page_at(sm + L::kOwnOff + own * L::kEntry, bar(L::bOwnFull + own), first_row);
            const uint32_t full = bar(L::bOtherFull + oth);
            expect_tx_at(full, first_row >= 0 ? L::kHalf : 0);
            if (first_row >= 0)
              tma_load_at(sm + L::kOtherOff + oth * L::kHalf, &data_map, static_cast<int>(c ^ 1) * 128, first_row, full);
          }
        }
        // The other CTA's pages are values only, so they are asked for an item later: this CTA's own, which are keys
        // first, do not wait behind them.  (Not two items: then own page 1 of item n would wait for the values of own
        // page 0 of item n - 2, which in the second CTA come behind that item's foreign pages.)
        if (n > 0) foreign(n - 1, last_row);
        last_row = first_row;
        if ((flags & (kCloses | kFromStart)) == (kCloses | kFromStart) && lane == 0 && c == 0) {
          // What the merge does about this unit, which begins here: read its own slot, or join the pieces of parts
          // `part` .. last when this part's end cuts it.
          const int share = static_cast<int>(lds32(sm + L::kMiscOff + 20));
          const bool cut_off = k + 1 < tiles;
          const int last = part + (share - 1 + tiles - k - 1) / share;
          *reinterpret_cast<int4*>(p.ws_info + static_cast<int64_t>(u) * 4) = make_int4(cut_off ? u : -1, part, last, 0);
        }
        if (++k == tiles && n + 1 < items) {
          k = 0;
          mid = false;
          u = next_u;
          __syncwarp();
          if (lane < kUnitWords) sts32(unit + lane * 4, lds32(unit + 32 + lane * 4));
          __syncwarp();
          // Its Q on the way to L2, a few items before it is read.
          const uint8_t* src = reinterpret_cast<const uint8_t*>(p.q + static_cast<int64_t>(of_unit(kRow0)) * kD);
          const int to = min(of_unit(kRows), static_cast<int>(c + 1) * kMine) * 8;
          for (int line = static_cast<int>(c) * kMine * 8 + lane; line < to; line += 32)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(src + line * 128));
        }
      }
      foreign(items - 1, last_row);
      // Every copy has landed before the CTA may end (they have, unless a wait gave up).
      const uint32_t pages = 2 * asked;
      for (uint32_t i = pages > L::kOwn ? pages - L::kOwn : 0; i < pages; ++i)
        drain_at(bar(L::bOwnFull + i % L::kOwn), (i / L::kOwn) & 1, p.d_error, kWaitNs);
      for (uint32_t i = pages > L::kOther ? pages - L::kOther : 0; i < pages; ++i)
        drain_at(bar(L::bOtherFull + i % L::kOther), (i / L::kOther) & 1, p.d_error, kWaitNs);
      const uint32_t foreign_pages = 2 * asked_foreign;
      for (uint32_t i = foreign_pages > L::kForeign ? foreign_pages - L::kForeign : 0; i < foreign_pages; ++i)
        drain_at(bar(L::bForeignFull + i % L::kForeign), (i / L::kForeign) & 1, p.d_error, kWaitNs);
    } else if (warp == kScoreWarp) {
      // ---------------------------------------------------------------- S^T = K Q^T, both CTAs' tokens
      if (c == 0) {
        constexpr uint32_t idesc = idesc_f16(256, NR, false, false);
        const uint64_t q_desc = make_smem_desc(sm + L::kQOff, 16, 1024, kSwizzle128);
        const uint32_t q_lo = static_cast<uint32_t>(q_desc), q_hi = static_cast<uint32_t>(q_desc >> 32);
        uint32_t q_parity = 0;
#pragma unroll 1
        for (uint32_t n = 0; n < items; ++n) {
          wait2(L::bSFree, (n & 1) ^ 1);
#pragma unroll 1
          for (int q = 0; q < kD / L::kKDims; ++q) {
            const int slot = q % L::kKSlots;
            wait2(L::bKFull + slot, (q / L::kKSlots) & 1);
            if (q == 0) {
              wait(L::bInfo + n % kInfoRing, (n / kInfoRing) & 1);
              if (item_word(n, 1) & kOpens) {
                wait2(L::bQFull, q_parity);
                q_parity ^= 1;
              }
            }
            tc_fence_after();
            const uint32_t a = tmem + L::cK + slot * (L::kKDims / 2), b = q_lo + ((q * kMine * 128) >> 4);
#pragma unroll
            for (int j = 0; j < L::kKDims / 16; ++j)
              mma2_ts(tmem + L::cS, a + j * 8, b + ((j * 32) >> 4), q_hi, idesc, (q | j) != 0);
            commit_both(bar(L::bKFree + slot));
          }
          commit_both(bar(L::bSFull));
        }
        commit_both(bar(L::bDrain));
      }
    } else if (c == 0) {
      // ---------------------------------------------------------------- O^T += V^T P^T, a block of dims each
      const int block = warp - kValueWarp0;
      constexpr uint32_t idesc = idesc_f16(256, NR, true, true);
      constexpr uint32_t p_sbo = 8 * 2 * kMine;  // eight rows of P^T
      const uint64_t v_desc = make_smem_desc(sm + L::kVOff + block * (L::kVSlots * L::kVUnit),
                                             L::kVTokens * 128, 1024, kSwizzle128);
      const uint64_t p_desc = make_smem_desc(sm + L::kPOff, 16 * p_sbo, p_sbo, kSwizzle128);
      const uint32_t v_lo = static_cast<uint32_t>(v_desc), p_lo = static_cast<uint32_t>(p_desc);
      const uint32_t v_hi = static_cast<uint32_t>(v_desc >> 32), p_hi = static_cast<uint32_t>(p_desc >> 32);
      const uint32_t d = tmem + L::cO + block * NR;
      uint32_t o_parity = 1;
      constexpr int kUnits = kStep / L::kVTokens, kPageUnits = kPage / L::kVTokens;
#pragma unroll 1
      for (uint32_t n = 0; n < items; ++n) {
        bool opens = false;
#pragma unroll 1
        for (int at = 0; at < kUnits; ++at) {
          // (Either half of P has rows from both CTAs, so with it goes that O^T is rescaled in both.)
          if (at % (kUnits / 2) == 0) {
            wait2(L::bPFull + at / (kUnits / 2), n & 1);
          }
          if (at == 0) {
            wait(L::bInfo + n % kInfoRing, (n / kInfoRing) & 1);
            opens = (item_word(n, 1) & kOpens) != 0;
            if (opens) {
              wait2(L::bOFree, o_parity);
              o_parity ^= 1;
            }
          }
          const uint32_t vs = at % L::kVSlots;
          wait2(L::bVFull + block * L::kVSlots + vs, (at / L::kVSlots) & 1);
          tc_fence_after();
          const uint32_t a = v_lo + ((vs * L::kVUnit) >> 4), b = p_lo + (((page_at_step(at / kPageUnits) * kPageUnits + at % kPageUnits) * (L::kVTokens / 8) * p_sbo) >> 4);
#pragma unroll
          for (int j = 0; j < L::kVTokens / 16; ++j)
            mma2_ss(d, a + ((j * 2048) >> 4), v_hi, b + ((j * 2 * p_sbo) >> 4), p_hi, idesc, !(opens && at == 0 && j == 0));
          commit_both(bar(L::bVFree + block * L::kVSlots + vs));
          if (at % (kUnits / 2) == kUnits / 2 - 1) commit_both(bar(L::bPFree + at / (kUnits / 2)));
        }
      }
      commit_both(bar(L::bDrain));
    }
  } else if (warp >= kKWarp0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDecodeRegs));
    const uint32_t items = run_items(), tmem = tmem_base(), c = cluster_rank();
    if (warp < kVWarp0) {
      // ---------------------------------------------------------------- K: lane = token of this CTA's 128
      const int quad = warp & 3;
      const uint32_t tK = tmem + (static_cast<uint32_t>(quad * 32) << 16) + L::cK;
      const int row = (quad & 1) * 32 + lane;  // of the page
      const uint32_t data = row * 128, turn = (row & 7) * 16;
      const uint32_t scales = L::kHalf + row * 32, scale_turn = (row & 4) * 4;
#pragma unroll 1
      for (uint32_t n = 0; n < items; ++n) {
        const uint32_t no = 2 * n + (quad >> 1), own = no % L::kOwn, oth = no % L::kOther;
        const uint32_t mine_at = sm + L::kOwnOff + own * L::kEntry;
        const uint32_t other_at = sm + L::kOtherOff + oth * L::kHalf;
        wait(L::bOwnFull + own, (no / L::kOwn) & 1);
        wait(L::bOtherFull + oth, (no / L::kOther) & 1);
#pragma unroll 1
        for (int q = 0; q < kD / L::kKDims; ++q) {
          const int slot = q % L::kKSlots;
          const uint32_t src = ((q >> 2) == static_cast<int>(cluster_rank()) ? mine_at : other_at) + data, at = (q & 3) * 32;
          const uint32_t sc = lds32(mine_at + scales + ((q * 4) ^ scale_turn));
          // A fresh barrier counts as one whose phase 1 is over.
          wait2(L::bKFree + slot, ((q / L::kKSlots) & 1) ^ 1);
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < 2; ++k) {
            const uint4 raw = lds128(src + ((at + 16 * k) ^ turn));
            uint32_t o[16];
            decode32<false>(raw, (sc >> (16 * k)) & 0xFFFFu, o);
            tmem_st16(tK + slot * (L::kKDims / 2) + k * 16, o);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_at(lead(L::bKFull + slot));
        }
        if (lane == 0) {
          uint32_t again = 2 * n + (quad >> 1);  // (computed anew, for registers)
          asm volatile("" : "+r"(again));
          arrive(bar(L::bOwnFree + again % L::kOwn));
          arrive(bar(L::bOtherFree + again % L::kOther));
        }
      }
    } else {
      // ---------------------------------------------------------------- V: this CTA's 256 dims, two blocks of 128
      // Two warps a block, a unit of 32 tokens in turn; eight lanes cover eight
      // tokens, four times eight the block's 16-byte pieces.
      const int block = (warp - kVWarp0) & 1, odd = (warp - kVWarp0) >> 1;
      const int tok = lane & 7, piece = lane >> 3;
      const uint32_t data = odd * (32 * 128) + tok * 128 + (((block * 4 + piece) ^ tok) * 16);
      const uint32_t scales = L::kHalf + odd * (32 * 32) + tok * 32 +
                              (((static_cast<int>(c) * 2 + block) * 8 + piece * 2) ^ ((tok & 4) * 4));
      // The lane's first 16-byte unit of a 128-byte row, swizzled; unit j is at this ^ 16 j.
      const uint32_t unit0 = sm + L::kVOff + (block * L::kVSlots + odd) * L::kVUnit + (piece >> 1) * (L::kVTokens * 128) +
                             tok * 128 + (((piece & 1) * 4) ^ tok) * 16;
#pragma unroll 1
      for (uint32_t n = 0; n < items; ++n) {
#pragma unroll 1
        for (int at = 0; at < 4; ++at) {
          const int g = page_at_step(at);
          const bool own = (g >> 1) == static_cast<int>(cluster_rank());
          const uint32_t no = 2 * n + (g & 1), slot = own ? no % L::kOwn : no % L::kForeign;
          const uint32_t page = sm + (own ? L::kOwnOff : L::kForeignOff) + slot * L::kEntry;
          wait(own ? L::bOwnFull + slot : L::bForeignFull + slot, own ? (no / L::kOwn) & 1 : (no / L::kForeign) & 1);
          if (at == 0) wait(L::bInfo + n % kInfoRing, (n / kInfoRing) & 1);
          const int have = ((item_word(n, 0) >> (8 * g)) & 0xFF) - odd * 32 - tok;  // tokens below it are there
          wait2(L::bVFree + block * L::kVSlots + odd, (at & 1) ^ 1);
#pragma unroll 1
          for (int w = 0; w < 2; ++w) {
            uint4 raw[2];
            uint32_t sc[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              raw[i] = lds128(page + data + w * 2048 + i * 1024);
              sc[i] = lds16(page + scales + w * 512 + i * 256);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t o[16];
              decode32<true>(raw[i], w * 16 + i * 8 < have ? sc[i] : 0u, o);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                sts128((unit0 ^ (16 * j)) + w * 2048 + i * 1024, o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) hand_at(lead(L::bVFull + block * L::kVSlots + odd));
          if (lane == 0) arrive(bar(own ? L::bOwnFree + slot : L::bForeignFree + slot));
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const uint32_t items = run_items(), tmem = tmem_base(), c = cluster_rank();
    const auto other = [&](int i) { return in_cta(bar(i), c ^ 1); };  // a barrier of the other CTA
    const int side = tid >> 7, row = tid & 127;                  // token of this CTA's 128
    const int c0 = side * NC;                                    // first row of this thread
    const uint32_t tO = tmem + (static_cast<uint32_t>(row & 96) << 16) + L::cO;
    const uint32_t tS = tO - L::cO + L::cS + c0;
    // Where this thread's P goes: its rows' CTA, its token's row of P^T; 16-byte piece k is at this ^ 16 k.
    const uint32_t p_at = ((side >> 1) == static_cast<int>(c) ? sm + L::kPOff : in_cta(sm + L::kPOff, c ^ 1)) +
                          (static_cast<uint32_t>(c) * 128 + row) * 128 + (((side & 1) * 64) ^ ((row & 7) * 16));
    // The largest score whose exponent is within the slack, rounded down.
    const auto most_under = [](float m, float scale) { return __fadd_rd(m, __fdividef(kSlack, scale)); };

    // A unit's Q becomes scaled f16 in place, a row per warp at a time (lane = 16
    // dims); rows past the unit's become zeros.  Both CTAs get the scale.
    uint32_t turns = 0;  // bit 0: exchanges of maxima and sums, bit 1: pieces begun
    const auto convert_q = [&](uint32_t unit) {
      enum { kB = 0, kRow0 = 1, kRows = 2, kFirst = 3, kHi = 5 };
      const int nrows = static_cast<int>(lds32(unit + kRows * 4));
      // (Conversions go one ahead of the pieces begun, but for the first.)
      wait(L::bQRaw, (turns >> 1) & 1);
      const uint32_t base = sm + L::kQOff + (lane >> 2) * (kMine * 128);
      const uint32_t to = sm + L::kScaleOff + ((turns >> 1) & 1) * (NR * 4);
#pragma unroll 1
      for (int r = warp; r < kMine; r += kSoftmaxWarps) {
        const uint32_t off = r * 128 + (lane & 3) * 32;
        const uint32_t pa = base + swz<128>(off), pb = base + swz<128>(off + 16);
        const uint4 a = lds128(pa), b = lds128(pb);
        uint32_t wv[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        const int whole_r = static_cast<int>(c) * kMine + r;  // of the unit
        // The largest magnitude of the row, two values to a word.
        uint32_t two = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (whole_r >= nrows) wv[k] = 0;
          asm("max.u16x2 %0, %0, %1;" : "+r"(two) : "r"(wv[k] & 0x7FFF7FFFu));
        }
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, max(two >> 16, two & 0xFFFFu)) >> 7;
        // Largest value to [2^14, 2^15); nothing to scale in a row of zeros or of infinities.
        const int e = top == 0 || top == 255 ? 0 : max(static_cast<int>(top) - 127 - 14, -100);
        // A negative scale's sign goes into Q, so that the largest product is the largest score.
        const float up = copysignf(__uint_as_float(static_cast<uint32_t>(127 - e) << 23), p.scale_log2);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          wv[k] = pack_f16x2(__uint_as_float(wv[k] << 16) * up, __uint_as_float(wv[k] & 0xFFFF0000u) * up);
        sts128(pa, wv[0], wv[1], wv[2], wv[3]);
        sts128(pb, wv[4], wv[5], wv[6], wv[7]);
        if (lane == 0) {
          // Never 0 or infinite, so that no score times it is NaN (scores are below 2^36).
          float s = fminf(fabsf(p.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 + e) << 23), 3.0e38f);
          s = s == 0.f ? 1e-30f : s;
          sts_f(to + whole_r * 4, s);
          store_at(in_cta(to + whole_r * 4, c ^ 1), __float_as_uint(s));
        }
      }
      if (tid < NR) {
        sts_f(sm + L::kMinusMOff + tid * 4, -kNoMax);
        sts_f(sm + L::kMinusMostOff + tid * 4, -kNoMax);  // (any score is past it)
        const int b = static_cast<int>(lds32(unit + kB * 4)), row0 = static_cast<int>(lds32(unit + kRow0 * 4));
        sts32(sm + L::kHiOff + tid * 4, b < 0 ? lds32(unit + kHi * 4)
                                              : lds32(unit + kFirst * 4) + min(row0 - b * p.rows + tid, p.rows - 1) / p.h);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        hand_at(lead(L::bQFull));
        arrive(bar(L::bUnit));
        release_at(other(L::bUnit));
      }
    };
    // This thread's exponents of rows h .. h + HC - 1 in an item: scale * (score - m) + kPBias, the difference first,
    // as it is exact near m.
    const auto scale = [&] { return sm + L::kScaleOff + (((turns >> 1) & 1) ^ 1) * (NR * 4); };  // where this unit's lie
    const auto exponents = [&](int h, float (&y)[HC]) {
      uint32_t r[HC];
      tmem_ld<HC>(tS + h, r);
      const float2 bias = make_float2(kPBias, kPBias);
#pragma unroll
      for (int k = 0; k < HC / 4; ++k) {
        const float4 s = lds_f4(scale() + (c0 + h + 4 * k) * 4), m = lds_f4(sm + L::kMinusMOff + (c0 + h + 4 * k) * 4);
        const float2 a = make_float2(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1]));
        const float2 b = make_float2(__uint_as_float(r[4 * k + 2]), __uint_as_float(r[4 * k + 3]));
        const float2 u = __ffma2_rn(__fadd2_rn(a, make_float2(m.x, m.y)), make_float2(s.x, s.y), bias);
        const float2 v = __ffma2_rn(__fadd2_rn(b, make_float2(m.z, m.w)), make_float2(s.z, s.w), bias);
        y[4 * k] = u.x, y[4 * k + 1] = u.y, y[4 * k + 2] = v.x, y[4 * k + 3] = v.y;
      }
    };

    convert_q(sm + L::kMiscOff + 304);
    float l[NC];
#pragma unroll 1
    for (uint32_t n = 0; n < items; ++n) {
      wait(L::bInfo + n % kInfoRing, (n / kInfoRing) & 1);
      const int flags = item_word(n, 1);
      if (flags & kOpens) {
#pragma unroll
        for (int k = 0; k < NC; ++k) l[k] = 0.f;
        wait2(L::bUnit, (turns >> 1) & 1);  // the scales of all rows
        turns ^= 2;
      }
      wait2(L::bSFull, n & 1);
      tc_fence_after();
      // The piece's last scores are there, so its Q has been read: the next unit's may come.
      // (None after a wait that gave up: the last one asked for has to have landed at the end.)
      if ((flags & kCloses) && n + 1 < items && tid == 0 && lds32(sm + L::kMiscOff + 4) == 0) {
        request_q(item_word(n, 5));
        sts32(sm + L::kMiscOff + 24, lds32(sm + L::kMiscOff + 24) ^ 1);
      }
      if (!(flags & kWhole)) {
        // Scores of tokens that a row does not see become minus infinity.
        const int pos = item_word(n, 2) * kStep + static_cast<int>(c) * 128 + row;
        const bool there = (row & 63) < ((item_word(n, 0) >> (8 * (c * 2 + (row >> 6)))) & 0xFF);
#pragma unroll 1
        for (int h = 0; h < NC; h += 8) {
          uint32_t r[8];
          tmem_ld<8>(tS + h, r);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (!(there && pos <= static_cast<int>(lds32(sm + L::kHiOff + (c0 + h + k) * 4)))) r[k] = 0xFF800000u;
          tmem_st8(tS + h, r);
        }
        tmem_wait_st();
      }
      // The vote: does a score outgrow the slack, here or in the other CTA?
      float top = -INFINITY;
#pragma unroll 1
      for (int h = 0; h < NC; h += HC) {
        uint32_t r[HC];
        tmem_ld<HC>(tS + h, r);
#pragma unroll
        for (int k = 0; k < HC / 4; ++k) {
          const float4 m = lds_f4(sm + L::kMinusMostOff + (c0 + h + 4 * k) * 4);
          top = fmaxf(top, fmaxf(fmaxf(__uint_as_float(r[4 * k]) + m.x, __uint_as_float(r[4 * k + 1]) + m.y),
                                 fmaxf(__uint_as_float(r[4 * k + 2]) + m.z, __uint_as_float(r[4 * k + 3]) + m.w)));
        }
      }
      const uint32_t vote = sm + L::kMiscOff + 32 + (n & 1) * 4;
      const bool over = __any_sync(0xFFFFFFFFu, top > 0.f);
      if (lane == 0) {
        if (over) {
          sts32(vote, n + 1);
          store_at(in_cta(vote, c ^ 1), n + 1);
          release_at(other(L::bVote + (n & 1)));
        } else {
          hand_at(other(L::bVote + (n & 1)));
        }
        arrive(bar(L::bVote + (n & 1)));
      }
      wait2(L::bVote + (n & 1), (n >> 1) & 1);
      if (lds32(vote) == n + 1) {
        // Exact maxima of the item's rows, over this CTA's tokens, then over both's.
#pragma unroll 1
        for (int h = 0; h < NC; h += 8) {
          uint32_t r[8];
          float y[8];
          tmem_ld<8>(tS + h, r);
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] = __uint_as_float(r[k]);
          LaneReduce<8, 16>::run(y, lane, OpMax());
          if (lane % 4 == 0) sts_f(sm + L::kRedOff + ((row >> 5) * NR + c0 + h + column_of<8>(lane)) * 4, y[0]);
        }
        named_bar_sync(1, kSoftmaxThreads);
        bool moved = false;
        if (tid < NR) {
          const uint32_t red = sm + L::kRedOff + tid * 4, x = sm + L::kXMaxOff + tid * 4;
          const float m0 = fmaxf(fmaxf(lds_f(red), lds_f(red + NR * 4)), fmaxf(lds_f(red + NR * 8), lds_f(red + NR * 12)));
          store_at(in_cta(x + c * (NR * 4), c ^ 1), __float_as_uint(m0));
          __syncwarp();
          if (lane == 0) {
            arrive(bar(L::bXchg));
            release_at(other(L::bXchg));
          }
          wait2(L::bXchg, turns & 1);
          const float m = fmaxf(m0, lds_f(x + (c ^ 1) * (NR * 4)));
          const float minus_old = lds_f(sm + L::kMinusMOff + tid * 4), s = lds_f(scale() + tid * 4);
          float alpha = 1.f;
          // Every row's that has grown, as O^T is rescaled as a whole: the votes to come are fewer (64 query tokens x
          // 128 heads over 4096 tokens, scores of deviation 7: 120 us if only rows past the slack move, 105 so).
          if (m + minus_old > 0.f) {
            alpha = ex2_approx(-(m + minus_old) * s);
            moved = minus_old != -kNoMax;
            sts_f(sm + L::kMinusMOff + tid * 4, -m);
            sts_f(sm + L::kMinusMostOff + tid * 4, -most_under(m, s));
          }
          sts_f(sm + L::kAlphaOff + tid * 4, alpha);
        }
        turns ^= 1;
        if (any_of(2, kSoftmaxThreads, moved)) {
#pragma unroll
          for (int k = 0; k < NC; ++k) l[k] *= lds_f(sm + L::kAlphaOff + (c0 + k) * 4);
          // O^T follows, once the product before this one is complete.
          if (!(flags & kOpens)) {
            wait2(L::bPFree, (n & 1) ^ 1);
            wait2(L::bPFree + 1, (n & 1) ^ 1);
            tc_fence_after();
#pragma unroll 1
            for (int i = side; i < 2 * (NR / 8); i += 4) {
              const int at = (i / (NR / 8)) * NR + (i % (NR / 8)) * 8;
              uint32_t o[8];
              tmem_ld<8>(tO + at, o);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                o[k] = __float_as_uint(__uint_as_float(o[k]) * lds_f(sm + L::kAlphaOff + ((i % (NR / 8)) * 8 + k) * 4));
              tmem_st8(tO + at, o);
            }
            tmem_wait_st();
            // A product adds to all lanes of O^T: no warp hands its P over before all of it is rescaled here.
            tc_fence_before();
            named_bar_sync(1, kSoftmaxThreads);
            tc_fence_after();
          }
        }
      }
      uint32_t e[NC / 2];
#pragma unroll
      for (int h = 0; h < NC; h += HC) {
        float y[HC];
        exponents(h, y);
        if (h + HC == NC) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_at(lead(L::bSFree));
        }
#pragma unroll
        for (int k = 0; k < HC; k += 2) {
          const float a = ex2_approx(y[k]), b = ex2_approx(y[k + 1]);
          l[h + k] += a;
          l[h + k + 1] += b;
          e[(h + k) / 2] = pack_f16x2(a, b);
        }
      }
      // Row `row` of P^T (MN-major), when the last product has read this half of the buffer.
      wait2(L::bPFree + (row >> 6), (n & 1) ^ 1);
      tc_fence_before();
      if ((side >> 1) == static_cast<int>(c)) {
#pragma unroll
        for (int k = 0; k < NC / 8; ++k) sts128(p_at ^ (k * 16), e[4 * k], e[4 * k + 1], e[4 * k + 2], e[4 * k + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) hand_at(lead(L::bPFull + (row >> 6)));
      } else {
        // Four lanes' pieces are transposed among them, so that a store's lanes write 64 bytes of a token's row together
        // (16 bytes a row of 128 each they went one by one: 64 x 128 heads over a prefix of 16k tokens 277 us, 271 so).
#pragma unroll
        for (int m = 1; m <= 2; m *= 2) {
          const bool up = (lane & m) != 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k & m) continue;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t send = up ? e[4 * k + w] : e[4 * (k + m) + w];
              const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, send, m);
              if (up)
                e[4 * k + w] = got;
              else
                e[4 * (k + m) + w] = got;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int token = (row & ~3) + k;
          const uint32_t at = sm + L::kPOff + (c * 128 + token) * 128 + (((side & 1) * 64 + (lane & 3) * 16) ^ ((token & 7) * 16));
          store_at4(in_cta(at, c ^ 1), e[4 * k], e[4 * k + 1], e[4 * k + 2], e[4 * k + 3]);
        }
        fence_proxy_async_cluster();
        __syncwarp();
        if (lane == 0) release_at(lead(L::bPFull + (row >> 6)));
      }
      if (!(flags & kCloses)) continue;

      // The piece's end: row sums over this CTA's tokens, then both's, then O^T / l.
#pragma unroll
      for (int h = 0; h < NC; h += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = l[h + k];
        LaneReduce<8, 16>::run(v, lane, OpAdd());
        if (lane % 4 == 0) sts_f(sm + L::kRedOff + ((row >> 5) * NR + c0 + h + column_of<8>(lane)) * 4, v[0]);
      }
      named_bar_sync(1, kSoftmaxThreads);
      // Where the piece's rows go: slot 2 part + 1 if it begins its unit, 2 part if it goes on with it; a whole unit has a
      // slot of its own behind those.
      const auto first_row = [&] {  // (a row is 2 KB of a workspace, so 32 bits count them)
        const int u = min(max(item_word(n, 3), 0), units - 1);  // (after a wait that gave up it may be anything)
        const int at = static_cast<int>(blockIdx.x >> 1), all = static_cast<int>(gridDim.x >> 1);
        const bool whole = (flags & (kFromStart | kToEnd)) == (kFromStart | kToEnd);
        return (whole ? 2 * all + u : 2 * at + ((flags & kFromStart) ? 1 : 0)) * NR;
      };
      if (tid < NR) {
        const uint32_t red = sm + L::kRedOff + tid * 4, x = sm + L::kXSumOff + tid * 4;
        const float s0 = (lds_f(red) + lds_f(red + NR * 4)) + (lds_f(red + NR * 8) + lds_f(red + NR * 12));
        store_at(in_cta(x + c * (NR * 4), c ^ 1), __float_as_uint(s0));
        __syncwarp();
        if (lane == 0) {
          arrive(bar(L::bXchg));
          release_at(other(L::bXchg));
        }
        wait2(L::bXchg, turns & 1);
        const float there = lds_f(x + (c ^ 1) * (NR * 4));
        const float sum = c == 0 ? s0 + there : there + s0;
        sts_f(sm + L::kLinvOff + tid * 4, sum > 0.f ? 1.f / sum : 0.f);
        const float lse = sum > 0.f ? fmaf(-lds_f(sm + L::kMinusMOff + tid * 4), lds_f(scale() + tid * 4), log2f(sum) - kPBias) *
                                          0.6931471805599453f
                                    : -INFINITY;
        if (c == 0) p.ws_lse[first_row() + tid] = lse;
      }
      turns ^= 1;
      named_bar_sync(1, kSoftmaxThreads);
      // The next unit's Q goes in while the last product runs (this piece's scores are all done).
      if (n + 1 < items) convert_q(sm + L::kInfoOff + (n % kInfoRing) * kItemBytes + 16);
      wait2(L::bPFree, n & 1);
      wait2(L::bPFree + 1, n & 1);
      tc_fence_after();
      // Lane = dim, columns = rows.
      const int row0 = first_row();
#pragma unroll 1
      for (int i = side; i < 2 * (NR / 8); i += 4) {
        const int block = i / (NR / 8), cc = (i % (NR / 8)) * 8;
        const int d = static_cast<int>(c) * 256 + block * 128 + row;
        uint32_t o[8];
        tmem_ld<8>(tO + block * NR + cc, o);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 s = lds_f4(sm + L::kLinvOff + (cc + 4 * k) * 4);
          o[4 * k] = __float_as_uint(__uint_as_float(o[4 * k]) * s.x);
          o[4 * k + 1] = __float_as_uint(__uint_as_float(o[4 * k + 1]) * s.y);
          o[4 * k + 2] = __float_as_uint(__uint_as_float(o[4 * k + 2]) * s.z);
          o[4 * k + 3] = __float_as_uint(__uint_as_float(o[4 * k + 3]) * s.w);
        }
        float* dst = p.ws_o + static_cast<int64_t>(row0 + cc) * kD + d;
#pragma unroll
        for (int k = 0; k < 8; ++k) dst[k * kD] = __uint_as_float(o[k]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_at(lead(L::bOFree));
      named_bar_sync(1, kSoftmaxThreads);  // the row sums' arrays may change again
    }
  }

  tc_fence_before();
  __syncthreads();
  // The products are complete: the softmax warps have read the last of them, unless a wait gave up.  (A barrier of one
  // phase.  To follow an item's barriers here instead would be a wait that nothing waits for: a warp held up for two items
  // takes the phase two on for the one that it waits for.)
  if (warp == kScoreWarp && run_items() > 0) drain_at(bar(L::bDrain), 0, p.d_error, 2 * kWaitNs);
  // (Q's copies have landed long ago, unless a wait gave up.)
  if (tid == 0 && run_items() > 0) drain_at(bar(L::bQRaw), lds32(sm + L::kMiscOff + 24), p.d_error, kWaitNs);
  if (lds32(sm + L::kMiscOff + 4) != 0) __nanosleep(100000);  // after a wait that gave up: stores on their way have landed
  __syncthreads();
  cluster_sync_all();  // the other CTA is done with this one's shared memory, the products with both's
  if (warp == kValueWarp0) {
    tc_fence_after();
    tmem2_dealloc(tmem_base(), 512);
  }
}

}  // namespace

cudaError_t launch_shared_pair(const SharedParams& p, const PagedPlan& plan, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = max_dynamic_smem_once(configured, reinterpret_cast<const void*>(paged_pair_kernel), L::kAlloc);
  if (e != cudaSuccess) return e;
  EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  // Q viewed as rows of 512 bf16; a box is a CTA's rows x 64 dims, 128-byte swizzled.
  CUtensorMap q_map, data_map, scale_map;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(p.batch) * p.rows};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kD) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(kMine)};
  const cuuint32_t estr[2] = {1, 1};
  // The pool viewed as rows of 288 bytes; a box is a page's rows x 128 data bytes or x the 32 scale bytes.
  const cuuint64_t kv_dims[2] = {static_cast<cuuint64_t>(kRecFp4), static_cast<cuuint64_t>(p.num_pages) * kPage};
  const cuuint64_t kv_strides[1] = {static_cast<cuuint64_t>(kRecFp4)};
  const cuuint32_t data_box[2] = {128, kPage}, scale_box[2] = {32, kPage};
  if (enc(&q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(p.q), dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      enc(&data_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p.kv), kv_dims, kv_strides, data_box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      enc(&scale_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p.kv), kv_dims, kv_strides, scale_box,
          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3(2 * static_cast<unsigned>(plan.num_parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::kAlloc;
  e = cudaLaunchKernelEx(&cfg, paged_pair_kernel, p, plan.groups, q_map, data_map, scale_map);
  if (e != cudaSuccess) return e;
  return launch_shared_merge(p, plan, stream);
}

}  // namespace mla
