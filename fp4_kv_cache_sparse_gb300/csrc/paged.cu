// paged.cu -- attention over the pages of a cache held in 4 bits
// (include/mla.h, mla_paged_decode_fp4), on the tensor cores of sm_103a.
//
// For every query row (query token x head) r of a sequence, over the cached
// tokens j that its mask lets it see, each decoded from its FP4 record to a
// 512-dim latent k_j that is key and value:
//     x_rj = scale <q_r, k_j>,  m_r = running maximum,  p_rj = 2^(x_rj - m_r),
//     l_r = sum_j p_rj,  O_r = sum_j p_rj k_j,  out = O / l,  lse = m + log l.
//
// Work.  A unit is one group of up to NR (16, 32 or 64) query rows of one
// sequence; its items are the 128-token tiles that some row of it sees (the
// tiles of the sinks and of the window only).  All units in order, each a
// fixed cost and then its items, are cut into gridDim.x runs of equal cost, one
// per CTA (one CTA per SM), or go whole to one CTA each where they are few and
// short; the lengths are on the device, so every CTA derives the cut itself by a
// scan over the units.  A unit cut by a run's end leaves
// normalised fp32 partials, merged by a second kernel.
//
// One CTA, 28 warps:
//   softmax (8; 16 with 64 rows)  thread = token x some of the rows: scale,
//                      mask, lazy running maximum, P^T to shared memory, row
//                      sums in registers; at a unit's end the epilogue, before
//                      it the next unit's Q.
//   K decode (8; 4 with 64 rows)  raw FP4 -> f16 into tensor memory, lane =
//                      token: the A operand of S^T = K Q^T, a 128-dim quarter
//                      at a time.
//   V decode (8; 4 with 64 rows)  raw FP4 -> f16 into shared memory (128-byte
//                      swizzle), a dim quarter each, in units of 64 tokens (32
//                      with 64 rows): the MN-major A operand of
//                      O^T += V^T P^T.
//   loader (1)         each tile's two pages by tensor copies into a ring of
//                      raw pages, swizzled.
//   score issuer (1)   S^T, two tiles ahead of
//   value issuers (2)  O^T, two dim quarters each: with one, what it waits for
//                      holds up the other quarters (64 x 64 heads over 1k to
//                      8k tokens 80 us against 72, 32 x 16 over 64k 266
//                      against 227).
// Every role's loop is kept rolled and short: the roles together have to stay
// in the instruction cache (issue loops unrolled over a tile, in an earlier
// build: 32 x 16 heads over 64k tokens 450 us against 273).
//
// A tile is decoded twice (K to tensor memory, V to shared memory) because
// that is cheaper than the shared memory it saves: one f16 tile is 128 KB,
// and kept from S^T to O^T it would leave room for nothing beside it; raw it
// is 36 KB, so two to four tiles are in flight and neither copy of a quarter
// lives longer than the product that reads it.
//
// What bounds it: shared memory.  A tile's 128 KB of V are written and read,
// the raw tile is written once and read twice (108 KB), Q is read once and P
// four times as B operands.  With 16 rows that and the small operands are 3820
// accesses of 128 bytes a tile (2540 by the warps, 1280 by the tensor core),
// with 64 rows 5270 (3220 and 2050), in 4230 and 6000 cycles: nine tenths of
// what shared memory can do, and the tensor core is busy for 510 and 2050 of
// them.  So 32 x 16 heads over 64k tokens take 222 us (604 MB, 40 % of a copy's
// bandwidth), 64 x 64 heads over 1k to 8k tokens 63 us (38.7 GFLOP, 32 % of the
// bf16 rate), 32 x 2 x 128 heads with a window of 4096 107 us (35 %).  One tile
// alone takes 8 us, 2 of them until the cut is known, 4 until the first scores
// are there, and a merge 3 us more.  (Those are times of a call among others.
// Pairs beside the rules below are one call alone between two events, L2
// written over before it: some 5 us more.)
//
// Numbers.  e2m1 x e4m3 has at most 6 significant bits and lies in f16's
// range, so K and V are exact in f16.  Q (bf16) is scaled by a power of two
// per row to put its largest value in [2^14, 2^15) and is then exact in f16
// down to 2^-28 of that; below, 2^-39 of the row's largest value is lost.  P
// is f16 with the maximum at 2^5 (at most 2^15 with the lazy maximum's slack
// of 2^10): 11 bits down to 2^-19 of the largest weight, where bf16 has 8, and
// weights down to 2^-29 of it still count.  Sums, maxima and O are fp32.
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mla_device.cuh"
#include "mla_internal.h"
#include "mla_tensor.cuh"
#include "shared_units.cuh"

namespace mla {

namespace {

// A page in shared memory: its rows' data bytes in two halves of 128 bytes a
// row (128-byte swizzle), then their 32 scale bytes a row (32-byte swizzle).
// As one copy of the records, 288 bytes apart, rows of a warp met in the same
// banks (16 heads: 1620 cycles of loads a tile, 1200 so; 32 x 16 heads over 64k
// tokens 229 and 221 us, in the build that laid them out so).
constexpr int kPageBytes = kPage * kRecFp4;
constexpr int kHalfBytes = kPage * 128;
constexpr int kInfoRing = 8;
constexpr uint64_t kPagedWaitNs = 2000000000ull;  // 2 s per wait
// What a unit's Q and epilogue take, in tiles (64 sequences of 1k to 8k tokens,
// 64 heads: 72 us, with nothing 79).
constexpr int kUnitCost = 2;
// What the partials and the merge of cut units take, in tiles (100 sequences of
// 700 tokens, 64 heads: 33.5 us whole, 37.7 cut; 54 of 350, 22 heads: 22.1, 24.0).
constexpr int kMergeCost = 3;
// The running maximum may lag by 2^10: O is rescaled seldom (32 x 2 x 128 heads,
// window 4096: 107.3 us among others, 110.5 with 2^8; with none 64 x 64 heads
// take 88 us instead of 72).  P has room for that and for 5 bits above 1.
constexpr float kSlack = 10.f;
constexpr float kPBias = 5.f;                // P of the maximum is 2^5
constexpr float kNoMax = -3.0e38f;           // running maximum, unscaled, before any visible token

template <int NR>
struct PSmem {
  // A softmax thread holds NR / kSides rows: sums and P stay in registers (with
  // two sides of 64 rows they spill: 64 x 64 heads over 1k to 8k tokens 73.7 us, 72.4 so).
  static constexpr int kSides = NR == 64 ? 4 : 2;
  static constexpr int kSoftmaxWarps = 4 * kSides;
  // Decode warps of each kind: eight hide more latency (32 x 16 heads
  // over 64k tokens: 227 us against 268; 32 x 32 over 16k: 80 against 88), but with 64
  // rows the softmax has twice the warps and no registers are left for more.
  static constexpr int kDecodeWarps = NR == 64 ? 4 : 8;
  static constexpr int kKWarp0 = kSoftmaxWarps, kVWarp0 = kKWarp0 + kDecodeWarps, kLoadWarp = kVWarp0 + kDecodeWarps;
  static constexpr int kScoreWarp = kLoadWarp + 1, kValueWarp0 = kScoreWarp + 1;
  static constexpr int kValueWarps = 2;
  static constexpr int kThreads = (kValueWarp0 + kValueWarps) * 32;
  // Rings: raw pages, K quarters in tensor memory, a V unit (kVTokens x 128
  // dims, two chunks of 64 dims) for each dim quarter.  A page lives from its
  // load to the end of its V decode, about ten thousand cycles.  With 64 rows
  // Q leaves so little that V units of half the size, and six pages instead of
  // four, gain more than their barriers cost (32 x 2 x 128
  // heads, window 4096: 111.4 us against 114.7); with 16 they only cost (32 x 16
  // heads over 64k tokens: 282 us against 227).
  static constexpr int kVTokens = NR == 64 ? 32 : 64;
  static constexpr int kVUnitBytes = kVTokens * 128 * 2;
  static constexpr int kRaw = NR == 16 ? 7 : 6;
  static constexpr int kKRing = NR == 64 ? 2 : 4;
  static constexpr int kVRing = 4;
  static constexpr int kQBytes = NR * kD * 2;
  static constexpr int kPBytes = kTile * NR * 2;
  static constexpr int kQOff = 0;
  static constexpr int kVOff = kQOff + kQBytes;
  static constexpr int kPOff = kVOff + kVRing * kVUnitBytes;
  static constexpr int kRawOff = kPOff + kPBytes;
  static constexpr int kBarOff = kRawOff + kRaw * kPageBytes;
  static constexpr int kNumBars = 2 * kRaw + 2 * kKRing + 2 * kVRing + 8 + 4 + kInfoRing;
  static constexpr int kColOff = (kBarOff + kNumBars * 8 + 15) & ~15;  // per-row arrays
  // float minus_m[NR], minus_most[NR], alpha[NR], scale[NR], linv[NR]; int hi[NR], lo[NR]; float red[4][NR]
  static constexpr int kInfoOff = kColOff + 11 * NR * 4;
  static constexpr int kMiscOff = kInfoOff + kInfoRing * 16;
  static constexpr int kEnd = kMiscOff + 336;
  static constexpr int kAlloc = kEnd + 1024;
  static_assert(kAlloc <= 232448, "shared memory of one CTA");
  // Barrier indices.
  static constexpr int bRawFull = 0, bRawFree = bRawFull + kRaw, bKFull = bRawFree + kRaw, bKFree = bKFull + kKRing,
                       bVFull = bKFree + kKRing, bVFree = bVFull + kVRing, bSFull = bVFree + kVRing,
                       bSFree = bSFull + 2, bPFull = bSFree + 2, bPFree = bPFull + 2, bQFull = bPFree + 2,
                       bOFree = bQFull + 1, bDrain = bOFree + 1, bQRaw = bDrain + 1, bInfo = bQRaw + 1;
  static_assert(bInfo + kInfoRing == kNumBars, "barriers");
  // How many arrivals complete a phase of barrier i.
  __device__ static int arrivals(int i) {
    if (i >= bRawFree && i < bKFull) return kDecodeWarps / 2 + kDecodeWarps;  // half of the K warps, all V warps
    if (i >= bKFull && i < bKFree) return 4;
    if (i >= bVFull && i < bVFree) return kDecodeWarps / 4;
    if (i >= bSFree && i < bPFull) return kSoftmaxWarps;
    if (i >= bPFull && i < bPFree) return kSoftmaxWarps / 2;  // P^T goes by halves of the tile's tokens
    if (i >= bPFree && i < bQFull) return kValueWarps;
    if (i == bQFull || i == bOFree) return kSoftmaxWarps;
    if (i == bDrain) return 1 + kValueWarps;
    return 1;
  }
  // Tensor memory columns: O^T quarters, S^T buffers, K quarters.
  static constexpr int cO = 0, cS = 4 * NR, cK = 6 * NR;
  static_assert(cK + kKRing * 64 <= 512, "tensor memory");
};

// ------------------------------------------------------------------ geometry

// The tiles that a unit's rows see.
struct Unit {
  int b, row0, nrows;   // sequence, first row of the group, rows in it
  int first;            // position of the sequence's first query token
  int p_lo, p_hi;       // positions of the group's first and last query token
  int sink_tiles;       // tiles of the sinks that lie before the window's
  int win_tile;         // first tile of the window
  int start;            // first position of the window
  int tiles;            // at least 1 (a unit that sees nothing still writes its rows)
};

__device__ __forceinline__ int checked_len(const PagedParams& p, int b, bool& bad) {
  const int len = load_i32(p.seq_lens + b);
  bad = len < 0 || len > p.max_pages * kPage;
  return bad ? 0 : len;
}

// First position that the window of a query token at `at` holds.
__device__ __forceinline__ int window_start(const PagedParams& p, int at) {
  const int64_t from = static_cast<int64_t>(at) - p.window + 1;
  return p.window > 0 && from > 0 ? static_cast<int>(from) : 0;
}

template <bool kShared>
using Params = std::conditional_t<kShared, SharedParams, PagedParams>;

// A prefix unit: b is -1 - group, row0 counts from the batch's first row, every row sees every token.
template <int NR>
__device__ __forceinline__ Unit prefix_unit_of(const SharedParams& p, int v, int num_groups, bool& bad) {
  const PrefixUnit at = prefix_unit_at<NR>(p, v, num_groups);
  Unit t{};
  bad = at.bad;
  t.b = -1 - at.group;
  t.row0 = at.row0;
  t.nrows = at.nrows;
  t.first = t.p_lo = t.p_hi = at.len - 1;
  t.tiles = (at.len + kTile - 1) / kTile;
  return t;
}

template <int NR, bool kShared>
__device__ __forceinline__ Unit unit_of(const Params<kShared>& p, int groups, int u, bool& bad, int num_groups) {
  if constexpr (kShared) {
    if (u >= p.batch * groups) return prefix_unit_of<NR>(p, u - p.batch * groups, num_groups, bad);
  }
  Unit t;
  t.b = u / groups;
  t.row0 = (u - t.b * groups) * NR;
  t.nrows = min(NR, p.rows - t.row0);
  const int len = checked_len(p, t.b, bad);
  t.first = len - p.s;
  t.p_lo = t.first + t.row0 / p.h;
  t.p_hi = t.first + (t.row0 + t.nrows - 1) / p.h;
  const int end = max(t.p_hi + 1, 0);
  t.start = window_start(p, t.p_lo);
  t.start = min(t.start, end);
  t.win_tile = t.start / kTile;
  t.sink_tiles = min((min(p.sinks, end) + kTile - 1) / kTile, t.win_tile);
  t.tiles = max(t.sink_tiles + (end + kTile - 1) / kTile - t.win_tile, 1);
  return t;
}

__device__ __forceinline__ int tile_of(const Unit& u, int k) {
  return k < u.sink_tiles ? k : u.win_tile + (k - u.sink_tiles);
}

// What the loader tells the other warps of an item: {tokens of page 0 |
// tokens of page 1 << 8 | flags << 16, tile, unit, -}.  A piece is the part of
// a unit that lies in this CTA's run.
enum : int {
  kOpens = 1 << 16,      // first item of a piece
  kCloses = 2 << 16,     // last item of a piece
  kFromStart = 4 << 16,  // the piece begins with its unit
  kToEnd = 8 << 16,      // the piece ends with its unit
  kWhole = 16 << 16      // every row sees every token
};
__device__ __forceinline__ bool token_there(int info, int row) {
  return (row & 63) < ((info >> (row >= 64 ? 8 : 0)) & 0xFF);
}

// ------------------------------------------------------------------ small wrappers

__device__ __forceinline__ void wait_for(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int32_t* d_error) {
  mbar_wait_warp(bar, parity, abort_flag, d_error, kPagedWaitNs);
}

// ------------------------------------------------------------------ the kernel

// kShared: sequences in groups that share a prefix (mla_paged_shared_decode_fp4).
// After the units of the sequences' own tokens come those of the prefixes, NR
// rows of a group at a time whichever sequences they belong to; every unit
// leaves partials, which launch_shared_merge joins.
template <int NR, bool kShared>
__global__ void __launch_bounds__(PSmem<NR>::kThreads, 1)
    paged_decode_kernel(const Params<kShared> p, const int groups, const __grid_constant__ CUtensorMap q_map,
                        const __grid_constant__ CUtensorMap data_map, const __grid_constant__ CUtensorMap scale_map) {
  using L = PSmem<NR>;
  constexpr int NC = NR / L::kSides;    // rows of a softmax thread
  constexpr bool kKeep = NR == 16;
  constexpr int HC = NR == 64 ? 16 : 8;  // of which it works on so many at a time (registers)
  constexpr int kPagedThreads = L::kThreads, kSoftmaxWarps = L::kSoftmaxWarps;
  constexpr int kKWarp0 = L::kKWarp0, kVWarp0 = L::kVWarp0, kLoadWarp = L::kLoadWarp;
  constexpr int kScoreWarp = L::kScoreWarp, kValueWarp0 = L::kValueWarp0;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + L::kQOff;
  uint8_t* sV = smem + L::kVOff;
  uint8_t* sP = smem + L::kPOff;
  uint8_t* sRaw = smem + L::kRawOff;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  float* c_minus_m = reinterpret_cast<float*>(smem + L::kColOff);  // minus the running maximum of the unscaled scores
  float* c_minus_most = c_minus_m + NR;  // minus the largest score that P has room for under that maximum
  float* c_alpha = c_minus_most + NR;
  float* c_scale = c_alpha + NR;
  float* c_linv = c_scale + NR;
  int* c_hi = reinterpret_cast<int*>(c_linv + NR);
  int* c_lo = c_hi + NR;
  float* red = reinterpret_cast<float*>(c_lo + NR);
  int4* info = reinterpret_cast<int4*>(smem + L::kInfoOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  // This part's run: first unit, its item that the run begins with, items; the
  // cost of every run; the phase of the last copy of Q asked for.
  int* cut = reinterpret_cast<int*>(smem + L::kMiscOff + 8);
  int* warp_sum = reinterpret_cast<int*>(smem + L::kMiscOff + 32);    // [warps]
  int* warp_most = reinterpret_cast<int*>(smem + L::kMiscOff + 160);  // [warps]
  Unit* first_unit = reinterpret_cast<Unit*>(smem + L::kMiscOff + 288);  // the run's first

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int part = blockIdx.x;

  if (tid < L::kNumBars) mbar_init(&bars[tid], L::arrivals(tid));
  if (tid == 0) {
    *abort_flag = 0;
    cut[2] = 0;
    cut[4] = 0;
  }
  if (tid < L::kNumBars) {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == kValueWarp0) tmem_alloc(tmem_slot, 512);

  // Launched as a programmatic dependent: what comes before this line runs
  // beside the end of the stream's previous kernel, nothing after it does.
  // (That kernel may write the lengths and tables, hence load_i32.)
  asm volatile("griddepcontrol.wait;" ::: "memory");

  int num_groups = 0;
  if constexpr (kShared) {
    num_groups = groups_in_order(p, tid, kPagedThreads, part == 0);
  }

  // A unit's Q arrives by TMA as bf16, K-major with 128-byte swizzle ...
  const auto request_q = [&](int u) {
    int b = u / groups, y = b * p.rows + (u - b * groups) * NR;
    if constexpr (kShared) {
      bool bad;
      if (u >= p.batch * groups) y = prefix_unit_of<NR>(p, u - p.batch * groups, num_groups, bad).row0;
    }
    expect_tx(&bars[L::bQRaw], L::kQBytes);
#pragma unroll 1
    for (int c = 0; c < 8; ++c) tma_load_2d(sQ + c * (NR * 128), &q_map, c * 64, y, &bars[L::bQRaw]);
  };

  // The cut: items of all units, this part's run, and the unit it begins in.
  int units = p.batch * groups;
  if constexpr (kShared) units = p.units;
  const int per = (units + kPagedThreads - 1) / kPagedThreads;
  const int u_a = min(units, tid * per), u_b = min(units, u_a + per);
  const auto cost_of = [](const Unit& t) { return kShared && t.tiles == 0 ? 0 : t.tiles + kUnitCost; };
  int mine = 0, most = 0;
  Unit unit{};  // this thread's last, which is its only one unless units are very many
  for (int u = u_a; u < u_b; ++u) {
    bool bad;
    unit = unit_of<NR, kShared>(p, groups, u, bad, num_groups);
    const int cost = cost_of(unit);
    mine += cost;
    most = max(most, cost);
    if (bad && part == 0 && p.d_error) atomicOr(p.d_error, MLA_DEVERR_BAD_LENGTH);
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (lane == 31) warp_sum[warp] = incl, warp_most[warp] = most;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const bool is_warp = lane < kPagedThreads / 32;
  const int sum = is_warp ? warp_sum[lane] : 0;
  const int total = __reduce_add_sync(0xFFFFFFFFu, sum), before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sum : 0);
  most = __reduce_max_sync(0xFFFFFFFFu, is_warp ? warp_most[lane] : 0);
  {
    const int share = (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    // Short units of about one length, no more than parts: one a part, for
    // cutting them would cost more than it spreads.
    const bool whole = units <= static_cast<int>(gridDim.x) && most <= share + kMergeCost;
    const int64_t from = static_cast<int64_t>(part) * share;
    const int g0 = static_cast<int>(min(from, static_cast<int64_t>(total)));
    const int g1 = static_cast<int>(min(from + share, static_cast<int64_t>(total)));
    // A unit takes kUnitCost, then one for each of its tiles.  The run begins
    // in the unit whose last tile lies at or past g0; the thread that summed
    // that unit counts the run's tiles.
    const int excl = before + incl - mine;
    if (whole ? u_a <= part && part < u_b : g0 < g1 && excl <= g0 && g0 < excl + mine) {
      int at = excl, u = whole ? part : u_a;
      bool bad;
      if (per > 1) unit = unit_of<NR, kShared>(p, groups, u, bad, num_groups);
      while (!whole && at + cost_of(unit) <= g0) {
        at += cost_of(unit);
        unit = unit_of<NR, kShared>(p, groups, ++u, bad, num_groups);
      }
      const int k = whole ? 0 : max(g0 - at - kUnitCost, 0);
      int count = unit.tiles;
      *first_unit = unit;
      cut[0] = u;
      cut[1] = k;
      cut[3] = share;
      if (!whole) {
        int tiles = unit.tiles, next = u;
        count = max(min(at + kUnitCost + tiles, g1) - (at + kUnitCost + k), 0);
        for (at += kUnitCost + tiles; at + kUnitCost < g1; at += kShared && tiles == 0 ? 0 : kUnitCost + tiles) {
          tiles = unit_of<NR, kShared>(p, groups, ++next, bad, num_groups).tiles;
          count += min(at + kUnitCost + tiles, g1) - (at + kUnitCost);
        }
      }
      cut[2] = count;
      if (count > 0) request_q(u);
    }
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  const uint32_t items = static_cast<uint32_t>(cut[2]);

  if (items == 0) {
    if (tid == 0 && !(kShared || p.info_by_unit)) p.ws_info[part * 4] = -1;
  } else {

    if (warp == kLoadWarp) {
      // ---------------------------------------------------------------- loader
      // It alone walks the units; the others read what it found.
      int u = cut[0], k = cut[1];
      const bool mid = k > 0;  // the run begins inside its first unit
      const int u_first = u;
      bool bad_len;
      Unit unit = *first_unit;
      int slot = 0;
      uint32_t parity = 1, asked = 0;  // pages asked for
      for (uint32_t n = 0; n < items; ++n) {
        const int tile = tile_of(unit, k);
        const int end = unit.p_hi + 1;
        // Lane j < 2 looks after page j of the tile: copied up to the last
        // visible token, not at all when the window and the sinks leave it out.
        int tokens = 0;
        bool bad = false;
        int first_row = 0;
        if (lane < 2) {
          const int pos = tile * kTile + lane * kPage;
          const bool seen = pos < end && (pos + kPage > unit.start || pos < p.sinks);
          if (seen) {
            const int32_t* row = p.block_table + static_cast<int64_t>(unit.b) * p.max_pages;
            if constexpr (kShared) {
              if (unit.b < 0) row = p.prefix_table + static_cast<int64_t>(-1 - unit.b) * p.max_prefix_pages;
            }
            const int page = load_i32(row + tile * 2 + lane);
            if (page >= 0 && page < p.num_pages) {
              tokens = min(kPage, end - pos);
              first_row = page * kPage;
            } else {
              bad = true;
            }
          }
        }
        if (bad && p.d_error) atomicOr(p.d_error, MLA_DEVERR_BAD_INDEX);
        const int t0 = __shfl_sync(0xFFFFFFFFu, tokens, 0), t1 = __shfl_sync(0xFFFFFFFFu, tokens, 1);
        int word = t0 | (t1 << 8);
        const int t_end = tile * kTile + kTile - 1;
        if (t0 + t1 == kTile && t_end <= unit.p_lo &&
            (p.window == 0 || tile * kTile > unit.p_hi - p.window || t_end < p.sinks))
          word |= kWhole;
        if (n == 0 || k == 0) word |= kOpens;
        if (n + 1 == items || k + 1 == unit.tiles) word |= kCloses;
        // A piece begins with its unit unless the run's first item lies inside the unit.
        if (!(mid && u == u_first)) word |= kFromStart;
        if (k + 1 == unit.tiles) word |= kToEnd;
        int next_u = u + 1;
        Unit next_unit;
        if constexpr (kShared) {
          // The next unit that has tiles (there is one, as items are left).
          if (k + 1 == unit.tiles && n + 1 < items) {
            next_unit = unit_of<NR, true>(p, groups, next_u, bad_len, num_groups);
            while (next_unit.tiles == 0 && next_u + 1 < units)
              next_unit = unit_of<NR, true>(p, groups, ++next_u, bad_len, num_groups);
          }
        }
#pragma unroll 1
        for (int j = 0; j < 2; ++j) {
          wait_for(&bars[L::bRawFree + slot], parity, abort_flag, p.d_error);
          if (j == 0 && lane == 0) {
            info[n % kInfoRing] = make_int4(word, tile, u, kShared ? next_u : 0);
            mbar_arrive(&bars[L::bInfo + n % kInfoRing]);
          }
          // After a wait that gave up nothing more is asked for.
          const bool ask = !__any_sync(0xFFFFFFFFu, *abort_flag);
          if (ask) ++asked;
          if (lane == j && ask) {
            uint64_t* bar = &bars[L::bRawFull + slot];
            uint8_t* dst = sRaw + slot * kPageBytes;
            expect_tx(bar, tokens > 0 ? kPageBytes : 0);
            if (tokens > 0) {
              tma_load_2d(dst, &data_map, 0, first_row, bar);
              tma_load_2d(dst + kHalfBytes, &data_map, 128, first_row, bar);
              tma_load_2d(dst + 2 * kHalfBytes, &scale_map, 256, first_row, bar);
            }
          }
          if (++slot == L::kRaw) slot = 0, parity ^= 1;
        }
        if ((word & (kCloses | kFromStart)) == (kCloses | kFromStart) && lane == 0) {
          // What the merge does about this unit, which begins here: nothing, or
          // join the pieces of parts `part` .. last when this part's end cuts it.
          const bool merges = k + 1 < unit.tiles;
          const int last = part + (cut[3] - 1 + unit.tiles - k - 1) / cut[3];
          if (kShared || p.info_by_unit)
            *reinterpret_cast<int4*>(p.ws_info + u * 4) = make_int4(merges ? u : -1, part, last, 0);
          else if (n + 1 == items)
            *reinterpret_cast<int4*>(p.ws_info + part * 4) = make_int4(merges ? u : -1, part, last, 0);
        } else if (n + 1 == items && lane == 0 && !(kShared || p.info_by_unit)) {
          p.ws_info[part * 4] = -1;
        }
        if (++k == unit.tiles && n + 1 < items) {
          k = 0;
          if constexpr (kShared) {
            unit = next_unit;
            u = next_u;
          } else {
            unit = unit_of<NR, false>(p, groups, ++u, bad_len, 0);
          }
          // Its Q on the way to L2, a few tiles before it is read.
          const uint8_t* next = reinterpret_cast<const uint8_t*>(
              p.q + (kShared && unit.b < 0 ? static_cast<int64_t>(unit.row0)
                                           : static_cast<int64_t>(unit.b) * p.rows + unit.row0) * kD);
          for (int line = lane; line < unit.nrows * 8; line += 32)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(next + line * 128));
        }
      }
      // Every copy has landed before the CTA may end (they have, unless a wait gave up).
      for (uint32_t i = asked > L::kRaw ? asked - L::kRaw : 0; i < asked; ++i)
        mbar_drain(&bars[L::bRawFull + i % L::kRaw], (i / L::kRaw) & 1, p.d_error, kPagedWaitNs);
    } else if (warp >= kKWarp0 && warp < kVWarp0) {
      // ---------------------------------------------------------------- K: lane = token
      // Four warps, one for each quadrant of tensor memory lanes, decode a
      // 128-dim quarter; of eight, two teams take quarters in turn.  (What
      // stands in rows past the visible tokens only makes masked scores.)
      constexpr int kTeams = L::kDecodeWarps / 4;
      const int quad = warp & 3, team = (warp - kKWarp0) >> 2;
      const uint32_t tK = tmem + (static_cast<uint32_t>(quad * 32) << 16) + L::cK;
      const int row = (quad & 1) * 32 + lane;  // of the page
      const uint32_t rows = smem_u32(sRaw) + row * 128, turn = (row & 7) * 16;
      const uint32_t scales = smem_u32(sRaw) + 2 * kHalfBytes + row * 32, scale_turn = (row & 4) * 4;
      int slot = quad >> 1;  // the warp's page of the tile
      uint32_t raw_parity = 0;
#pragma unroll 1
      for (uint32_t n = 0; n < items; ++n) {
        wait_for(&bars[L::bRawFull + slot], raw_parity, abort_flag, p.d_error);
#pragma unroll 1
        for (int qq = team; qq < 4; qq += kTeams) {
          const int ks = qq % L::kKRing;
          const uint32_t parity = (L::kKRing == 4 ? n : static_cast<uint32_t>(qq / L::kKRing)) & 1;
          const uint32_t src = rows + slot * kPageBytes + (qq >> 1) * kHalfBytes, at = (qq & 1) * 64;
          const uint2 sc = lds64(scales + slot * kPageBytes + ((qq * 8) ^ scale_turn));
          uint4 data[2] = {lds128(src + (at ^ turn)), lds128(src + ((at + 16) ^ turn))};
          // A fresh barrier counts as one whose phase 1 is over.
          wait_for(&bars[L::bKFree + ks], parity ^ 1, abort_flag, p.d_error);
          tc_fence_after();
          const uint32_t t = tK + ks * 64;
#pragma unroll 1
          for (int hh = 0; hh < 2; ++hh) {
            const uint32_t s = hh ? sc.y : sc.x;
            uint32_t o[16];
            decode32<false>(data[0], s & 0xFFFFu, o);
            tmem_st16(t + hh * 32, o);
            if (hh == 0) data[0] = lds128(src + ((at + 32) ^ turn));
            decode32<false>(data[1], s >> 16, o);
            tmem_st16(t + hh * 32 + 16, o);
            if (hh == 0) data[1] = lds128(src + ((at + 48) ^ turn));
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[L::bKFull + ks]);
        }
        if (lane == 0) mbar_arrive(&bars[L::bRawFree + slot]);
        if ((slot += 2) >= L::kRaw) slot -= L::kRaw, raw_parity ^= 1;
      }
    } else if (warp >= kVWarp0 && warp < kLoadWarp) {
      // ---------------------------------------------------------------- V: shared memory
      // A warp owns one dim quarter (of eight, two share it, half of a unit's
      // tokens each).  Eight lanes cover eight tokens, four times eight the
      // quarter's 16-byte pieces: swizzled both ways, so free of bank conflicts.
      constexpr int kShare = L::kDecodeWarps / 4;
      const int qq = (warp - kVWarp0) & 3;
      const int tok = lane & 7, piece = lane >> 3;
      const int first = ((warp - kVWarp0) >> 2) * (L::kVTokens / kShare) + tok;  // this lane's first record of a unit
      const uint32_t rows =
          smem_u32(sRaw) + (qq >> 1) * kHalfBytes + first * 128 + ((((qq & 1) * 4 + piece) ^ tok) * 16);
      const uint32_t scales = smem_u32(sRaw) + 2 * kHalfBytes + first * 32 + ((qq * 8 + piece * 2) ^ ((tok & 4) * 4));
      const uint32_t dst = smem_u32(sV) + qq * L::kVUnitBytes + (piece >> 1) * (L::kVTokens * 128) + first * 128;
      // The lane's first 16-byte unit of a 128-byte row, swizzled; unit j is at this ^ 16 j.
      const uint32_t unit0 = dst + (((piece & 1) * 4) ^ tok) * 16;
      int slot = 0;
      uint32_t raw_parity = 0;
#pragma unroll 1
      for (uint32_t n = 0; n < items; ++n) {
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          wait_for(&bars[L::bRawFull + slot], raw_parity, abort_flag, p.d_error);
          const int have = ((info[n % kInfoRing].x >> (8 * half)) & 0xFF) - first;  // rows of this lane below it are there
          constexpr int kSteps = L::kVTokens / kShare / 8, kAtOnce = kSteps < 4 ? kSteps : 4;
          constexpr int kUnits = kPage / L::kVTokens;
#pragma unroll 1
          for (int w = 0; w < kUnits; ++w) {
#pragma unroll 1
            for (int i0 = 0; i0 < kSteps; i0 += kAtOnce) {
              uint4 data[kAtOnce];
              uint32_t sc[kAtOnce];
              const uint32_t page = slot * kPageBytes, skip = w * L::kVTokens + i0 * 8;
#pragma unroll
              for (int i = 0; i < kAtOnce; ++i) {
                data[i] = lds128(rows + page + (skip + i * 8) * 128);
                sc[i] = lds16(scales + page + (skip + i * 8) * 32);
              }
              if (i0 == 0) wait_for(&bars[L::bVFree + qq], kUnits == 2 ? w ^ 1 : half ^ 1, abort_flag, p.d_error);
#pragma unroll
              for (int i = 0; i < kAtOnce; ++i) {
                uint32_t o[16];
                decode32<true>(data[i], w * L::kVTokens + (i0 + i) * 8 < have ? sc[i] : 0u, o);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  sts128((unit0 ^ (16 * j)) + (i0 + i) * 1024, o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[L::bVFull + qq]);
          }
          if (lane == 0) mbar_arrive(&bars[L::bRawFree + slot]);
          if (++slot == L::kRaw) slot = 0, raw_parity ^= 1;
        }
      }
    } else if (warp == kScoreWarp) {
      // ---------------------------------------------------------------- S^T = K Q^T
      constexpr uint32_t idesc = idesc_f16(128, NR, false, false);
      const uint64_t q_desc = make_smem_desc(smem_u32(sQ), 16, 1024, kSwizzle128);
      const uint32_t q_lo = static_cast<uint32_t>(q_desc);
      const uint32_t q_hi = static_cast<uint32_t>(q_desc >> 32);
      uint32_t q_parity = 0;
#pragma unroll 1
      for (uint32_t n = 0; n < items; ++n) {
        const uint32_t d = tmem + L::cS + (n & 1) * NR;
        wait_for(&bars[L::bSFree + (n & 1)], ((n >> 1) & 1) ^ 1, abort_flag, p.d_error);
#pragma unroll 1
        for (int qq = 0; qq < 4; ++qq) {
          const int ks = qq % L::kKRing;
          const uint32_t parity = (L::kKRing == 4 ? n : static_cast<uint32_t>(qq / L::kKRing)) & 1;
          wait_for(&bars[L::bKFull + ks], parity, abort_flag, p.d_error);
          if (qq == 0 && (info[n % kInfoRing].x & kOpens)) {
            wait_for(&bars[L::bQFull], q_parity, abort_flag, p.d_error);
            q_parity ^= 1;
          }
          tc_fence_after();
          const uint32_t a = tmem + L::cK + ks * 64, b = q_lo + ((2 * qq * NR * 128) >> 4);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            mma_f16_ts(d, a + j * 8, b + (((j >> 2) * NR * 128 + (j & 3) * 32) >> 4), q_hi, idesc, (qq | j) != 0);
          commit_one(&bars[L::bKFree + ks]);
        }
        commit_one(&bars[L::bSFull + (n & 1)]);
      }
      commit_one(&bars[L::bDrain]);
      mbar_drain(&bars[L::bDrain], 0, p.d_error, kPagedWaitNs);
    } else if (warp >= kValueWarp0) {
      // ---------------------------------------------------------------- O^T += V^T P^T
      // Two warps, two dim quarters each: what waiting for one costs the other issues through.
      constexpr int kMine = 4 / L::kValueWarps;
      const int q0 = (warp - kValueWarp0) * kMine;
      constexpr uint32_t idesc = idesc_f16(128, NR, true, true);
      constexpr uint32_t p_sbo = 8 * 2 * NR;  // eight rows of P^T
      constexpr uint32_t p_swz = NR == 64 ? kSwizzle128 : (NR == 32 ? kSwizzle64 : kSwizzle32);
      const uint64_t v_desc = make_smem_desc(smem_u32(sV), L::kVTokens * 128, 1024, kSwizzle128);
      const uint64_t p_desc = make_smem_desc(smem_u32(sP), 16 * p_sbo, p_sbo, p_swz);
      const uint32_t v_lo = static_cast<uint32_t>(v_desc), p_lo = static_cast<uint32_t>(p_desc);
      const uint32_t v_hi = static_cast<uint32_t>(v_desc >> 32), p_hi = static_cast<uint32_t>(p_desc >> 32);
      uint32_t o_parity = 1;
#pragma unroll 1
      for (uint32_t n = 0; n < items; ++n) {
        bool opens = false;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          wait_for(&bars[L::bPFull + half], n & 1, abort_flag, p.d_error);
          if (half == 0) {
            opens = (info[n % kInfoRing].x & kOpens) != 0;
            if (opens) {
              wait_for(&bars[L::bOFree], o_parity, abort_flag, p.d_error);
              o_parity ^= 1;
            }
          }
          constexpr int kUnits = kPage / L::kVTokens;
#pragma unroll 1
          for (int w = 0; w < kUnits * kMine; ++w) {
            const int qq = q0 + w % kMine, at = half * kUnits + w / kMine;
            wait_for(&bars[L::bVFull + qq], at & 1, abort_flag, p.d_error);
            tc_fence_after();
            const uint32_t d = tmem + L::cO + qq * NR, a = v_lo + ((qq * L::kVUnitBytes) >> 4);
            const uint32_t b = p_lo + ((at * (L::kVTokens / 8) * p_sbo) >> 4);
#pragma unroll
            for (int j = 0; j < L::kVTokens / 16; ++j)
              mma_f16_ss(d, a + ((j * 2048) >> 4), v_hi, b + ((j * 2 * p_sbo) >> 4), p_hi, idesc,
                         !(opens && at == 0 && j == 0));
            commit_one(&bars[L::bVFree + qq]);
          }
          commit_one(&bars[L::bPFree + half]);
        }
      }
      commit_one(&bars[L::bDrain]);
      mbar_drain(&bars[L::bDrain], 0, p.d_error, kPagedWaitNs);
    } else if (warp < kSoftmaxWarps) {
      // ---------------------------------------------------------------- softmax
      constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
      const int quad = warp & 3, side = warp >> 2;
      const int row = quad * 32 + lane;      // token of the tile
      const int c0 = side * NC;              // first row of this thread
      const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
      const uint32_t tS = tmem + lanes + L::cS + c0, tO = tmem + lanes + L::cO;

      // The largest score whose exponent is within the slack, rounded down: with
      // 32 rows and more, whose exponents are computed again for P, comparing
      // scores with it takes one sum each (32 x 2 x 128 heads, window 4096: 105.5
      // us among others, 107.5 with whole exponents).
      const auto most_under = [](float m, float scale) { return __fadd_rd(m, __fdividef(kSlack, scale)); };

      // A unit's Q becomes scaled f16 in place, a row per warp at a time (lane =
      // 16 dims); rows past the unit's become zeros.
      uint32_t q_parity = 0;
      const auto convert_q = [&](int u, bool first) {
        constexpr int kRowsAtOnce = NR == 16 ? 2 : 1;  // (registers)
        bool bad_len;
        const Unit t = first ? *first_unit : unit_of<NR, kShared>(p, groups, u, bad_len, num_groups);
        wait_for(&bars[L::bQRaw], q_parity, abort_flag, p.d_error);
        q_parity ^= 1;
        uint8_t* base = sQ + (lane >> 2) * (NR * 128);
#pragma unroll kRowsAtOnce
        for (int r = warp; r < NR; r += kSoftmaxWarps) {
          const uint32_t off = r * 128 + (lane & 3) * 32;
          uint4* pa = reinterpret_cast<uint4*>(base + swz<128>(off));
          uint4* pb = reinterpret_cast<uint4*>(base + swz<128>(off + 16));
          const uint4 a = *pa, b = *pb;
          uint32_t wv[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          // The largest magnitude of the row, two values to a word.
          uint32_t two = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            if (r >= t.nrows) wv[k] = 0;
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
          *pa = make_uint4(wv[0], wv[1], wv[2], wv[3]);
          *pb = make_uint4(wv[4], wv[5], wv[6], wv[7]);
          if (lane == 0) {
            // Never 0 or infinite, so that no score times it is NaN (scores are below 2^36).
            const float s = fminf(fabsf(p.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 + e) << 23), 3.0e38f);
            c_scale[r] = s == 0.f ? 1e-30f : s;
            c_minus_m[r] = -kNoMax;
            c_minus_most[r] = -most_under(kNoMax, c_scale[r]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::bQFull]);
        if (tid < NR) {
          const int hi = kShared && t.b < 0 ? t.p_hi : t.first + min(t.row0 + tid, p.rows - 1) / p.h;
          c_hi[tid] = hi;
          c_lo[tid] = window_start(p, hi);
        }
        named_bar_sync(1, kSoftmaxThreads);  // the row arrays are complete
      };
      // This thread's exponents of rows h .. h + HC - 1 in an item: scale *
      // (score - m) + kPBias.  The difference comes first, as it is exact near m:
      // scale * score rounded into m would leave the maximum's own exponent half
      // a step of that product off, and P infinite or 0 for scores past 2^27.
      const auto exponents = [&](uint32_t s_col, int h, float (&y)[HC]) {
        uint32_t r[HC];
        tmem_ld<HC>(s_col + h, r);
        const float4* sc4 = reinterpret_cast<const float4*>(c_scale + c0 + h);
        const float4* mm4 = reinterpret_cast<const float4*>(c_minus_m + c0 + h);
        const float2 bias = make_float2(kPBias, kPBias);
#pragma unroll
        for (int k = 0; k < HC / 4; ++k) {
          const float4 s = sc4[k], m = mm4[k];
          const float2 a = make_float2(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1]));
          const float2 b = make_float2(__uint_as_float(r[4 * k + 2]), __uint_as_float(r[4 * k + 3]));
          const float2 u = __ffma2_rn(__fadd2_rn(a, make_float2(m.x, m.y)), make_float2(s.x, s.y), bias);
          const float2 v = __ffma2_rn(__fadd2_rn(b, make_float2(m.z, m.w)), make_float2(s.z, s.w), bias);
          y[4 * k] = u.x, y[4 * k + 1] = u.y, y[4 * k + 2] = v.x, y[4 * k + 3] = v.y;
        }
      };

      convert_q(cut[0], true);
      float l[NC];
#pragma unroll 1
      for (uint32_t n = 0; n < items; ++n) {
        wait_for(&bars[L::bInfo + n % kInfoRing], (n / kInfoRing) & 1, abort_flag, p.d_error);
        const int2 it = *reinterpret_cast<const int2*>(&info[n % kInfoRing]);
        if (it.x & kOpens) {
#pragma unroll
          for (int c = 0; c < NC; ++c) l[c] = 0.f;
        }
        wait_for(&bars[L::bSFull + (n & 1)], (n >> 1) & 1, abort_flag, p.d_error);
        tc_fence_after();
        const uint32_t s_col = tS + (n & 1) * NR;
        // The piece's last scores are there, so its Q has been read: the next unit's may come.
        // (None after a wait that gave up: the last one asked for has to have landed at the end.)
        if ((it.x & kCloses) && n + 1 < items && tid == 0 && !*abort_flag) {
          request_q(min(kShared ? max(info[n % kInfoRing].w, 0) : max(info[n % kInfoRing].z, 0) + 1, units - 1));
          cut[4] ^= 1;
        }
        if (!(it.x & kWhole)) {
          // Scores of tokens that a row does not see become minus infinity.
          const int pos = it.y * kTile + row;
          const bool there = token_there(it.x, row), sink = pos < p.sinks;
#pragma unroll 1
          for (int h = 0; h < NC; h += 8) {
            uint32_t r[8];
            tmem_ld<8>(s_col + h, r);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const int i = c0 + h + c;
              const bool see = there && pos <= c_hi[i] && (sink || pos >= c_lo[i]);
              if (!see) r[c] = 0xFF800000u;
            }
            tmem_st8(s_col + h, r);
          }
          tmem_wait_st();
        }
        float top = -INFINITY;
        float kept[kKeep ? NC : 1];  // with few rows the exponents stay in registers
#pragma unroll
        for (int h = 0; h < NC; h += HC) {
          float y[HC];
          if constexpr (kKeep) {
            exponents(s_col, h, y);
#pragma unroll
            for (int c = 0; c < HC; ++c) kept[h + c] = y[c];
          } else {
            uint32_t r[HC];
            tmem_ld<HC>(s_col + h, r);
            const float4* most4 = reinterpret_cast<const float4*>(c_minus_most + c0 + h);
#pragma unroll
            for (int k = 0; k < HC / 4; ++k) {
              const float4 m = most4[k];
              y[4 * k] = __uint_as_float(r[4 * k]) + m.x, y[4 * k + 1] = __uint_as_float(r[4 * k + 1]) + m.y;
              y[4 * k + 2] = __uint_as_float(r[4 * k + 2]) + m.z, y[4 * k + 3] = __uint_as_float(r[4 * k + 3]) + m.w;
            }
          }
#pragma unroll
          for (int c = 0; c < HC; ++c) top = fmaxf(top, y[c]);
        }
        if (any_of(2, kSoftmaxThreads, top > (kKeep ? kSlack + kPBias : 0.f))) {
          // Exact maxima of the tile's rows.
#pragma unroll 1
          for (int h = 0; h < NC; h += HC) {
            uint32_t r[HC];
            float y[HC];
            tmem_ld<HC>(s_col + h, r);
#pragma unroll
            for (int c = 0; c < HC; ++c) y[c] = __uint_as_float(r[c]);
            LaneReduce<HC, 16>::run(y, lane, OpMax());
            if (lane % (32 / HC) == 0) red[quad * NR + c0 + h + column_of<HC>(lane)] = y[0];
          }
          named_bar_sync(1, kSoftmaxThreads);
          bool moved = false;
          if (tid < NR) {
            const float m = fmaxf(fmaxf(red[tid], red[NR + tid]), fmaxf(red[2 * NR + tid], red[3 * NR + tid]));
            const float minus_old = c_minus_m[tid], scale = c_scale[tid];
            float alpha = 1.f;
            if (fmaf(m + minus_old, scale, kPBias) > kSlack + kPBias) {  // (its exponent, as above)
              alpha = ex2_approx(-(m + minus_old) * scale);
              moved = minus_old != -kNoMax;
              c_minus_m[tid] = -m;
              c_minus_most[tid] = -most_under(m, scale);
            }
            c_alpha[tid] = alpha;
          }
          const bool any_moved = any_of(2, kSoftmaxThreads, moved);
          if constexpr (kKeep) {
#pragma unroll
            for (int h = 0; h < NC; h += HC) {
              float y[HC];
              exponents(s_col, h, y);
#pragma unroll
              for (int c = 0; c < HC; ++c) kept[h + c] = y[c];
            }
          }
          if (any_moved) {
#pragma unroll
            for (int c = 0; c < NC; ++c) l[c] *= c_alpha[c0 + c];
            // O^T follows, once the product before this one is complete.
            if (!(it.x & kOpens)) {
              wait_for(&bars[L::bPFree + 1], (n & 1) ^ 1, abort_flag, p.d_error);
              tc_fence_after();
#pragma unroll 1
              for (int i = side; i < 4 * (NR / 16); i += L::kSides) {
                const int qq = i / (NR / 16), cc = (i % (NR / 16)) * 16;
                uint32_t o[16];
                tmem_ld16(tO + qq * NR + cc, o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * c_alpha[cc + k]);
                tmem_st16(tO + qq * NR + cc, o);
              }
              tmem_wait_st();
              // A product adds to all lanes of O^T, and the first half's needs the P of two lane quadrants only: no
              // warp hands its P over before every quadrant is rescaled.
              tc_fence_before();
              named_bar_sync(1, kSoftmaxThreads);
              tc_fence_after();
            }
          }
        }
        // P = 2^y, row `row` of P^T (MN-major); all of it is at hand when the
        // last product has read this half of the buffer.
        uint32_t e[NC / 2];
#pragma unroll
        for (int h = 0; h < NC; h += HC) {
          float y[HC];
          if constexpr (kKeep) {
#pragma unroll
            for (int c = 0; c < HC; ++c) y[c] = kept[h + c];
          } else {
            exponents(s_col, h, y);
          }
          if (h + HC == NC) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[L::bSFree + (n & 1)]);
          }
#pragma unroll
          for (int c = 0; c < HC; c += 2) {
            const float a = ex2_approx(y[c]), b = ex2_approx(y[c + 1]);
            l[h + c] += a;
            l[h + c + 1] += b;
            e[(h + c) / 2] = pack_f16x2(a, b);
          }
        }
        wait_for(&bars[L::bPFree + (quad >> 1)], (n & 1) ^ 1, abort_flag, p.d_error);
#pragma unroll
        for (int k = 0; k < NC / 8; ++k)
          *reinterpret_cast<uint4*>(sP + swz<2 * NR>(row * (2 * NR) + c0 * 2 + k * 16)) =
              make_uint4(e[4 * k], e[4 * k + 1], e[4 * k + 2], e[4 * k + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::bPFull + (quad >> 1)]);
        if (!(it.x & kCloses)) continue;

        // The piece's end: row sums over the tile's tokens, then O^T / l.
        LaneReduce<NC, 16>::run(l, lane, OpAdd());
        if (lane % (32 / NC) == 0) red[quad * NR + c0 + column_of<NC>(lane)] = l[0];
        named_bar_sync(1, kSoftmaxThreads);
        const bool whole_unit = !kShared && (it.x & (kFromStart | kToEnd)) == (kFromStart | kToEnd);
        // Partials: slot 2 part + 1 for a piece that begins its unit, 2 part for one that goes on with it.
        std::conditional_t<kShared, int64_t, int> prow = (part * 2 + ((it.x & kFromStart) ? 1 : 0)) * NR;
        const int u = min(max(info[n % kInfoRing].z, 0), units - 1);  // (after a wait that gave up it may be anything)
        if constexpr (kShared) {
          // A whole unit has a slot of its own behind those.
          if ((it.x & (kFromStart | kToEnd)) == (kFromStart | kToEnd))
            prow = (2 * static_cast<int64_t>(gridDim.x) + u) * NR;
        }
        const int ub = u / groups, urow0 = (u - ub * groups) * NR;
        const int orow = ub * p.rows + urow0, nrows = min(NR, p.rows - urow0);
        if (tid < NR) {
          const float sum = (red[tid] + red[NR + tid]) + (red[2 * NR + tid] + red[3 * NR + tid]);
          c_linv[tid] = sum > 0.f ? 1.f / sum : 0.f;
          const float lse =
              sum > 0.f ? fmaf(-c_minus_m[tid], c_scale[tid], log2f(sum) - kPBias) * 0.6931471805599453f : -INFINITY;
          if (!whole_unit)
            p.ws_lse[prow + tid] = lse;
          else if (tid < nrows)
            p.lse[orow + tid] = lse;
        }
        named_bar_sync(1, kSoftmaxThreads);
        // The next unit's Q goes in while the last product runs (this piece's scores are all done).
        if (n + 1 < items) convert_q(min(kShared ? max(info[n % kInfoRing].w, 0) : u + 1, units - 1), false);
        wait_for(&bars[L::bPFree + 1], n & 1, abort_flag, p.d_error);
        tc_fence_after();
        // Lane = dim, columns = rows.
        constexpr int EC = 16;  // columns at a time (registers)
#pragma unroll 1
        for (int i = side; i < 4 * (NR / EC); i += L::kSides) {
          const int qq = i / (NR / EC), cc = (i % (NR / EC)) * EC;
          const int d = qq * 128 + row;
          uint32_t o[EC];
          tmem_ld<EC>(tO + qq * NR + cc, o);
          const float4* l4 = reinterpret_cast<const float4*>(c_linv + cc);
#pragma unroll
          for (int k = 0; k < EC / 4; ++k) {
            const float4 s = l4[k];
            o[4 * k] = __float_as_uint(__uint_as_float(o[4 * k]) * s.x);
            o[4 * k + 1] = __float_as_uint(__uint_as_float(o[4 * k + 1]) * s.y);
            o[4 * k + 2] = __float_as_uint(__uint_as_float(o[4 * k + 2]) * s.z);
            o[4 * k + 3] = __float_as_uint(__uint_as_float(o[4 * k + 3]) * s.w);
          }
          if (whole_unit) {
            // Even lanes take row cc + k of dims (d, d + 1), odd lanes row cc + k + 1.
            const bool odd = (lane & 1) != 0;
            uint16_t* dst = p.out + static_cast<int64_t>(orow + cc + (odd ? 1 : 0)) * kD + (d & ~1);
            const int left = nrows - cc - (odd ? 1 : 0);
#pragma unroll
            for (int k = 0; k < EC; k += 2) {
              const float a = __uint_as_float(o[k]), b = __uint_as_float(o[k + 1]);
              const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 1);
              const __nv_bfloat162 v = odd ? __floats2bfloat162_rn(got, b) : __floats2bfloat162_rn(a, got);
              if (k < left) *reinterpret_cast<__nv_bfloat162*>(dst + k * kD) = v;
            }
          } else {
            float* dst = p.ws_o + static_cast<int64_t>(prow + cc) * kD + d;
#pragma unroll
            for (int k = 0; k < EC; ++k) dst[k * kD] = __uint_as_float(o[k]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::bOFree]);
        named_bar_sync(1, kSoftmaxThreads);  // the row sums' arrays may change again
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  // (Q's copies have landed long ago, unless a wait gave up.)
  if (tid == 0 && items > 0) mbar_drain(&bars[L::bQRaw], cut[4], p.d_error, kPagedWaitNs);
  if (warp == kValueWarp0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Merge of a unit cut by parts: pieces with normalised outputs o_i and
// log-sum-exps L_i give L = ln sum exp L_i and sum exp(L_i - L) o_i.  An entry
// of the info table (a part's last unit, or a unit) names the parts that hold
// pieces.  A row is joined by a warp where units have a few pieces (many rows,
// each a short chain of loads, so blocks of four), by four groups of 128
// threads that share its pieces where few units are cut into many.
struct Pieces {
  int part, count, r, nr;
  // Piece 0 is the first part's slot 2 part + 1, piece i part + i's slot 2 (part + i).
  __device__ __forceinline__ int64_t row(int i) const {
    return (static_cast<int64_t>(part + i) * 2 + (i == 0 ? 1 : 0)) * nr + r;
  }
};
// The pieces' largest log-sum-exp (0 if all are empty) and the sum of their weights.
__device__ __forceinline__ float piece_weights(const PagedParams& p, const Pieces& q, float& m) {
  const int lane = threadIdx.x & 31;
  m = -INFINITY;
  for (int i = lane; i < q.count; i += 32) m = fmaxf(m, p.ws_lse[q.row(i)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (m == -INFINITY) m = 0.f;
  float z = 0.f;
  for (int i = lane; i < q.count; i += 32) z += expf(p.ws_lse[q.row(i)] - m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
  return z;
}
__device__ __forceinline__ void add_piece(float4& acc, float w, const float4& v) {
  acc.x = fmaf(w, v.x, acc.x);
  acc.y = fmaf(w, v.y, acc.y);
  acc.z = fmaf(w, v.z, acc.z);
  acc.w = fmaf(w, v.w, acc.w);
}
__device__ __forceinline__ uint2 four_bf16(const float4& v) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

__global__ void __launch_bounds__(128) paged_merge_kernel(const PagedParams p, const int groups, const int nr) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 entry = *reinterpret_cast<const int4*>(p.ws_info + blockIdx.x * 4);
  const int lane = threadIdx.x & 31;
  const int r = static_cast<int>(blockIdx.y) * 4 + (threadIdx.x >> 5);
  if (entry.x < 0) return;
  const int b = entry.x / groups, row0 = (entry.x - b * groups) * nr;
  if (row0 + r >= p.rows) return;
  const Pieces q{entry.y, entry.z - entry.y + 1, r, nr};
  float m;
  const float z = piece_weights(p, q, m);
  const float inv = z > 0.f ? 1.f / z : 0.f;
  float4 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int i = 0; i < q.count; ++i) {
    const int64_t pr = q.row(i);
    const float4* src = reinterpret_cast<const float4*>(p.ws_o + pr * kD);
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = src[k * 32 + lane];
    const float w = expf(p.ws_lse[pr] - m) * inv;
#pragma unroll
    for (int k = 0; k < 4; ++k) add_piece(acc[k], w, v[k]);
  }
  const int64_t row = static_cast<int64_t>(b) * p.rows + row0 + r;
  uint2* dst = reinterpret_cast<uint2*>(p.out + row * kD);
#pragma unroll
  for (int k = 0; k < 4; ++k) dst[k * 32 + lane] = four_bf16(acc[k]);
  if (lane == 0) p.lse[row] = z > 0.f ? m + logf(z) : -INFINITY;
}

__global__ void __launch_bounds__(512) paged_merge_many_kernel(const PagedParams p, const int groups, const int nr) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float4 sums[3][128];
  const int4 entry = *reinterpret_cast<const int4*>(p.ws_info + blockIdx.x * 4);
  const int r = blockIdx.y, group = threadIdx.x >> 7, tid = threadIdx.x & 127;
  if (entry.x < 0) return;
  const int b = entry.x / groups, row0 = (entry.x - b * groups) * nr;
  if (row0 + r >= p.rows) return;
  const Pieces q{entry.y, entry.z - entry.y + 1, r, nr};
  float m;
  const float z = piece_weights(p, q, m);
  const float inv = z > 0.f ? 1.f / z : 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = group; i < q.count; i += 16) {  // four of the group's pieces in flight
    float4 v[4];
    float w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t pr = q.row(min(i + 4 * j, q.count - 1));
      v[j] = *reinterpret_cast<const float4*>(p.ws_o + pr * kD + tid * 4);
      w[j] = i + 4 * j < q.count ? p.ws_lse[pr] : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) add_piece(acc, expf(w[j] - m) * inv, v[j]);
  }
  if (group > 0) sums[group - 1][tid] = acc;
  __syncthreads();
  if (group > 0) return;
#pragma unroll
  for (int g = 0; g < 3; ++g) add_piece(acc, 1.f, sums[g][tid]);
  const int64_t row = static_cast<int64_t>(b) * p.rows + row0 + r;
  *reinterpret_cast<uint2*>(p.out + row * kD + tid * 4) = four_bf16(acc);
  if (tid == 0) p.lse[row] = z > 0.f ? m + logf(z) : -INFINITY;
}

template <int NR, bool kShared>
cudaError_t launch(Params<kShared> p, const PagedPlan& plan, cudaStream_t stream) {
  p.info_by_unit = kShared || static_cast<int64_t>(p.batch) * plan.groups <= plan.num_parts;
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = max_dynamic_smem_once(configured, reinterpret_cast<const void*>(paged_decode_kernel<NR, kShared>),
                                        PSmem<NR>::kAlloc);
  if (e != cudaSuccess) return e;
  // Q viewed as rows of 512 bf16; a box is NR rows x 64 dims, 128-byte swizzled.
  EncodeTiledFn enc = tensor_map_encoder();
  if (enc == nullptr) return cudaErrorNotSupported;
  CUtensorMap q_map;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(p.batch) * p.rows};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(kD) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(NR)};
  const cuuint32_t estr[2] = {1, 1};
  if (enc(&q_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(p.q), dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  // The pool viewed as rows of 288 bytes; a box is a page's rows x 128 data
  // bytes or x the 32 scale bytes.
  CUtensorMap data_map, scale_map;
  const cuuint64_t kv_dims[2] = {static_cast<cuuint64_t>(kRecFp4), static_cast<cuuint64_t>(p.num_pages) * kPage};
  const cuuint64_t kv_strides[1] = {static_cast<cuuint64_t>(kRecFp4)};
  const cuuint32_t data_box[2] = {128, kPage}, scale_box[2] = {32, kPage};
  if (enc(&data_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p.kv), kv_dims, kv_strides, data_box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS ||
      enc(&scale_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p.kv), kv_dims, kv_strides, scale_box,
          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  // Both kernels are programmatic dependents: each may be scheduled while the
  // one before it drains and waits for its end (griddepcontrol.wait) before it
  // touches memory.
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3(static_cast<unsigned>(plan.num_parts));
  cfg.blockDim = dim3(PSmem<NR>::kThreads);
  cfg.dynamicSmemBytes = PSmem<NR>::kAlloc;
  e = cudaLaunchKernelEx(&cfg, paged_decode_kernel<NR, kShared>, p, plan.groups, q_map, data_map, scale_map);
  if (e != cudaSuccess) return e;
  if constexpr (kShared) return launch_shared_merge(p, plan, stream);
  // Units that are few against the parts are cut into many pieces (one
  // sequence of 64k tokens, 16 heads: 32 us so, 66 by single warps; 64 x 64
  // heads over 1k to 8k, in three pieces: 89 against 72).
  const int units = p.batch * plan.groups;
  const bool many = units * 6 <= plan.num_parts;
  cfg.gridDim = dim3(static_cast<unsigned>(p.info_by_unit ? units : plan.num_parts), many ? NR : NR / 4);
  cfg.blockDim = dim3(many ? 512 : 128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, many ? paged_merge_many_kernel : paged_merge_kernel,
                            static_cast<const PagedParams&>(p), plan.groups, NR);
}

}  // namespace

PagedPlan paged_plan(const mla_paged_problem_t* p, int num_parts) {
  PagedPlan pl{};
  const int64_t rows = static_cast<int64_t>(p->seq_len_q) * p->h_q;
  // Rows of a unit: as few as hold them all, for a tile's decode is most of its
  // cost (32 sequences of 8k tokens, 24 heads: 50 us by 32, 59 by 64, 72 by 16;
  // 64 of 1k to 8k, 64 heads: 72 by 64, 96 by 32; 32 of 64k, 16 heads: 227 by 16,
  // 249 by 32).  Where the lengths that the table and the window allow leave no
  // part more than three or four tiles even so, as few as that takes: the start
  // and the end of a unit are then most of its cost, and shorter (7 x 3 x 24
  // heads, window 1000: 22.5 us by 16, 26.6 by 64; 16 of 1000 tokens, 64 heads:
  // 24.6 by 32, 28.7 by 64; 2 of 446, 128 heads: 18.4 by 16, 22.3 by 64).  The
  // lengths themselves are on the device: short sequences under a wide table
  // without a window get what the width says.
  int64_t tiles = (p->max_pages + 1) / 2;
  if (p->window > 0) {
    const int64_t seen = (int64_t(p->window) + p->seq_len_q) / kTile + 2 + (p->sinks + kTile - 1ll) / kTile;
    if (seen < tiles) tiles = seen;
  }
  const auto fits = [&](int nr) {
    return rows <= nr || 2ll * p->batch * ((rows + nr - 1) / nr) * (tiles + kUnitCost) <= int64_t(7) * num_parts;
  };
  pl.nr = fits(16) ? 16 : (fits(32) ? 32 : 64);
  pl.groups = static_cast<int>((rows + pl.nr - 1) / pl.nr);
  pl.num_parts = num_parts;
  pl.ws_o_bytes = static_cast<size_t>(num_parts) * 2 * pl.nr * MLA_HEAD_DIM * sizeof(float);
  pl.ws_lse_bytes = static_cast<size_t>(num_parts) * 2 * pl.nr * sizeof(float);
  pl.ws_bytes = pl.ws_o_bytes + pl.ws_lse_bytes + static_cast<size_t>(num_parts) * 4 * sizeof(int32_t);
  return pl;
}

cudaError_t launch_paged_decode(const PagedParams& p, const PagedPlan& plan, cudaStream_t stream) {
  switch (plan.nr) {
    case 16: return launch<16, false>(p, plan, stream);
    case 32: return launch<32, false>(p, plan, stream);
    default: return launch<64, false>(p, plan, stream);
  }
}

PagedPlan shared_plan(const mla_paged_shared_problem_t* p, int num_parts) {
  PagedPlan pl{};
  const int64_t rows = static_cast<int64_t>(p->seq_len_q) * p->h_q, all = rows * p->batch;
  // Rows of a unit, by the same reasoning as above: as few as hold a group's
  // rows, or as leave no part more than three or four tiles.  The groups' starts are
  // on the device: the batch counts as split evenly over them (groups past its
  // sequences are empty), and a group's last unit may be part full.
  const int64_t held = p->groups < p->batch ? p->groups : p->batch, group_rows = (all + held - 1) / held;
  const auto prefix_units = [&](int64_t nr) { return held * ((group_rows + nr - 1) / nr); };
  const auto own_units = [&](int64_t nr) { return p->batch * ((rows + nr - 1) / nr); };
  const int64_t tiles = (p->max_prefix_pages + 1) / 2 + kUnitCost, own = (p->max_pages + 1) / 2 + kUnitCost;
  const auto fits = [&](int nr) {
    return group_rows <= nr || 2 * (prefix_units(nr) * tiles + own_units(nr) * own) <= int64_t(7) * num_parts;
  };
  pl.nr = fits(16) ? 16 : (fits(32) ? 32 : 64);
  pl.num_parts = num_parts;
  // By pairs of SMs where there are many rows to a prefix and long ones: an item of 256 tokens x 128 rows takes a pair
  // some 8000 cycles, a tile of 128 x 64 an SM 6000, and a pair's start, exchanges and end 10 us more.  Both kernels
  // without the merge: 64 x 128 heads over a prefix of 16k tokens 267 us by pairs, 354 by single SMs; several groups over
  // 64k tokens each, 10 of 200 rows 312 and 414, 8 of 128 rows 145 and 176, 20 of 64 rows 321 and 216, 40 of 48 rows 618
  // and 422; 16 of 192 rows over 16k tokens 152 and 138; 31 x 2 x 24 heads over three of up to 9k 52 and 45; 8 x 16 heads
  // over 4k 24 and 14.  (With half a unit a group beside all rows together, many small groups went by pairs.)
  const auto work = [&](int64_t nr, int64_t tokens) {
    const auto items = [&](int64_t pages) { return (pages * kPage + tokens - 1) / tokens + kUnitCost; };
    return static_cast<double>(prefix_units(nr)) * items(p->max_prefix_pages) +
           static_cast<double>(own_units(nr)) * items(p->max_pages);
  };
  if (num_parts >= 2 && work(128, 256) * 8000 / (num_parts / 2) + 20000 < work(64, 128) * 6000 / num_parts) {
    pl.pair = true;
    pl.nr = 128;
    pl.num_parts = num_parts / 2;
  }
  pl.groups = static_cast<int>((rows + pl.nr - 1) / pl.nr);
  const int64_t units = p->batch * static_cast<int64_t>(pl.groups) + all / pl.nr + p->groups;
  pl.units = static_cast<int>(units);
  const size_t slots = 2 * static_cast<size_t>(pl.num_parts) + static_cast<size_t>(units);
  pl.ws_o_bytes = slots * pl.nr * MLA_HEAD_DIM * sizeof(float);
  pl.ws_lse_bytes = slots * pl.nr * sizeof(float);
  pl.ws_bytes = pl.ws_o_bytes + pl.ws_lse_bytes + (static_cast<size_t>(units) + 1) * 4 * sizeof(int32_t);
  return pl;
}

cudaError_t launch_shared_decode(const SharedParams& p, const PagedPlan& plan, cudaStream_t stream) {
  if (plan.pair) return launch_shared_pair(p, plan, stream);
  switch (plan.nr) {
    case 16: return launch<16, true>(p, plan, stream);
    case 32: return launch<32, true>(p, plan, stream);
    default: return launch<64, true>(p, plan, stream);
  }
}

}  // namespace mla
