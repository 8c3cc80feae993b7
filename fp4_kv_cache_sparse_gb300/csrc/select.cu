// select.cu -- which pages a query token attends to (include/mla.h,
// mla_paged_sparse_decode_fp4): a cheap score of every full page from the
// pages' 8-bit means, and the best of them.
//
// With a row's codes a_hd = q_hd 2^-e_h rounded to whole numbers in [-127, 127]
// (e_h the least that allows it) and a page's mean codes c_d 2^e,
//     score(page) = 2^e max over heads h of 2^(e_h - max e) <a_h, c>.
// The products' sums are whole numbers below 2^23 and everything else is a power
// of two, so a score is exact in fp32 whatever the order of its sums, and the
// choice (ties to the lower page) is a function of the inputs alone.
#include <cstdint>

#include "mla_device.cuh"
#include "mla_internal.h"
#include "mla_tensor.cuh"

namespace mla {

namespace {

// Where a query token stands and what may be left out of its pages.
struct Query {
  int at;      // position, below 0 when there is no such token
  int pages;   // pages up to its own
  int lo, hi;  // pages whose scores count: all but the sinks and the last ones
};

__device__ __forceinline__ Query query_of(const SelectParams& p, int b, int i, bool& bad) {
  const int len = load_i32(p.seq_lens + b);
  bad = len < 0 || len > p.max_pages * kPage;
  Query q;
  q.at = bad ? -1 : len - p.s + i;
  q.pages = q.at < 0 ? 0 : q.at / kPage + 1;
  q.lo = p.sinks;
  q.hi = q.pages - p.local;
  return q;
}

// ------------------------------------------------------------------ the best of them

// A key that orders as the scores do (0 and -0 are equal).
__device__ __forceinline__ uint32_t key_of(float score) {
  const uint32_t u = __float_as_uint(score + 0.f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// Exclusive prefix sum of two counts (each below 2^31) over the block (of at most 32 warps).
__device__ __forceinline__ int2 block_prefix(int2 mine, int2* warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, incl.x, o), y = __shfl_up_sync(0xFFFFFFFFu, incl.y, o);
    if (lane >= o) incl.x += x, incl.y += y;
  }
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  const int2 other = lane < warp ? warps[lane] : make_int2(0, 0);
  return make_int2(incl.x - mine.x + __reduce_add_sync(0xFFFFFFFFu, other.x),
                   incl.y - mine.y + __reduce_add_sync(0xFFFFFFFFu, other.y));
}

// The pages of one query token, by a whole CTA, its scores in place.  The k-th
// largest key by its bytes, the highest first: a count of each value of the next
// byte among the keys that agree with what is known.  Then the keys above it, and
// as many of the equal ones as are missing, from the lowest page on.
template <int kThreads>
__device__ __forceinline__ void choose(const SelectParams& p, int query, const Query& at, uint32_t* keys, int room,
                                       int* counts) {
  int* found = counts + 256;
  int2* warps = reinterpret_cast<int2*>(found + 4);
  const int tid = threadIdx.x;
  const int32_t* row = p.block_table + static_cast<int64_t>(query / p.s) * p.max_pages;
  int32_t* selected = p.selected ? p.selected + static_cast<int64_t>(query) * p.top : nullptr;
  int32_t* ids = p.sel_table + static_cast<int64_t>(query) * p.top;
  const auto take = [&](int place, int page) {
    ids[place] = load_i32(row + page);
    if (selected) selected[place] = page;
  };
  if (tid == 0) p.sel_lens[query] = at.at < 0 ? 0 : (min(at.pages, p.top) - 1) * kPage + at.at % kPage + 1;
  if (at.pages <= p.top) {
    for (int j = tid; j < p.top; j += kThreads) {
      if (j < at.pages)
        take(j, j);
      else if (selected)
        selected[j] = -1;
    }
    return;
  }
  const int k = p.top - p.sinks - p.local, n = at.hi - at.lo;  // n > k
  const float* scores = p.scores + static_cast<int64_t>(query) * p.max_pages + at.lo;
  const auto key_at = [&](int j) { return j < room ? keys[j] : key_of(__ldcg(scores + j)); };
  uint32_t least = ~0u, most = 0;
  constexpr int kBatch = 4;  // loads under way together (one by one 32.5 us for 64 query tokens of 128 heads, 31.3 so)
#pragma unroll 1
  for (int j0 = tid; j0 < n; j0 += kBatch * kThreads) {
    float score[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) score[i] = __ldcg(scores + min(j0 + i * kThreads, n - 1));
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int j = j0 + i * kThreads;
      const uint32_t key = key_of(score[i]);
      if (j < min(n, room)) keys[j] = key;
      least = min(least, key);
      most = max(most, key);
    }
  }
  least = __reduce_min_sync(0xFFFFFFFFu, least);
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if (tid % 32 == 0) warps[tid / 32] = make_int2(least, most);
  for (int j = tid; j < 256; j += kThreads) counts[j] = 0;
  __syncthreads();
  const int2 range = warps[tid % 32 % (kThreads / 32)];
  least = __reduce_min_sync(0xFFFFFFFFu, static_cast<uint32_t>(range.x));
  most = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(range.y));
  __syncthreads();
  // Bits from `bit` up agree with `known` for every key that still counts.
  int bit = k > 0 ? 32 - __clz(least ^ most) : 0, left = k;
  uint32_t known = bit == 32 ? 0 : most >> bit << bit;
  // The keys from `known` on are taken, all of them when `left` says so.
#pragma unroll 1
  for (bool all = false; bit > 0 && !all;) {
    const int digit = min(bit, 8), shift = bit - digit;
#pragma unroll 2
    for (int j = tid; j < n; j += kThreads) {
      const uint32_t key = key_at(j);
      if (((key ^ known) >> shift) < (1u << digit)) atomicAdd(&counts[(key >> shift) & ((1u << digit) - 1)], 1);
    }
    __syncthreads();
    if (tid < 32) {
      // Lane l: values 255 - 8 l and the seven below.
      int of[8], sum = 0;
#pragma unroll
      for (int v = 0; v < 8; ++v) sum += of[v] = counts[255 - 8 * tid - v];
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (tid >= o) incl += x;
      }
      int above = incl - sum;
      if (above < left && left <= incl) {
        int v = 0;
#pragma unroll
        for (int w = 0; w < 7; ++w)
          if (v == w && above + of[w] < left) above += of[w], ++v;
        found[0] = 255 - 8 * tid - v;
        found[1] = left - above;
        found[2] = counts[255 - 8 * tid - v];
      }
    }
    __syncthreads();
    known |= static_cast<uint32_t>(found[0]) << shift;
    left = found[1];
    all = left == found[2];
    bit = shift;
    for (int j = tid; j < 256; j += kThreads) counts[j] = 0;
    __syncthreads();
  }
  // Thread t: `per` pages in a row.  A key counts by its bits above those that were not looked at.
  const int per = (n + kThreads - 1) / kThreads;
  const int j0 = min(n, tid * per), j1 = min(n, j0 + per);
  known >>= bit;
  int2 mine = make_int2(0, 0);
#pragma unroll 2
  for (int j = j0; j < j1; ++j) {
    const uint32_t key = key_at(j) >> bit;
    mine.x += key > known;
    mine.y += key == known;
  }
  int2 before = block_prefix(mine, warps);
  // The pages go into a list first, so that their ids are looked up side by side.
  const bool listed = n + k <= room;
  uint32_t* list = keys + n;
#pragma unroll 1
  for (int j = j0; j < j1; ++j) {
    const uint32_t key = key_at(j) >> bit;
    if (key > known || (key == known && before.y < left)) {
      const uint32_t place = before.x + min(before.y, left);
      if (place >= static_cast<uint32_t>(k)) break;  // (after a wait that gave up the keys may have changed)
      if (listed)
        list[place] = at.lo + j;
      else
        take(p.sinks + place, at.lo + j);
    }
    before.x += key > known;
    before.y += key == known;
  }
  __syncthreads();
  for (int j = tid; j < p.top; j += kThreads) {
    const int i = j - p.sinks;
    if (i < 0)
      take(j, j);
    else if (i >= k)
      take(j, at.pages - p.top + j);
    else if (listed)
      take(j, min(list[i], static_cast<uint32_t>(at.pages) - 1));
  }
}

// ------------------------------------------------------------------ scores
//
// D[page, head] = <c, a_head> on the tensor core: 128 pages on M, their codes
// turned from bytes to f16 (exact) into tensor memory, a dim quarter at a time;
// the heads' codes as f16 in shared memory, made once per query token; whole
// numbers below 2^24, so the fp32 accumulator holds every partial sum exactly.
// The epilogue's thread is a page: the largest of its row, times the page's power
// of two.
//
// Work: a cluster of up to eight CTAs takes a query token at a time, its tiles
// of 128 pages in turn; behind the cluster's barrier one of them chooses.  With
// the choice in a kernel of its own the two took 41 + 9 us for 64 query tokens
// of 128 heads over 2048 pages and 11 + 6 us for one of 16 heads over 125; this
// kernel takes 31 and 7.8.
//
// What bounds it where there are many pages is the way of their means to the SMs
// and through shared memory: a tile of 128 pages is 68 KB, in 2.5 us with 128 heads
// and 2.2 with 16 (the slope of the time over 512 to 4096 pages, the choice's part in
// it) 3.5 TB/s out of L2 in pieces of 256 bytes; its decode costs
// 64 KB more, its products the 128 KB of 128 heads' codes (2048 cycles).  (The heads'
// codes in tensor memory and the pages' in shared memory moved more bytes: 35.4 us
// against 34.5 in the same arrangement.)  For few pages it is the chain of loads,
// lengths, page ids, records, scores, the choice: 7.8 us.
//
// One CTA, 16 warps: decode (8), epilogue (4, of which the first issues the
// products, a tile ahead), loads (4).  Loads by one warp took 20.5 us for 32
// query tokens of 64 heads over 1024 pages, by two 16.0, by four 15.4, with a
// bulk copy per record or 16-byte copies by all lanes; asked for by the epilogue's
// warps 18.2.  (14.3 now.)  Decode and epilogue warps also make a query token's
// codes, while its first pages are on their way.
constexpr int kTeams = 2;
constexpr int kScoreDecodeWarps = 4 * kTeams, kScoreEpilogueWarps = 4;
constexpr int kCodeWarps = kScoreDecodeWarps + kScoreEpilogueWarps;
constexpr int kScoreLoadWarp0 = kCodeWarps, kScoreWarps = kScoreLoadWarp0 + 4, kScoreThreads = kScoreWarps * 32;
constexpr int kScoreMmaWarp = kScoreDecodeWarps;  // the first of the epilogue
constexpr uint64_t kScoreWaitNs = 2000000000ull;

template <int NR>
struct ScoreSmem {
  // A stage is half of the dims of 32 pages, a quadrant of the tile's lanes, in rows
  // of an odd number of 16-byte units, so that the rows of a warp meet in no bank;
  // behind the first half's the 16 bytes with the scale.  (Whole records: 36.1 us
  // instead of 33.0 at 128 heads, where shared memory holds one tile; quarters 33.7.)
  static constexpr int kParts = 2, kRing = NR == 128 ? 2 : 4;
  static constexpr int kRecords = 32, kPartDims = kD / kParts, kPitch = kPartDims + 16, kStageBytes = kRecords * kPitch;
  static constexpr int kStages = 4 * kRing;
  // Its uses are one load warp's and the same decode warps', in order.  (Who runs
  // ahead of another's use would take the phase two before for its own.)
  static_assert(kScoreLoadWarp0 % 4 == 0, "stages by quadrants");
  static constexpr int kKeys = kStages * kStageBytes / 4;  // scores that the choice keeps where the stages were
  static constexpr int kQOff = 0;
  static constexpr int kRawOff = NR * kD * 2;
  static constexpr int kWeightOff = kRawOff + kStages * kStageBytes;  // float[NR]
  static constexpr int kExpOff = kWeightOff + NR * 4;                 // int[NR]
  static constexpr int kScaleOff = kExpOff + NR * 4;                  // float[2][128]
  static constexpr int kMaskOff = kScaleOff + 2 * kTile * 4;          // uint32[kStages]
  static constexpr int kBarOff = (kMaskOff + kStages * 4 + 7) & ~7;
  static constexpr int bRawFull = 0, bRawFree = bRawFull + kStages, bKFull = bRawFree + kStages, bKFree = bKFull + 4,
                       bSFull = bKFree + 4, bSFree = bSFull + 2, bScale = bSFree + 2, bQFull = bScale + 2,
                       bDrain = bQFull + 1, kNumBars = bDrain + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kCountOff = kMiscOff + 16;         // int[256], then the choice's small things
  static constexpr int kAlloc = kCountOff + 1024 + 256 + 1024;
  static_assert(kBarOff % 8 == 0 && kAlloc <= 232448, "shared memory of one CTA");
  __device__ static int arrivals(int i) {
    if (i < bRawFree) return 33;                // the lanes whose copies have landed, and the mask's
    if (i < bKFull) return kTeams;
    if (i >= bKFull && i < bKFree) return kScoreDecodeWarps;
    if (i >= bSFree && i < bQFull) return 4;
    if (i == bQFull) return kCodeWarps;
    return 1;
  }
  // Tensor memory columns: the codes' quarters, two score buffers.
  static constexpr int cA = 0, cS = 256;
};

__device__ __forceinline__ int tiles_of(const SelectParams& p, const Query& q) {
  return q.pages <= p.top ? 0 : max(q.hi - q.lo + kTile - 1, 0) / kTile;
}

// Four signed bytes -> four f16: 1024 + (byte + 128) has the byte in its low bits.
__device__ __forceinline__ void bytes_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t x = w ^ 0x80808080u;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(x, 0x64646464u, 0x4140)), "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(x, 0x64646464u, 0x4342)), "r"(0x64806480u));
}

// 32 codes in shared memory.
__device__ __forceinline__ void codes_to_f16(uint32_t src, uint32_t (&o)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint4 v = lds128(src + h * 16);
    bytes_to_f16(v.x, o[8 * h + 0], o[8 * h + 1]);
    bytes_to_f16(v.y, o[8 * h + 2], o[8 * h + 3]);
    bytes_to_f16(v.z, o[8 * h + 4], o[8 * h + 5]);
    bytes_to_f16(v.w, o[8 * h + 6], o[8 * h + 7]);
  }
}

__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.volatile.shared.u8 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// 16 bytes into shared memory, and this thread's arrival once its copies so far have landed.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

template <int NR>
__global__ void __launch_bounds__(kScoreThreads, 1) page_select_kernel(const SelectParams p, const int cluster) {
  using L = ScoreSmem<NR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + L::kQOff;
  uint8_t* sRaw = smem + L::kRawOff;
  float* weight = reinterpret_cast<float*>(smem + L::kWeightOff);
  int* exps = reinterpret_cast<int*>(smem + L::kExpOff);
  float* scales = reinterpret_cast<float*>(smem + L::kScaleOff);
  uint32_t* masks = reinterpret_cast<uint32_t*>(smem + L::kMaskOff);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMiscOff + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int first = static_cast<int>(blockIdx.x) / cluster, step = static_cast<int>(gridDim.x) / cluster;

  if (tid < L::kNumBars) mbar_init(&bars[tid], L::arrivals(tid));
  if (tid == 0) *abort_flag = 0;
  if (tid < L::kNumBars) {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == kScoreMmaWarp) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const auto wait = [&](int bar, uint32_t parity) {
    mbar_wait_warp(&bars[bar], parity, abort_flag, p.d_error, kScoreWaitNs);
  };
  uint32_t n0 = 0, scored = 0;  // tiles and query tokens of this CTA so far
  const int queries = p.batch * p.s;
  for (int u = first, round = 0; u < queries; u += step, ++round) {
    // The heads by rows, one per warp at a time, lane = 16 dims; the first are under way while the lengths are.
    constexpr int kRows = (NR + kCodeWarps - 1) / kCodeWarps, kAtOnce = kRows < 6 ? kRows : 6;
    uint4 raw[kAtOnce][2];
    const auto load_heads = [&](int i0) {
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int r = warp + (i0 + i) * kCodeWarps;
        raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
        if (r < p.h) {
          const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(u) * p.h + r) * kD + 16 * lane);
          raw[i][0] = src[0];
          raw[i][1] = src[1];
        }
      }
    };
    if (warp < kCodeWarps) load_heads(0);
    bool bad;
    const Query query = query_of(p, u / p.s, u % p.s, bad);
    // Tiles rank, rank + cluster, ...
    const int tiles = (max(tiles_of(p, query) - rank, 0) + cluster - 1) / cluster;
    const auto first_page = [&](uint32_t n) {
      return query.lo + (rank + static_cast<int>(n - n0) * cluster) * kTile;
    };
    // Load warp `quad` asks for its quadrant's records of a tile: lane = record for
    // the ids, then a record at a time, lane = 16 bytes.
    const int quad = warp & 3;
    const int32_t* table = p.block_table + static_cast<int64_t>(u / p.s) * p.max_pages;
    const auto look_up = [&](uint32_t n) {
      const int page = first_page(n) + quad * 32 + lane;
      return n < n0 + tiles && page < query.hi ? load_i32(table + page) : -1;
    };
    const auto ask = [&](uint32_t n, int id) {
      const bool ok = id >= 0 && id < p.num_pages;
      if (!ok && first_page(n) + quad * 32 + lane < query.hi && p.d_error) atomicOr(p.d_error, MLA_DEVERR_BAD_INDEX);
      const uint32_t there = __ballot_sync(0xFFFFFFFFu, ok);
#pragma unroll 1
      for (int part = 0; part < L::kParts; ++part) {
        const uint32_t no = n * L::kParts + part, stage = no % L::kRing * 4 + quad;
        wait(L::bRawFree + stage, ((no / L::kRing) & 1) ^ 1);
        if (lane == 0) {
          masks[stage] = there;
          mbar_arrive(&bars[L::bRawFull + stage]);
        }
        constexpr int kLanes = L::kPartDims / 16;  // of a record
        const uint32_t dst = smem_u32(sRaw) + stage * L::kStageBytes;
        const uint8_t* src = p.means + part * L::kPartDims + lane % kLanes * 16;
#pragma unroll 8
        for (int r0 = 0; r0 < 32; r0 += 32 / kLanes) {
          const int r = r0 + lane / kLanes, from = __shfl_sync(0xFFFFFFFFu, id, r);
          if ((there >> r) & 1)
            copy16(dst + r * L::kPitch + lane % kLanes * 16, src + static_cast<int64_t>(from) * MLA_MEAN_BYTES);
        }
        if (part == 0 && ok)
          copy16(dst + lane * L::kPitch + L::kPartDims, p.means + static_cast<int64_t>(id) * MLA_MEAN_BYTES + kD);
        __syncwarp();
        copies_arrive(&bars[L::bRawFull + stage]);
      }
    };
    if (tiles > 0 && warp < kCodeWarps) {
      // The heads' codes; rows past the heads become zeros.  (Every product with the last token's has been read, as
      // the CTA's barrier behind its scores says.)
#pragma unroll 1
      for (int i0 = 0; i0 < kRows; i0 += kAtOnce) {
        if (i0 > 0) load_heads(i0);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
          const int r = warp + (i0 + i) * kCodeWarps;
          if (r >= NR) break;
          const uint4 a = raw[i][0], b = raw[i][1];
          uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          uint32_t two = 0;
#pragma unroll
          for (int k = 0; k < 8; ++k) asm("max.u16x2 %0, %0, %1;" : "+r"(two) : "r"(w[k] & 0x7FFF7FFFu));
          const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, max(two >> 16, two & 0xFFFFu));
          // amax = m 2^E, m in [1, 2): the least e with amax 2^-e <= 127 is E - 6, but for m above 127/64 (all bits
          // set) E - 5.
          const int e = max(static_cast<int>((top + 1) >> 7) - 127 - 6, -120);
          const float up = copysignf(__uint_as_float(static_cast<uint32_t>(127 - e) << 23), p.sign);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            w[k] = pack_f16x2(rintf(__uint_as_float(w[k] << 16) * up), rintf(__uint_as_float(w[k] & 0xFFFF0000u) * up));
          uint8_t* base = sQ + (lane >> 2) * (NR * 128);
          const uint32_t off = r * 128 + (lane & 3) * 32;
          *reinterpret_cast<uint4*>(base + swz<128>(off)) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(base + swz<128>(off + 16)) = make_uint4(w[4], w[5], w[6], w[7]);
          if (lane == 0) exps[r] = top == 0 ? -1000 : e;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[L::bQFull]);
      named_bar_sync(1, kCodeWarps * 32);
      if (warp >= kScoreDecodeWarps) {
        const int i = tid - kScoreDecodeWarps * 32;
        int most = -1000;
#pragma unroll
        for (int k = 0; k < (NR + 31) / 32; ++k) most = max(most, lane + 32 * k < NR ? exps[lane + 32 * k] : -1000);
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        // NaN for rows that are none: no maximum takes it.
        if (i < NR)
          weight[i] = i < p.h ? __uint_as_float(static_cast<uint32_t>(127 + max(exps[i] - most, -100)) << 23)
                              : __uint_as_float(0x7FC00000u);
        named_bar_sync(2, kScoreEpilogueWarps * 32);
      }
    }

    if (warp < kScoreDecodeWarps) {
      // ---------------------------------------------------------------- codes to f16: lane = page
      const int team = warp >> 2;
      const uint32_t tA = tmem + (static_cast<uint32_t>(quad * 32) << 16) + L::cA;
      for (uint32_t n = n0; n < n0 + tiles; ++n) {
        uint32_t e = 0;  // this page's scale byte, 256 for a page that is none
#pragma unroll 1
        for (int part = 0; part < L::kParts; ++part) {
          const uint32_t no = n * L::kParts + part, stage = no % L::kRing * 4 + quad;
          wait(L::bRawFull + stage, (no / L::kRing) & 1);
          const uint32_t rec = smem_u32(sRaw) + stage * L::kStageBytes + lane * L::kPitch;
          if (part == 0) e = (masks[stage] >> lane) & 1 ? lds8(rec + L::kPartDims) : 256u;
          // A team takes 64 of a quarter's dims.
#pragma unroll 1
          for (int j = 0; j < 4 / L::kParts; ++j) {
            const int qq = part * (4 / L::kParts) + j;
            wait(L::bKFree + qq, (n & 1) ^ 1);
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t o[16];
              codes_to_f16(rec + j * 128 + team * 64 + k * 32, o);
              tmem_st16(tA + qq * 64 + team * 32 + k * 16, o);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[L::bKFull + qq]);
          }
          if (lane == 0) mbar_arrive(&bars[L::bRawFree + stage]);
        }
        if (team == 0) {
          wait(L::bSFree + (n & 1), ((n >> 1) & 1) ^ 1);
          // 2^(e - 127), a negative mark for a page that is none
          scales[(n & 1) * kTile + quad * 32 + lane] =
              e == 256 ? -1.f : (e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23));
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[L::bScale + (n & 1)]);
        }
      }
    } else if (warp < kCodeWarps) {
      // ---------------------------------------------------------------- the largest of a page's row
      const uint32_t tS = tmem + (static_cast<uint32_t>(quad * 32) << 16) + L::cS;
      float* dst = p.scores + static_cast<int64_t>(u) * p.max_pages;
      // D = C A^T of a tile, before the last one's maxima.
      constexpr uint32_t idesc = idesc_f16(128, NR, false, false);
      const uint64_t desc = make_smem_desc(smem_u32(sQ), 16, 1024, kSwizzle128);
      const uint32_t lo = static_cast<uint32_t>(desc), hi = static_cast<uint32_t>(desc >> 32);
      const auto multiply = [&](uint32_t n) {
        const uint32_t d = tmem + L::cS + (n & 1) * NR;
        wait(L::bSFree + (n & 1), ((n >> 1) & 1) ^ 1);
#pragma unroll 1
        for (int qq = 0; qq < 4; ++qq) {
          wait(L::bKFull + qq, n & 1);
          tc_fence_after();
          const uint32_t a = tmem + L::cA + qq * 64, b = lo + ((2 * qq * NR * 128) >> 4);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            mma_f16_ts(d, a + j * 8, b + (((j >> 2) * NR * 128 + (j & 3) * 32) >> 4), hi, idesc, (qq | j) != 0);
          commit_one(&bars[L::bKFree + qq]);
        }
        commit_one(&bars[L::bSFull + (n & 1)]);
      };
      if (warp == kScoreMmaWarp && tiles > 0) {
        wait(L::bQFull, scored & 1);
        multiply(n0);
      }
      for (uint32_t n = n0; n < n0 + tiles; ++n) {
        if (warp == kScoreMmaWarp && n + 1 < n0 + tiles) multiply(n + 1);
        wait(L::bScale + (n & 1), (n >> 1) & 1);
        wait(L::bSFull + (n & 1), (n >> 1) & 1);
        tc_fence_after();
        float best = -INFINITY;
#pragma unroll 2
        for (int c = 0; c < NR; c += 16) {
          uint32_t r[16];
          tmem_ld16(tS + (n & 1) * NR + c, r);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 w = *reinterpret_cast<const float4*>(weight + c + 4 * i);
            best = fmaxf(fmaxf(fmaxf(best, __uint_as_float(r[4 * i]) * w.x), __uint_as_float(r[4 * i + 1]) * w.y),
                         fmaxf(__uint_as_float(r[4 * i + 2]) * w.z, __uint_as_float(r[4 * i + 3]) * w.w));
          }
        }
        const float scale = scales[(n & 1) * kTile + quad * 32 + lane];
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[L::bSFree + (n & 1)]);
        const int page = first_page(n) + quad * 32 + lane;
        if (page < query.hi) dst[page] = scale < 0.f ? -INFINITY : best * scale;
      }
    } else {
      // ---------------------------------------------------------------- records
      int id = look_up(n0);
      for (uint32_t n = n0; n < n0 + tiles; ++n) {
        const int next = look_up(n + 1);
        ask(n, id);
        id = next;
      }
    }
    n0 += tiles;
    scored += tiles > 0;

    // Every score of the query token is there; the CTAs choose in turn.
    __syncwarp();
    if (cluster > 1)
      cluster_barrier();
    else
      __syncthreads();
    if (round % cluster == rank) {
      if (bad && tid == 0 && u % p.s == 0 && p.d_error) atomicOr(p.d_error, MLA_DEVERR_BAD_LENGTH);
      choose<kScoreThreads>(p, u, query, reinterpret_cast<uint32_t*>(sRaw), L::kKeys,
                            reinterpret_cast<int*>(smem + L::kCountOff));
      __syncthreads();  // copies go where the keys were
    }
  }

  if (warp == kScoreMmaWarp && n0 > 0) {
    commit_one(&bars[L::bDrain]);
    mbar_drain(&bars[L::bDrain], 0, p.d_error, kScoreWaitNs);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");  // (they have landed, unless a wait gave up)
  tc_fence_before();
  __syncthreads();
  if (warp == kScoreMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int NR>
cudaError_t launch(const SelectParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = max_dynamic_smem_once(configured, reinterpret_cast<const void*>(page_select_kernel<NR>),
                                              ScoreSmem<NR>::kAlloc);
  if (e != cudaSuccess) return e;
  // As many CTAs to a query token as there are for all of them, and as its tiles
  // by the table's width; the lengths are on the device.
  const int64_t queries = static_cast<int64_t>(p.batch) * p.s;
  const int64_t tiles = (static_cast<int64_t>(p.max_pages) - p.sinks - p.local + kTile - 1) / kTile;
  int cluster = 8;
  while (cluster > 1 && (queries * cluster > p.num_parts || cluster > tiles)) cluster /= 2;
  const int64_t clusters = p.num_parts / cluster;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cfg.stream = stream;
  cfg.gridDim = dim3(static_cast<unsigned>((queries < clusters ? queries : clusters) * cluster));
  cfg.blockDim = dim3(kScoreThreads);
  cfg.dynamicSmemBytes = ScoreSmem<NR>::kAlloc;
  return cudaLaunchKernelEx(&cfg, page_select_kernel<NR>, p, cluster);
}

}  // namespace

cudaError_t launch_page_select(const SelectParams& p, cudaStream_t stream) {
  return p.h <= 16   ? launch<16>(p, stream)
         : p.h <= 32 ? launch<32>(p, stream)
         : p.h <= 64 ? launch<64>(p, stream)
                     : launch<128>(p, stream);
}

}  // namespace mla
