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

constexpr int kTopThreads = 512;
constexpr int kKeys = 8192;  // scores kept in shared memory

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

// ------------------------------------------------------------------ scores
//
// D[page, head] = <c, a_head> on the tensor core: 128 pages on M, their codes
// turned from bytes to f16 (exact) into tensor memory, a dim quarter at a time;
// the heads' codes as f16 in shared memory, made once per query token; whole
// numbers below 2^24, so the fp32 accumulator holds every partial sum exactly.
// The epilogue's thread is a page: the largest of its row, times the page's power
// of two.
//
// Work: a query token's tiles of 128 pages, all tokens in order, each two for
// its codes and then its tiles, cut into gridDim.x runs of equal cost.  The lengths are on the device,
// so every CTA derives the cut itself.
//
// One CTA, 14 warps: decode (8), epilogue (4), loader, product issuer; all of
// them make a query token's codes.
constexpr int kScoreDecodeWarps = 8, kScoreEpilogueWarps = 4;
constexpr int kScoreLoadWarp = kScoreDecodeWarps + kScoreEpilogueWarps, kScoreMmaWarp = kScoreLoadWarp + 1;
constexpr int kScoreWarps = kScoreMmaWarp + 1, kScoreThreads = kScoreWarps * 32;
constexpr int kQueryCost = 2;  // what a query token's codes take, in tiles
constexpr uint64_t kScoreWaitNs = 2000000000ull;

template <int NR>
struct ScoreSmem {
  // A stage is the records of 64 pages, 528 bytes apart as in memory: an odd
  // number of 16-byte units, so rows of a warp meet in no bank.
  static constexpr int kRecords = 64, kStageBytes = kRecords * MLA_MEAN_BYTES;
  static constexpr int kStages = NR == 128 ? 2 : 4;
  static constexpr int kQOff = 0;
  static constexpr int kRawOff = NR * kD * 2;
  static constexpr int kWeightOff = kRawOff + kStages * kStageBytes;  // float[NR]
  static constexpr int kExpOff = kWeightOff + NR * 4;                 // int[NR]
  static constexpr int kScaleOff = kExpOff + NR * 4;                  // float[2][128]
  static constexpr int kMaskOff = kScaleOff + 2 * kTile * 4;          // uint32[kStages][2]
  static constexpr int kBarOff = kMaskOff + kStages * 8;
  static constexpr int bRawFull = 0, bRawFree = bRawFull + kStages, bKFull = bRawFree + kStages, bKFree = bKFull + 4,
                       bSFull = bKFree + 4, bSFree = bSFull + 2, bScale = bSFree + 2, bDrain = bScale + 2,
                       kNumBars = bDrain + 1;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kAlloc = kMiscOff + 192 + 1024;
  static_assert(kBarOff % 8 == 0 && kAlloc <= 232448, "shared memory of one CTA");
  __device__ static int arrivals(int i) {
    if (i >= bRawFree && i < bKFull) return 4;  // two quadrants, both teams
    if (i >= bKFull && i < bKFree) return 4;
    if (i >= bSFree && i < bDrain) return 4;
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

template <int NR>
__global__ void __launch_bounds__(kScoreThreads, 1) page_score_kernel(const SelectParams p) {
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
  int* cut = reinterpret_cast<int*>(smem + L::kMiscOff + 8);          // query token, its tile, tiles of the run
  int* warp_sum = reinterpret_cast<int*>(smem + L::kMiscOff + 32);    // [warps]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid < L::kNumBars) mbar_init(&bars[tid], L::arrivals(tid));
  if (tid == 0) {
    *abort_flag = 0;
    cut[2] = 0;
  }
  if (tid < L::kNumBars) {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async_smem();
  }
  if (warp == kScoreMmaWarp) tmem_alloc(tmem_slot, 512);
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const auto query_at = [&](int u) {
    bool bad;
    return query_of(p, u / p.s, u % p.s, bad);
  };
  const auto wait = [&](int bar, uint32_t parity) {
    mbar_wait_warp(&bars[bar], parity, abort_flag, p.d_error, kScoreWaitNs);
  };
  // The cut: cost of all query tokens, this part's run.
  const int queries = p.batch * p.s;
  const int per = (queries + kScoreThreads - 1) / kScoreThreads;
  const int u_a = min(queries, tid * per), u_b = min(queries, u_a + per);
  int mine = 0;
  const auto cost_of = [](int tiles) { return tiles > 0 ? tiles + kQueryCost : 0; };
  for (int u = u_a; u < u_b; ++u) mine += cost_of(tiles_of(p, query_at(u)));
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  {
    const int sum = lane < kScoreWarps ? warp_sum[lane] : 0;
    const int total = __reduce_add_sync(0xFFFFFFFFu, sum);
    const int excl = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? sum : 0) + incl - mine;
    const int share = (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x);
    const int64_t from = static_cast<int64_t>(blockIdx.x) * share;
    const int g0 = static_cast<int>(min(from, static_cast<int64_t>(total)));
    const int g1 = static_cast<int>(min(from + share, static_cast<int64_t>(total)));
    if (g0 < g1 && excl <= g0 && g0 < excl + mine) {
      int at = excl, u = u_a, tiles = tiles_of(p, query_at(u));
      while (at + cost_of(tiles) <= g0) {
        at += cost_of(tiles);
        tiles = tiles_of(p, query_at(++u));
      }
      const int k = max(g0 - at - kQueryCost, 0);
      int count = max(min(at + kQueryCost + tiles, g1) - (at + kQueryCost + k), 0);
      cut[0] = u;
      cut[1] = k;
      for (at += cost_of(tiles); at + kQueryCost < g1; at += cost_of(tiles)) {
        tiles = tiles_of(p, query_at(++u));
        count += min(at + kQueryCost + tiles, g1) - (at + kQueryCost);
      }
      cut[2] = count;
    }
  }
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  int left = cut[2], k0 = cut[1];
  uint32_t n0 = 0;  // tiles done
  uint32_t asked = 0;  // stages asked for, by the loader

  for (int u = cut[0]; left > 0 && u < queries; ++u, k0 = 0) {
    const Query query = query_at(u);
    const int tiles = min(max(tiles_of(p, query) - k0, 0), left);  // of this query token in this run
    if (tiles == 0) continue;
    left -= tiles;

    // The heads' codes: a row per warp at a time, lane = 16 dims; rows past the heads become zeros.
    for (int r = warp; r < NR; r += kScoreWarps) {
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = 0;
      if (r < p.h) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(u) * p.h + r) * kD + 16 * lane);
        const uint4 a = src[0], b = src[1];
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
      }
      uint32_t two = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) asm("max.u16x2 %0, %0, %1;" : "+r"(two) : "r"(w[k] & 0x7FFF7FFFu));
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, max(two >> 16, two & 0xFFFFu));
      // amax = m 2^E, m in [1, 2): the least e with amax 2^-e <= 127 is E - 6, but for m above 127/64 (all bits set) E - 5.
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
    fence_proxy_async_smem();
    __syncthreads();
    if (warp < kScoreEpilogueWarps) {
      // (The epilogue reads the weights behind a product that these warps' codes take part in.)
      int most = -1000;
#pragma unroll
      for (int i = 0; i < (NR + 31) / 32; ++i) most = max(most, lane + 32 * i < NR ? exps[lane + 32 * i] : -1000);
      most = __reduce_max_sync(0xFFFFFFFFu, most);
      // NaN for rows that are none: no maximum takes it.
      if (tid < NR)
        weight[tid] = tid < p.h ? __uint_as_float(static_cast<uint32_t>(127 + max(exps[tid] - most, -100)) << 23)
                                : __uint_as_float(0x7FC00000u);
    }
    __syncthreads();

    if (warp < kScoreDecodeWarps) {
      // ---------------------------------------------------------------- codes to f16: lane = page
      const int quad = warp & 3, team = warp >> 2;
      const uint32_t tA = tmem + (static_cast<uint32_t>(quad * 32) << 16) + L::cA;
      const int row = (quad & 1) * 32 + lane;
      for (uint32_t n = n0; n < n0 + tiles; ++n) {
        const uint32_t stage_no = 2 * n + (quad >> 1), stage = stage_no % L::kStages;
        wait(L::bRawFull + stage, (stage_no / L::kStages) & 1);
        const uint8_t* rec = sRaw + stage * L::kStageBytes + row * MLA_MEAN_BYTES;
        if (team == 0) {
          wait(L::bSFree + (n & 1), ((n >> 1) & 1) ^ 1);
          const bool there = (masks[stage * 2 + (quad & 1)] >> lane) & 1;
          const uint32_t e = there ? rec[kD] : 255u;
          // 2^(e - 127), minus infinity's mark for a page that is none
          scales[(n & 1) * kTile + quad * 32 + lane] =
              !there ? -1.f : (e == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23));
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[L::bScale + (n & 1)]);
        }
#pragma unroll 1
        for (int qq = team; qq < 4; qq += 2) {
          wait(L::bKFree + qq, (n & 1) ^ 1);
          tc_fence_after();
          const uint32_t src = smem_u32(rec) + qq * 128;
#pragma unroll
          for (int part = 0; part < 4; ++part) {
            uint32_t o[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 v = lds128(src + part * 32 + h * 16);
              bytes_to_f16(v.x, o[8 * h + 0], o[8 * h + 1]);
              bytes_to_f16(v.y, o[8 * h + 2], o[8 * h + 3]);
              bytes_to_f16(v.z, o[8 * h + 4], o[8 * h + 5]);
              bytes_to_f16(v.w, o[8 * h + 6], o[8 * h + 7]);
            }
            tmem_st16(tA + qq * 64 + part * 16, o);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars[L::bKFull + qq]);
        }
        if (lane == 0) mbar_arrive(&bars[L::bRawFree + stage]);
      }
    } else if (warp < kScoreLoadWarp) {
      // ---------------------------------------------------------------- the largest of a page's row
      const int quad = warp & 3;
      const uint32_t tS = tmem + (static_cast<uint32_t>(quad * 32) << 16) + L::cS;
      float* dst = p.scores + static_cast<int64_t>(u) * p.max_pages;
      for (uint32_t n = n0; n < n0 + tiles; ++n) {
        wait(L::bScale + (n & 1), (n >> 1) & 1);
        wait(L::bSFull + (n & 1), (n >> 1) & 1);
        tc_fence_after();
        float best = -INFINITY;
#pragma unroll
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
        const int page = query.lo + (k0 + static_cast<int>(n - n0)) * kTile + quad * 32 + lane;
        if (page < query.hi) dst[page] = scale < 0.f ? -INFINITY : best * scale;
      }
    } else if (warp == kScoreLoadWarp) {
      // ---------------------------------------------------------------- loader: lane = record
      const int32_t* table = p.block_table + static_cast<int64_t>(u / p.s) * p.max_pages;
      for (uint32_t n = n0; n < n0 + tiles; ++n) {
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const uint32_t stage_no = 2 * n + half, stage = stage_no % L::kStages;
          const int page = query.lo + (k0 + static_cast<int>(n - n0)) * kTile + half * 64 + lane;
          int id[2];
          uint32_t there[2];
          bool bad = false;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            id[j] = page + 32 * j < query.hi ? load_i32(table + page + 32 * j) : -1;
            const bool ok = id[j] >= 0 && id[j] < p.num_pages;
            bad = bad || (!ok && page + 32 * j < query.hi);
            there[j] = __ballot_sync(0xFFFFFFFFu, ok);
          }
          if (bad && p.d_error) atomicOr(p.d_error, MLA_DEVERR_BAD_INDEX);
          wait(L::bRawFree + stage, ((stage_no / L::kStages) & 1) ^ 1);
          // After a wait that gave up nothing more is asked for.
          if (__any_sync(0xFFFFFFFFu, *abort_flag)) continue;
          ++asked;
          uint64_t* bar = &bars[L::bRawFull + stage];
          if (lane == 0) {
            masks[stage * 2] = there[0];
            masks[stage * 2 + 1] = there[1];
            expect_tx(bar, (__popc(there[0]) + __popc(there[1])) * MLA_MEAN_BYTES);
          }
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if ((there[j] >> lane) & 1)
              bulk_load(sRaw + stage * L::kStageBytes + (lane + 32 * j) * MLA_MEAN_BYTES,
                        p.means + static_cast<int64_t>(id[j]) * MLA_MEAN_BYTES, MLA_MEAN_BYTES, bar);
          }
        }
      }
    } else {
      // ---------------------------------------------------------------- D = C A^T
      constexpr uint32_t idesc = idesc_f16(128, NR, false, false);
      const uint64_t desc = make_smem_desc(smem_u32(sQ), 16, 1024, kSwizzle128);
      const uint32_t lo = static_cast<uint32_t>(desc), hi = static_cast<uint32_t>(desc >> 32);
      for (uint32_t n = n0; n < n0 + tiles; ++n) {
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
      }
    }
    n0 += tiles;
    // The codes and weights may change again once every product has been read.
    __syncthreads();
  }

  if (warp == kScoreMmaWarp && n0 > 0) {
    commit_one(&bars[L::bDrain]);
    mbar_drain(&bars[L::bDrain], 0, p.d_error, kScoreWaitNs);
  } else if (warp == kScoreLoadWarp) {
    // Every copy has landed before the CTA may end (they have, unless a wait gave up).
    for (uint32_t i = asked > L::kStages ? asked - L::kStages : 0; i < asked; ++i)
      mbar_drain(&bars[L::bRawFull + i % L::kStages], (i / L::kStages) & 1, p.d_error, kScoreWaitNs);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kScoreMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ the best of them

// A key that orders as the scores do (0 and -0 are equal).
__device__ __forceinline__ uint32_t key_of(float score) {
  const uint32_t u = __float_as_uint(score + 0.f);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}

// Exclusive prefix sum of two counts (each below 2^31) over the block.
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
  int2 before = make_int2(incl.x - mine.x, incl.y - mine.y);
  for (int w = 0; w < warp; ++w) before.x += warps[w].x, before.y += warps[w].y;
  return before;
}

// The k-th largest key by its bytes, the highest first: a count of each value
// of the next byte among the keys that agree with what is known.  Then the keys
// above it, and as many of the equal ones as are missing, from the lowest page on.
__global__ void __launch_bounds__(kTopThreads) page_top_kernel(const SelectParams p) {
  __shared__ uint32_t keys[kKeys];
  __shared__ int counts[256];
  __shared__ int found[2];
  __shared__ int2 warps[kTopThreads / 32];
  const int tid = threadIdx.x, query = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  bool bad;
  const Query at = query_of(p, query / p.s, query % p.s, bad);
  if (bad && tid == 0 && p.d_error) atomicOr(p.d_error, MLA_DEVERR_BAD_LENGTH);
  const int32_t* row = p.block_table + static_cast<int64_t>(query / p.s) * p.max_pages;
  int32_t* selected = p.selected ? p.selected + static_cast<int64_t>(query) * p.top : nullptr;
  int32_t* ids = p.sel_table + static_cast<int64_t>(query) * p.top;
  const auto take = [&](int place, int page) {
    ids[place] = row[page];
    if (selected) selected[place] = page;
  };
  if (tid == 0)
    p.sel_lens[query] = at.at < 0 ? 0 : (min(at.pages, p.top) - 1) * kPage + at.at % kPage + 1;
  if (at.pages <= p.top) {
    for (int j = tid; j < p.top; j += kTopThreads) {
      if (j < at.pages)
        take(j, j);
      else if (selected)
        selected[j] = -1;
    }
    return;
  }
  for (int j = tid; j < p.sinks; j += kTopThreads) take(j, j);
  for (int j = tid; j < p.local; j += kTopThreads) take(p.top - p.local + j, at.pages - p.local + j);
  const int k = p.top - p.sinks - p.local, n = at.hi - at.lo;  // n > k
  if (k == 0) return;
  const float* scores = p.scores + static_cast<int64_t>(query) * p.max_pages + at.lo;
  const auto key_at = [&](int j) { return j < kKeys ? keys[j] : key_of(scores[j]); };
  for (int j = tid; j < min(n, kKeys); j += kTopThreads) keys[j] = key_of(scores[j]);
  uint32_t known = 0;
  int left = k;  // of the keys that agree with `known` so far, how many are taken
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) counts[tid] = 0;
    __syncthreads();
    for (int j = tid; j < n; j += kTopThreads) {
      const uint32_t key = key_at(j);
      if (shift == 24 || (key >> (shift + 8)) == (known >> (shift + 8))) atomicAdd(&counts[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid < 32) {
      // Lane l: values 255 - 8 l and the seven below.
      int sum = 0;
      for (int v = 0; v < 8; ++v) sum += counts[255 - 8 * tid - v];
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (tid >= o) incl += x;
      }
      int above = incl - sum;
      if (above < left && left <= incl) {
        int v = 255 - 8 * tid;
        while (above + counts[v] < left) above += counts[v--];
        found[0] = v;
        found[1] = left - above;
      }
    }
    __syncthreads();
    known |= static_cast<uint32_t>(found[0]) << shift;
    left = found[1];
  }
  // Thread t: `per` pages in a row.
  const int per = (n + kTopThreads - 1) / kTopThreads;
  const int j0 = min(n, tid * per), j1 = min(n, j0 + per);
  int2 mine = make_int2(0, 0);
  for (int j = j0; j < j1; ++j) {
    const uint32_t key = key_at(j);
    mine.x += key > known;
    mine.y += key == known;
  }
  int2 before = block_prefix(mine, warps);
  for (int j = j0; j < j1; ++j) {
    const uint32_t key = key_at(j);
    if (key > known || (key == known && before.y < left)) take(p.sinks + before.x + min(before.y, left), at.lo + j);
    before.x += key > known;
    before.y += key == known;
  }
}

template <int NR>
cudaError_t launch_score(const SelectParams& p, cudaLaunchConfig_t cfg) {
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = max_dynamic_smem_once(configured, reinterpret_cast<const void*>(page_score_kernel<NR>),
                                              ScoreSmem<NR>::kAlloc);
  if (e != cudaSuccess) return e;
  // Tiles by the table's width at most; the lengths are on the device.
  const int64_t tiles = (p.max_pages - p.sinks - p.local + kTile - 1) / kTile;
  const int64_t most = tiles * p.batch * p.s;
  cfg.gridDim = dim3(static_cast<unsigned>(most < p.num_parts ? most : p.num_parts));
  cfg.blockDim = dim3(kScoreThreads);
  cfg.dynamicSmemBytes = ScoreSmem<NR>::kAlloc;
  return cudaLaunchKernelEx(&cfg, page_score_kernel<NR>, p);
}

}  // namespace

cudaError_t launch_page_select(const SelectParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  if (p.max_pages > p.top && p.top > p.sinks + p.local) {
    const cudaError_t e = p.h <= 16   ? launch_score<16>(p, cfg)
                          : p.h <= 32 ? launch_score<32>(p, cfg)
                          : p.h <= 64 ? launch_score<64>(p, cfg)
                                      : launch_score<128>(p, cfg);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(p.batch) * static_cast<unsigned>(p.s));
  cfg.blockDim = dim3(kTopThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, page_top_kernel, p);
}

}  // namespace mla
