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

namespace mla {

namespace {

constexpr int kScoreThreads = 256;
constexpr int kScorePages = 64;   // pages of a block
constexpr int kCodeRow = kD + 16;  // bytes of a row of codes in shared memory, skewed
constexpr int kTopThreads = 512;
constexpr int kKeys = 8192;  // scores kept in shared memory

// Where a query token stands and what may be left out of its pages.
struct Query {
  int at;      // position, below 0 when there is no such token
  int pages;   // pages up to its own
  int lo, hi;  // pages whose scores count: all but the sinks and the last ones
};

__device__ __forceinline__ Query query_of(const SelectParams& p, int b, int i, bool& bad) {
  int len;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(len) : "l"(p.seq_lens + b) : "memory");
  bad = len < 0 || len > p.max_pages * kPage;
  Query q;
  q.at = bad ? -1 : len - p.s + i;
  q.pages = q.at < 0 ? 0 : q.at / kPage + 1;
  q.lo = p.sinks;
  q.hi = q.pages - p.local;
  return q;
}

__global__ void __launch_bounds__(kScoreThreads, 3) page_score_kernel(const SelectParams p, const int tiles) {
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* codes = smem;                                                        // [h][kCodeRow]
  uint8_t* mean = codes + p.h * kCodeRow;                                       // [warps][512]
  float* weight = reinterpret_cast<float*>(mean + (kScoreThreads / 32) * kD);  // [h]
  int* exps = reinterpret_cast<int*>(weight + p.h);                             // [h]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int query = blockIdx.x / tiles, tile = blockIdx.x - query * tiles;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  bool bad;
  const Query at = query_of(p, query / p.s, query % p.s, bad);
  if (at.pages <= p.top) return;  // all of them
  const int first = max(tile * kScorePages, at.lo), last = min((tile + 1) * kScorePages, at.hi);
  if (first >= last) return;

  for (int r = warp; r < p.h; r += kScoreThreads / 32) {
    const uint4* src = reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(query) * p.h + r) * kD + 16 * lane);
    const uint4 a = src[0], b = src[1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t two = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) asm("max.u16x2 %0, %0, %1;" : "+r"(two) : "r"(w[k] & 0x7FFF7FFFu));
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, max(two >> 16, two & 0xFFFFu));
    // amax = m 2^E, m in [1, 2): the least e with amax 2^-e <= 127 is E - 6, but for m above 127/64 (all bits set).
    const int e = max(static_cast<int>((top + 1) >> 7) - 127 - 6, -120);
    const float up = copysignf(__uint_as_float(static_cast<uint32_t>(127 - e) << 23), p.sign);
    uint32_t packed[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t v = 0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int lo = __float2int_rn(__uint_as_float(w[2 * k + j] << 16) * up);
        const int hi = __float2int_rn(__uint_as_float(w[2 * k + j] & 0xFFFF0000u) * up);
        v |= ((lo & 0xFF) | ((hi & 0xFF) << 8)) << (16 * j);
      }
      packed[k] = v;
    }
    *reinterpret_cast<uint4*>(codes + r * kCodeRow + 16 * lane) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
    if (lane == 0) exps[r] = top == 0 ? -1000 : e;
  }
  __syncthreads();
  int most = -1000;
  for (int r = 0; r < p.h; ++r) most = max(most, exps[r]);
  for (int r = tid; r < p.h; r += kScoreThreads) weight[r] = __uint_as_float(static_cast<uint32_t>(127 + max(exps[r] - most, -100)) << 23);
  __syncthreads();

  for (int page = first + warp; page < last; page += kScoreThreads / 32) {
    const int id = p.block_table[static_cast<int64_t>(query / p.s) * p.max_pages + page];
    float score = -INFINITY;
    if (id >= 0 && id < p.num_pages) {
      const uint8_t* rec = p.means + static_cast<int64_t>(id) * MLA_MEAN_BYTES;
      uint4* mine = reinterpret_cast<uint4*>(mean + warp * kD);
      mine[lane] = reinterpret_cast<const uint4*>(rec)[lane];
      const int e = static_cast<int>(rec[kD]) - 127;
      __syncwarp();
      for (int r = lane; r < p.h; r += 32) {
        const uint4* row = reinterpret_cast<const uint4*>(codes + r * kCodeRow);
        int dot = 0;
#pragma unroll 8
        for (int k = 0; k < kD / 16; ++k) {
          const uint4 a = row[k], c = mine[k];
          dot = __dp4a(static_cast<int>(a.x), static_cast<int>(c.x), dot);
          dot = __dp4a(static_cast<int>(a.y), static_cast<int>(c.y), dot);
          dot = __dp4a(static_cast<int>(a.z), static_cast<int>(c.z), dot);
          dot = __dp4a(static_cast<int>(a.w), static_cast<int>(c.w), dot);
        }
        score = fmaxf(score, static_cast<float>(dot) * weight[r]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) score = fmaxf(score, __shfl_xor_sync(0xFFFFFFFFu, score, o));
      score = ldexpf(score, e);
      __syncwarp();
    } else if (lane == 0 && p.d_error) {
      atomicOr(p.d_error, MLA_DEVERR_BAD_INDEX);
    }
    if (lane == 0) p.scores[static_cast<int64_t>(query) * p.max_pages + page] = score;
  }
}

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

}  // namespace

cudaError_t launch_page_select(const SelectParams& p, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  cudaError_t e = max_dynamic_smem_once(configured, reinterpret_cast<const void*>(page_score_kernel),
                                        128 * kCodeRow + (kScoreThreads / 32) * kD + 128 * 8);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  const int queries = p.batch * p.s;
  const int tiles = (p.max_pages + kScorePages - 1) / kScorePages;
  if (p.max_pages > p.top && p.top > p.sinks + p.local) {
    cfg.gridDim = dim3(static_cast<unsigned>(queries) * static_cast<unsigned>(tiles));
    cfg.blockDim = dim3(kScoreThreads);
    cfg.dynamicSmemBytes = p.h * kCodeRow + (kScoreThreads / 32) * kD + p.h * 8;
    e = cudaLaunchKernelEx(&cfg, page_score_kernel, p, tiles);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(queries));
  cfg.blockDim = dim3(kTopThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, page_top_kernel, p);
}

}  // namespace mla
