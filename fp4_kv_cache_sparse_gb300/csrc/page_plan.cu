// page_plan.cu -- block tables and slot maps from request lengths, on the
// device (include/mla.h, mla_page_plan).
//
// One cluster of eight CTAs changes the state.  Every CTA scans all requests
// (three prefix sums: new tokens, pages taken, pages given back) into its own
// shared memory, so nothing but one cluster barrier stands between reading the
// old state and writing the new one in place: before it the ended requests'
// pages are pushed, after it pages are popped and lengths replaced.  A short
// slot map is written by the same 8192 threads, each finding its tokens'
// request by a binary search of the prefix in shared memory; a long one by a
// second kernel over the whole GPU, from the tables and lengths that the first
// has left (1000 requests: 512,000 slots 24.6 us in the cluster, 10.4 us so;
// 64,000 slots 8.5 against 10.3).  One decode step of 256 requests takes 5.5
// us: latency alone, a launch, three dependent trips to memory and three
// barriers.
#include <cstdint>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {

namespace {

constexpr int kCtas = 8;
constexpr int kPlanThreads = 1024;
constexpr int kLongMap = 96 * 1024;  // slots from which a kernel of its own writes the map

struct Sums {
  int64_t tokens, take, give;
};

__device__ __forceinline__ int64_t shfl_up64(int64_t v, int d) { return __shfl_up_sync(0xFFFFFFFFu, v, d); }

// Inclusive scan over the block's threads; total gets the block's sums.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* warp_sums, Sums& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t a = shfl_up64(v.tokens, d), b = shfl_up64(v.take, d), c = shfl_up64(v.give, d);
    if (lane >= d) v.tokens += a, v.take += b, v.give += c;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    Sums w = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t a = shfl_up64(w.tokens, d), b = shfl_up64(w.take, d), c = shfl_up64(w.give, d);
      if (lane >= d) w.tokens += a, w.take += b, w.give += c;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  if (warp > 0) {
    const Sums w = warp_sums[warp - 1];
    v.tokens += w.tokens, v.take += w.take, v.give += w.give;
  }
  total = warp_sums[31];
  return v;
}

__device__ __forceinline__ int32_t pages_of(uint32_t tokens) { return static_cast<int32_t>((tokens + 63u) >> 6); }

// The last request that starts at or before token i < prefix[batch].
__device__ __forceinline__ int request_of(const int32_t* prefix, int batch, int32_t i) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= i)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ void store_four(int32_t* slots, int32_t* positions, int64_t i0, int max_new,
                                           const int32_t (&slot)[4], const int32_t (&pos)[4]) {
  if (i0 + 4 <= max_new && ((reinterpret_cast<uintptr_t>(slots) | reinterpret_cast<uintptr_t>(positions)) & 15u) == 0) {
    *reinterpret_cast<int4*>(slots + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    *reinterpret_cast<int4*>(positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i0 + k < max_new) {
        slots[i0 + k] = slot[k];
        positions[i0 + k] = pos[k];
      }
    }
  }
}

// The slot map of a plan that has been made: request r's new tokens stand at
// the end of its new length, and its row holds every page.  (No __restrict__ on
// what the plan writes: this kernel starts while that one ends, and a
// non-coherent load may be moved above the wait.)
__global__ void __launch_bounds__(256) slot_map_kernel(const int32_t* cu_new, const int32_t* seq_lens, int batch,
                                                       const int32_t* block_table, int max_pages, int num_pages,
                                                       int32_t* __restrict__ slots,
                                                       int32_t* __restrict__ positions, int max_new, int32_t* d_error) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int32_t tokens = cu_new[batch];
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (i0 >= max_new) return;
  int32_t slot[4], pos[4];
  bool bad_page = false;
  int r = i0 < tokens ? request_of(cu_new, batch, static_cast<int32_t>(i0)) : 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t i = i0 + k;
    slot[k] = -1;
    pos[k] = 0;
    if (i < tokens) {
      while (i >= cu_new[r + 1]) ++r;
      const int32_t p = seq_lens[r] - (cu_new[r + 1] - static_cast<int32_t>(i));
      const int32_t page = block_table[static_cast<int64_t>(r) * max_pages + (p >> 6)];
      const bool good = page >= 0 && page < num_pages;
      bad_page |= !good;
      slot[k] = good ? page * 64 + (p & 63) : -1;
      pos[k] = p;
    }
  }
  store_four(slots, positions, i0, max_new, slot, pos);
  if (bad_page && d_error) atomicOr(d_error, MLA_DEVERR_BAD_INDEX);
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kPlanThreads)
    page_plan_kernel(const int32_t* cached_lens, const int32_t* __restrict__ new_lens, int batch,
                     int32_t* __restrict__ block_table, int max_pages, int32_t* free_pages, int num_pages,
                     const int32_t* num_free, int32_t* seq_lens, int32_t* num_free_out, int32_t* __restrict__ cu_new,
                     int32_t* __restrict__ slots, int32_t* __restrict__ positions, int max_new, int map_len,
                     int32_t* d_error) {
  extern __shared__ int32_t sm[];
  int32_t* s_cu = sm;                    // [batch + 1] first new token
  int32_t* s_take = s_cu + batch + 1;    // [batch + 1] pages taken before this request
  int32_t* s_give = s_take + batch + 1;  // [batch + 1] pages given back before it
  int32_t* s_len = s_give + batch + 1;   // [batch] cached tokens (seq_lens may be cached_lens)
  __shared__ Sums warp_sums[32];
  const int tid = threadIdx.x;
  const int rank = static_cast<int>(blockIdx.x);

  // Each thread sums a run of consecutive requests.
  const int per = (batch + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(batch, tid * per), r1 = min(batch, r0 + per);
  const int64_t most = static_cast<int64_t>(max_pages) * 64;
  Sums mine{0, 0, 0};
  bool bad = false;
  for (int r = r0; r < r1; ++r) {
    const int32_t c = cached_lens[r], n = new_lens[r];
    s_len[r] = c;
    bad |= c < 0 || n < -1 || static_cast<int64_t>(c) + max(n, 0) > most;
    if (n >= 0) {
      mine.tokens += n;
      mine.take += pages_of(static_cast<uint32_t>(c) + n) - pages_of(c);
    } else {
      mine.give += pages_of(c);
    }
  }
  const int32_t nf = *num_free;
  Sums total;
  const Sums upto = block_scan(mine, warp_sums, total);
  bad = __syncthreads_or(bad);
  int32_t why = 0;
  if (bad) why |= MLA_DEVERR_BAD_LENGTH;
  if (nf < 0 || nf > num_pages || (!bad && total.give > num_pages - nf)) why |= MLA_DEVERR_BAD_METADATA;
  if (!why && (total.tokens > max_new || total.take > nf + total.give)) why |= MLA_DEVERR_NO_ROOM;
  const bool ok = why == 0;
  const int32_t top = ok ? nf + static_cast<int32_t>(total.give) : nf;
  const int32_t tokens = ok ? static_cast<int32_t>(total.tokens) : 0;
  Sums run{upto.tokens - mine.tokens, upto.take - mine.take, upto.give - mine.give};
  for (int r = r0; r < r1; ++r) {
    const int32_t c = s_len[r], n = new_lens[r];
    s_cu[r] = ok ? static_cast<int32_t>(run.tokens) : 0;
    s_take[r] = ok ? static_cast<int32_t>(run.take) : 0;
    s_give[r] = ok ? static_cast<int32_t>(run.give) : 0;
    if (n >= 0) {
      run.tokens += n;
      run.take += pages_of(static_cast<uint32_t>(c) + n) - pages_of(c);
    } else {
      run.give += pages_of(c);
    }
  }
  if (tid == 0) {
    s_cu[batch] = tokens;
    s_take[batch] = ok ? static_cast<int32_t>(total.take) : 0;
    s_give[batch] = ok ? static_cast<int32_t>(total.give) : 0;
  }
  __syncthreads();

  // A warp to each request where that takes one round of a few pages; else a
  // thread to each page, its request found by a search (256 requests of one
  // token: 5.5 us by warps, 5.8 by pages; 1000 of up to 512 tokens: 12.7 and 10.3;
  // 4 of 50,000: 9.9 and 6.1; 500 of which 250 end: 11.3 and 12.4).
  const int gtid = rank * kPlanThreads + tid, lane = tid & 31, warp = gtid >> 5;
  constexpr int kAll = kCtas * kPlanThreads;
  const bool by_warp = batch <= kAll / 32 && s_give[batch] + s_take[batch] <= 32 * batch;
  bool bad_page = false;
  const auto give = [&](int r, int32_t i, int32_t k) {  // page i of all comes back: entry k of request r's row
    const int32_t page = block_table[static_cast<int64_t>(r) * max_pages + k];
    bad_page |= page < 0 || page >= num_pages;
    free_pages[nf + i] = page;
  };
  if (by_warp) {
    if (warp < batch) {
      const int32_t g0 = s_give[warp], n = s_give[warp + 1] - g0;
      for (int k = lane; k < n; k += 32) give(warp, g0 + k, k);
    }
  } else {
    for (int32_t i = gtid; i < s_give[batch]; i += kAll) {
      const int r = request_of(s_give, batch, i);
      give(r, i, i - s_give[r]);
    }
  }
  // Everyone has read the old lengths and the pushed pages are visible.
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");

  const auto take = [&](int r, int32_t i) {  // page i of all goes to request r
    const int32_t page = free_pages[top - 1 - i];
    bad_page |= page < 0 || page >= num_pages;
    block_table[static_cast<int64_t>(r) * max_pages + pages_of(s_len[r]) + (i - s_take[r])] = page;
  };
  if (by_warp) {
    if (warp < batch)
      for (int32_t i = s_take[warp] + lane; i < s_take[warp + 1]; i += 32) take(warp, i);
  } else {
    for (int32_t i = gtid; i < s_take[batch]; i += kAll) take(request_of(s_take, batch, i), i);
  }
  for (int r = gtid; r < batch; r += kAll) {
    seq_lens[r] = ok ? (new_lens[r] < 0 ? 0 : s_len[r] + s_cu[r + 1] - s_cu[r]) : s_len[r];
    cu_new[r] = s_cu[r];
  }
  if (gtid == 0) {
    cu_new[batch] = tokens;
    *num_free_out = top - s_take[batch];
    if (why && d_error) atomicOr(d_error, why);
  }

  // Slots and positions, four tokens to a thread (none here when the map is long).
  for (int64_t i0 = static_cast<int64_t>(gtid) * 4; i0 < map_len; i0 += static_cast<int64_t>(kAll) * 4) {
    int32_t slot[4], pos[4];
    int r = i0 < tokens ? request_of(s_cu, batch, static_cast<int32_t>(i0)) : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = i0 + k;
      slot[k] = -1;
      pos[k] = 0;
      if (i < tokens) {
        while (i >= s_cu[r + 1]) ++r;
        const int32_t p = s_len[r] + static_cast<int32_t>(i - s_cu[r]);
        const int32_t held = pages_of(s_len[r]), at = p >> 6;
        const int32_t page = at < held ? block_table[static_cast<int64_t>(r) * max_pages + at]
                                       : free_pages[top - 1 - (s_take[r] + at - held)];
        const bool good = page >= 0 && page < num_pages;
        bad_page |= !good;
        slot[k] = good ? page * 64 + (p & 63) : -1;
        pos[k] = p;
      }
    }
    store_four(slots, positions, i0, max_new, slot, pos);
  }
  if (bad_page && d_error) atomicOr(d_error, MLA_DEVERR_BAD_INDEX);
}

}  // namespace

cudaError_t launch_page_plan(const int32_t* cached_lens, const int32_t* new_lens, int batch, int32_t* block_table,
                             int max_pages, int32_t* free_pages, int num_pages, const int32_t* num_free,
                             int32_t* seq_lens, int32_t* num_free_out, int32_t* cu_new, int32_t* slots,
                             int32_t* positions, int max_new, int32_t* d_error, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  constexpr int kMost = (4 * kPlanMaxBatch + 3) * static_cast<int>(sizeof(int32_t));
  const cudaError_t e = max_dynamic_smem_once(configured, reinterpret_cast<const void*>(page_plan_kernel), kMost);
  if (e != cudaSuccess) return e;
  const size_t smem = (4 * static_cast<size_t>(batch) + 3) * sizeof(int32_t);
  const bool long_map = max_new > kLongMap;
  page_plan_kernel<<<kCtas, kPlanThreads, smem, stream>>>(
      cached_lens, new_lens, batch, block_table, max_pages, free_pages, num_pages, num_free, seq_lens, num_free_out,
      cu_new, slots, positions, max_new, long_map ? 0 : max_new, d_error);
  cudaError_t launched = cudaGetLastError();
  if (launched != cudaSuccess || !long_map) return launched;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<int64_t>(max_new) + 1023) / 1024));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, slot_map_kernel, static_cast<const int32_t*>(cu_new),
                            static_cast<const int32_t*>(seq_lens), batch, static_cast<const int32_t*>(block_table),
                            max_pages, num_pages, slots, positions, max_new, d_error);
}

}  // namespace mla
