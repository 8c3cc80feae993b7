// page_means.cu -- the mean of a full page's 64 latents in 8 bits
// (include/mla.h, mla_page_means): what a page is about, for the selection of
// pages to read 513 bytes of it instead of 18432.
//
// A decoded value is a multiple of 2^-10 (e2m1 in halves, e4m3 in 2^-9) below
// 2^12, so the sum S_d of 64 of them is an integer below 2^28 in that unit,
// and every step here is exact: four tokens' sums fit fp32 (4 * 2688 * 2^10 <
// 2^24), the rest are 32-bit integers, in any order.  With the least e' that
// gives max |S| 2^-e' <= 127 the codes are S_d 2^-e', rounded half to even, and
// the page's scale is 2^(e' - 16).
//
// One block per page, 16 lanes to a record's 512 dims (32 each), four records a
// thread.  The next page's records are on their way while this one is summed up.
// Which pages: those whose last slot (offset 63) is in the list, as tokens are
// appended in order.  Blocks take the list's entries at an odd stride, so that
// the pages of one request, 64 entries apart, spread over all of them.
//
// 4096 pages, 78 MB, take 22.0 us: 3.5 TB/s, 53 % of a copy.  What bounds it is
// the decode, 32 conversions and 32 multiply-adds a thread and record and half
// of them again for the sums' way through shared memory (with f16 products
// turned to fp32 and added by instructions of their own 32.2 us, with the
// mixed-precision ones 25.9, with four blocks to an SM and the next page on its
// way 22.0); 128 pages, as a long prompt's chunk of 8192 tokens completes, take 3.6.
#include <cstdint>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = kPage / (kThreads / 16);  // records of a thread

struct Piece {
  uint4 data;
  uint32_t sc;
};

// acc += the 32 dims' values under two e4m3 scales: f16 codes times f16 scales
// into fp32 by single instructions, exact each.  A NaN scale counts as 448 of its sign.
__device__ __forceinline__ void add32(const Piece& p, float (&acc)[32]) {
  uint32_t s2 = e4m3x2_to_f16x2(p.sc & 0x7F7Fu);
  asm("min.f16x2 %0, %0, %1;" : "+r"(s2) : "r"(0x5F005F00u));
  s2 |= (p.sc & 0x80u) << 8 | (p.sc & 0x8000u) << 16;
  const uint32_t w[4] = {p.data.x, p.data.y, p.data.z, p.data.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t s = k < 2 ? s2 : s2 >> 16;
    float* o = acc + 8 * k;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t.reg .b32 h0, h1, h2, h3;\n\t.reg .b16 s, t, l0, u0, l1, u1, l2, u2, l3, u3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %8;\n\t"
        "mov.b32 {s, t}, %9;\n\t"
        "cvt.rn.f16x2.e2m1x2 h0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 h1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 h2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 h3, b3;\n\t"
        "mov.b32 {l0, u0}, h0;\n\tmov.b32 {l1, u1}, h1;\n\tmov.b32 {l2, u2}, h2;\n\tmov.b32 {l3, u3}, h3;\n\t"
        "fma.rn.f32.f16 %0, l0, s, %0;\n\t"
        "fma.rn.f32.f16 %1, u0, s, %1;\n\t"
        "fma.rn.f32.f16 %2, l1, s, %2;\n\t"
        "fma.rn.f32.f16 %3, u1, s, %3;\n\t"
        "fma.rn.f32.f16 %4, l2, s, %4;\n\t"
        "fma.rn.f32.f16 %5, u2, s, %5;\n\t"
        "fma.rn.f32.f16 %6, l3, s, %6;\n\t"
        "fma.rn.f32.f16 %7, u3, s, %7;\n\t}"
        : "+f"(o[0]), "+f"(o[1]), "+f"(o[2]), "+f"(o[3]), "+f"(o[4]), "+f"(o[5]), "+f"(o[6]), "+f"(o[7])
        : "r"(w[k]), "r"(s));
  }
}

// Every 32 dims the columns are skewed by 4 words, so that lanes that write 32
// words each do not meet in the same banks.
__device__ __forceinline__ int column(int d) { return d + (d >> 5) * 4; }
constexpr int kRow = kD + (kD / 32) * 4;

__global__ void __launch_bounds__(kThreads, 4)
    page_means_kernel(const uint8_t* pool, int64_t pool_tokens, const int32_t* slots, int64_t n, uint8_t* means,
                      int32_t* d_error) {
  __shared__ float sums[kThreads / 16][kRow];  // of four tokens each
  __shared__ int32_t pages[kThreads];
  __shared__ uint32_t counts[kThreads / 32];
  __shared__ uint32_t tops[kThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");

  for (int64_t base = blockIdx.x; base < n; base += static_cast<int64_t>(gridDim.x) * kThreads) {
    // Up to kThreads entries of the list; those that complete a page, in order.
    const int64_t i = base + static_cast<int64_t>(tid) * gridDim.x;
    int32_t slot = -1;
    if (i < n) slot = slots[i];
    const bool good = slot >= 0 && slot < pool_tokens;
    if (!good && slot != -1 && d_error) atomicOr(d_error, MLA_DEVERR_BAD_INDEX);
    const bool full = good && slot % kPage == kPage - 1;
    const uint32_t vote = __ballot_sync(0xFFFFFFFFu, full);
    if (lane == 0) counts[warp] = __popc(vote);
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += counts[w];
      total += counts[w];
    }
    if (full) pages[before + __popc(vote & ((1u << lane) - 1))] = slot / kPage;
    __syncthreads();

    Piece next[kTokens];
    const auto fetch = [&](int k) {
      const uint8_t* rec = pool + (static_cast<int64_t>(pages[k]) * kPage + (tid >> 4) * kTokens) * kRecFp4;
#pragma unroll
      for (int j = 0; j < kTokens; ++j) {
        next[j].data = *reinterpret_cast<const uint4*>(rec + j * kRecFp4 + (tid & 15) * 16);
        next[j].sc = *reinterpret_cast<const uint16_t*>(rec + j * kRecFp4 + 256 + (tid & 15) * 2);
      }
    };
    if (total > 0) fetch(0);
    for (int k = 0; k < total; ++k) {
      float acc[32];
#pragma unroll
      for (int c = 0; c < 32; ++c) acc[c] = 0.f;
#pragma unroll
      for (int j = 0; j < kTokens; ++j) add32(next[j], acc);
      if (k + 1 < total) fetch(k + 1);
      float* mine = &sums[tid >> 4][column((tid & 15) * 32)];
#pragma unroll
      for (int c = 0; c < 32; c += 4)
        *reinterpret_cast<float4*>(mine + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
      __syncthreads();
      // Thread t: dims 2 t and 2 t + 1, in units of 2^-10.
      int a = 0, b = 0;
#pragma unroll
      for (int g = 0; g < kThreads / 16; ++g) {
        const float2 v = *reinterpret_cast<const float2*>(&sums[g][column(2 * tid)]);
        a += static_cast<int>(v.x * 1024.f);
        b += static_cast<int>(v.y * 1024.f);
      }
      uint32_t top = max(abs(a), abs(b));
      top = __reduce_max_sync(0xFFFFFFFFu, top);
      if (lane == 0) tops[warp] = top;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) top = max(top, tops[w]);
      // 2^e' with top * 2^-e' in (63.5, 127].
      int e = 0;
      if (top > 0) {
        e = 25 - __clz(top);  // the leading bit to 2^6
        if (e > 0 && top > (127u << e)) ++e;
      }
      const auto code = [&](int v) -> uint32_t {
        if (e <= 0) return static_cast<uint32_t>(v * (1 << -e)) & 0xFFu;
        // Half to even: what is added makes exact halves carry only into odd codes.
        return static_cast<uint32_t>((v + (1 << (e - 1)) - 1 + ((v >> e) & 1)) >> e) & 0xFFu;
      };
      uint8_t* rec = means + static_cast<int64_t>(pages[k]) * MLA_MEAN_BYTES;
      *reinterpret_cast<uint16_t*>(rec + 2 * tid) = static_cast<uint16_t>(code(a) | (code(b) << 8));
      if (tid < 4)
        *reinterpret_cast<uint32_t*>(rec + kD + 4 * tid) = tid == 0 ? static_cast<uint32_t>(127 + (top > 0 ? e - 16 : 0)) : 0u;
    }
    __syncthreads();  // the page list may change again
  }
}

}  // namespace

cudaError_t launch_page_means(const uint8_t* pool, int64_t pool_tokens, const int32_t* slots, int64_t n, uint8_t* means,
                              int32_t* d_error, cudaStream_t stream) {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t most = static_cast<int64_t>(sms) * 4 - 1;  // odd; all of them resident
  const int64_t blocks = n < most ? n : most;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  return cudaLaunchKernelEx(&cfg, page_means_kernel, pool, pool_tokens, slots, n, means, d_error);
}

}  // namespace mla
