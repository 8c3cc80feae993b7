// paged.cu -- attention over the pages of a cache held in 4 bits
// (include/mla.h, mla_paged_decode_fp4).
//
// One block per sixteen query rows of a sequence; tiles of 32 tokens are
// decoded to fp32 in shared memory and attended with an online softmax.
#include <cstdint>
#include <cuda_bf16.h>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {

namespace {

constexpr int kRows = 16;
constexpr int kTokens = 32;
constexpr int kStride = 516;
constexpr int kSmem = (kRows + kTokens) * kStride * 4 + kRows * (kTokens + 3) * 4;

__global__ void __launch_bounds__(256) paged_simple_kernel(const PagedParams p, int groups) {
  extern __shared__ float smf[];
  float* sq = smf;
  float* sk = sq + kRows * kStride;
  float* sp = sk + kTokens * kStride;
  float* sm = sp + kRows * kTokens;
  float* sl = sm + kRows;
  float* sa = sl + kRows;
  const int tid = threadIdx.x;
  const int b = blockIdx.x / groups, r0 = (blockIdx.x % groups) * kRows;
  int len = p.seq_lens[b];
  if (len < 0 || len > p.max_pages * 64) {
    if (tid == 0 && p.d_error) atomicOr(p.d_error, MLA_DEVERR_BAD_LENGTH);
    len = 0;
  }
  const uint16_t* q = p.q + (static_cast<int64_t>(b) * p.rows + r0) * 512;
  for (int e = tid; e < kRows * 512; e += 256) {
    const int r = e >> 9;
    sq[r * kStride + (e & 511)] = r0 + r < p.rows ? __uint_as_float(static_cast<uint32_t>(q[e]) << 16) * p.scale_log2 : 0.f;
  }
  if (tid < kRows) {
    sm[tid] = -INFINITY;
    sl[tid] = 0.f;
  }
  float acc[2][kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) acc[0][r] = acc[1][r] = 0.f;
  const int first = len - p.s;
  int p_lo = first + r0 / p.h, p_hi = first + min(p.rows - 1, r0 + kRows - 1) / p.h;
  for (int t0 = 0; t0 <= p_hi; t0 += kTokens) {
    if (p.window > 0 && t0 >= p.sinks && t0 + kTokens - 1 <= p_lo - p.window) continue;
    __syncthreads();
    for (int e = tid; e < kTokens * 256; e += 256) {
      const int t = e >> 8, k = e & 255;
      float lo = 0.f, hi = 0.f;
      if (t0 + t < len) {
        const int page = p.block_table[static_cast<int64_t>(b) * p.max_pages + ((t0 + t) >> 6)];
        if (page >= 0 && page < p.num_pages) {
          const uint8_t* rec = p.kv + (static_cast<int64_t>(page) * 64 + ((t0 + t) & 63)) * kRecFp4;
          const uint32_t s16 = e4m3x2_to_f16x2(rec[256 + (k >> 3)]);
          const uint32_t v16 = e2m1x2_to_f16x2(rec[k]);
          const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(s16 & 0xFFFF)));
          lo = s * __half2float(__ushort_as_half(static_cast<unsigned short>(v16 & 0xFFFF)));
          hi = s * __half2float(__ushort_as_half(static_cast<unsigned short>(v16 >> 16)));
        }
      }
      sk[t * kStride + 2 * k] = lo;
      sk[t * kStride + 2 * k + 1] = hi;
    }
    __syncthreads();
    for (int e = tid; e < kRows * kTokens; e += 256) {
      const int r = e / kTokens, t = e % kTokens, j = t0 + t;
      const int at = first + (r0 + r) / p.h;
      bool see = r0 + r < p.rows && j <= at && (p.window == 0 || j > at - p.window || j < p.sinks);
      if (see) {
        const int page = p.block_table[static_cast<int64_t>(b) * p.max_pages + (j >> 6)];
        if (page < 0 || page >= p.num_pages) {
          see = false;
          if (p.d_error) atomicOr(p.d_error, MLA_DEVERR_BAD_INDEX);
        }
      }
      float x = 0.f;
      if (see)
        for (int d = 0; d < 512; ++d) x = fmaf(sq[r * kStride + d], sk[t * kStride + d], x);
      sp[e] = see ? x : -INFINITY;
    }
    __syncthreads();
    if (tid < kRows) {
      float m = sm[tid];
      for (int t = 0; t < kTokens; ++t) m = fmaxf(m, sp[tid * kTokens + t]);
      const float a = m == -INFINITY ? 0.f : exp2f(sm[tid] - m);
      float l = 0.f;  // the tile's own sum first, so that long rows lose no digits
      for (int t = 0; t < kTokens; ++t) {
        const float e = m == -INFINITY ? 0.f : exp2f(sp[tid * kTokens + t] - m);
        sp[tid * kTokens + t] = e;
        l += e;
      }
      sm[tid] = m;
      sl[tid] = sl[tid] * a + l;
      sa[tid] = a;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float u = acc[0][r] * sa[r], v = acc[1][r] * sa[r];
      for (int t = 0; t < kTokens; ++t) {
        u = fmaf(sp[r * kTokens + t], sk[t * kStride + 2 * tid], u);
        v = fmaf(sp[r * kTokens + t], sk[t * kStride + 2 * tid + 1], v);
      }
      acc[0][r] = u;
      acc[1][r] = v;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (r0 + r >= p.rows) break;
    const int64_t row = static_cast<int64_t>(b) * p.rows + r0 + r;
    const float inv = sl[r] > 0.f ? 1.f / sl[r] : 0.f;
    *reinterpret_cast<__nv_bfloat162*>(p.out + row * 512 + 2 * tid) =
        __floats2bfloat162_rn(acc[0][r] * inv, acc[1][r] * inv);
    if (tid == 0) p.lse[row] = sl[r] > 0.f ? (sm[r] + log2f(sl[r])) * 0.6931471805599453f : -INFINITY;
  }
}

}  // namespace

PagedPlan paged_plan(const mla_paged_problem_t* p, int num_parts) {
  PagedPlan pl{};
  const int64_t rows = static_cast<int64_t>(p->seq_len_q) * p->h_q;
  pl.nr = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
  pl.groups = static_cast<int>((rows + pl.nr - 1) / pl.nr);
  pl.num_parts = num_parts;
  pl.ws_o_bytes = static_cast<size_t>(num_parts) * 2 * pl.nr * MLA_HEAD_DIM * sizeof(float);
  pl.ws_lse_bytes = static_cast<size_t>(num_parts) * 2 * pl.nr * sizeof(float);
  pl.ws_bytes = pl.ws_o_bytes + pl.ws_lse_bytes + static_cast<size_t>(num_parts) * 4 * sizeof(int32_t);
  return pl;
}

cudaError_t launch_paged_decode(const PagedParams& p, const PagedPlan& plan, cudaStream_t stream) {
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = max_dynamic_smem_once(configured, reinterpret_cast<const void*>(paged_simple_kernel), kSmem);
  if (e != cudaSuccess) return e;
  const int groups = (p.rows + kRows - 1) / kRows;
  paged_simple_kernel<<<static_cast<unsigned>(p.batch) * groups, 256, kSmem, stream>>>(p, groups);
  return cudaGetLastError();
}

}  // namespace mla
