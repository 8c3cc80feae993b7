// shared_merge.cu -- the end of a decode with shared prefixes (include/mla.h,
// mla_paged_shared_decode_fp4): a query row's partials over its own tokens and
// over its group's prefix, each in one piece or in several, become its output.
//
// Pieces with normalised outputs o_i and log-sum-exps L_i give
// L = ln sum exp L_i and out = sum exp(L_i - L) o_i, in fp32, rounded once.
// The pieces' order is that of the sum, so the result is the same every time.
//
// Bound by bytes: 8192 rows (64 x 128 heads) with some three pieces of 2 KB each
// are 58 MB with their outputs and take 11 us behind the kernel that writes them,
// 5 TB/s, out of L2 for the most part.
#include <cstdint>
#include <cuda_bf16.h>

#include "mla_device.cuh"
#include "mla_internal.h"
#include "mla_tensor.cuh"

namespace mla {

namespace {

// Where the pieces of a unit lie: in its own slot when it is whole, otherwise
// in the first part's slot 2 part + 1 and the slots 2 part of those that follow.
struct Pieces {
  int part, count;  // count 0: none
  int64_t whole;    // slot when it is whole, else -1
  int r;            // row of the unit
  __device__ __forceinline__ int64_t slot(int i) const {
    return whole >= 0 ? whole : (static_cast<int64_t>(part) + i) * 2 + (i == 0 ? 1 : 0);
  }
};
__device__ __forceinline__ Pieces pieces_of(const SharedParams& p, int num_parts, int u, int r) {
  const int4 entry = *reinterpret_cast<const int4*>(p.ws_info + static_cast<int64_t>(u) * 4);
  if (entry.x < 0) return Pieces{0, 1, 2ll * num_parts + u, r};
  return Pieces{entry.y, entry.z - entry.y + 1, -1, r};
}

// A query row and its pieces: first those of its own tokens, then the prefix's.
struct Row {
  Pieces own, prefix;
  int nr;
  __device__ __forceinline__ int count() const { return own.count + prefix.count; }
  __device__ __forceinline__ int64_t at(int i) const {
    return i < own.count ? own.slot(i) * nr + own.r : prefix.slot(i - own.count) * nr + prefix.r;
  }
};
__device__ __forceinline__ Row row_of(const SharedParams& p, int groups, int nr, int num_parts, int row) {
  Row t{};
  t.nr = nr;
  const int b = row / p.rows, r = row - b * p.rows;
  t.own = pieces_of(p, num_parts, b * groups + r / nr, r % nr);
  const int len = load_i32(p.seq_lens + b);
  const int num_groups = load_i32(p.ws_info + static_cast<int64_t>(p.units) * 4);
  const bool bad = len < 0 || len > p.max_pages * kPage;
  // A query token that does not exist sees no prefix either.
  if (num_groups == 0 || bad || len - p.s + r / p.h < 0) return t;
  int g = 0;  // the last group that begins at or before b
  for (int n = num_groups; n > 1;) {
    const int half = n / 2;
    if (load_i32(p.group_start + g + half) <= b) g += half;
    n -= half;
  }
  const int from = load_i32(p.group_start + g), to = load_i32(p.group_start + g + 1);
  const int prefix = load_i32(p.prefix_lens + g);
  if (b < from || b >= to || prefix <= 0 || prefix > p.max_prefix_pages * kPage) return t;
  const int off = row - from * p.rows;
  t.prefix = pieces_of(p, num_parts, p.batch * groups + from * p.rows / nr + g + off / nr, off % nr);
  return t;
}

// The pieces' largest log-sum-exp (0 if all are empty) and the sum of their weights.
__device__ __forceinline__ float weights(const SharedParams& p, const Row& t, float& m) {
  const int lane = threadIdx.x & 31;
  m = -INFINITY;
  for (int i = lane; i < t.count(); i += 32) m = fmaxf(m, p.ws_lse[t.at(i)]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (m == -INFINITY) m = 0.f;
  float z = 0.f;
  for (int i = lane; i < t.count(); i += 32) z += expf(p.ws_lse[t.at(i)] - m);
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

// A warp per row, for units in few pieces.
__global__ void __launch_bounds__(128) shared_merge_kernel(const SharedParams p, const int groups, const int nr,
                                                           const int num_parts) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(p.batch) * p.rows) return;
  const Row t = row_of(p, groups, nr, num_parts, static_cast<int>(row));
  float m;
  const float z = weights(p, t, m);
  const float inv = z > 0.f ? 1.f / z : 0.f;
  float4 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int i = 0; i < t.count(); ++i) {
    const int64_t at = t.at(i);
    const float4* src = reinterpret_cast<const float4*>(p.ws_o + at * kD);
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = src[k * 32 + lane];
    const float w = expf(p.ws_lse[at] - m) * inv;
#pragma unroll
    for (int k = 0; k < 4; ++k) add_piece(acc[k], w, v[k]);
  }
  uint2* dst = reinterpret_cast<uint2*>(p.out + row * kD);
#pragma unroll
  for (int k = 0; k < 4; ++k) dst[k * 32 + lane] = four_bf16(acc[k]);
  if (lane == 0) p.lse[row] = z > 0.f ? m + logf(z) : -INFINITY;
}

// A block per row, for units in many: four groups of 128 threads share them.
__global__ void __launch_bounds__(512) shared_merge_many_kernel(const SharedParams p, const int groups, const int nr,
                                                                const int num_parts) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float4 sums[3][128];
  const int team = threadIdx.x >> 7, tid = threadIdx.x & 127;
  const int64_t row = blockIdx.x;
  const Row t = row_of(p, groups, nr, num_parts, static_cast<int>(row));
  float m;
  const float z = weights(p, t, m);
  const float inv = z > 0.f ? 1.f / z : 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = team; i < t.count(); i += 16) {  // four of the team's pieces in flight
    float4 v[4];
    float w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t at = t.at(min(i + 4 * j, t.count() - 1));
      v[j] = *reinterpret_cast<const float4*>(p.ws_o + at * kD + tid * 4);
      w[j] = i + 4 * j < t.count() ? p.ws_lse[at] : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) add_piece(acc, expf(w[j] - m) * inv, v[j]);
  }
  if (team > 0) sums[team - 1][tid] = acc;
  __syncthreads();
  if (team > 0) return;
#pragma unroll
  for (int g = 0; g < 3; ++g) add_piece(acc, 1.f, sums[g][tid]);
  *reinterpret_cast<uint2*>(p.out + row * kD + tid * 4) = four_bf16(acc);
  if (tid == 0) p.lse[row] = z > 0.f ? m + logf(z) : -INFINITY;
}

}  // namespace

cudaError_t launch_shared_merge(const SharedParams& p, const PagedPlan& plan, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.batch) * p.rows;
  const bool many = static_cast<int64_t>(plan.units) * 6 <= plan.num_parts;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3(static_cast<unsigned>(many ? rows : (rows + 3) / 4));
  cfg.blockDim = dim3(many ? 512 : 128);
  return cudaLaunchKernelEx(&cfg, many ? shared_merge_many_kernel : shared_merge_kernel, p, plan.groups, plan.nr,
                            plan.num_parts);
}

}  // namespace mla
