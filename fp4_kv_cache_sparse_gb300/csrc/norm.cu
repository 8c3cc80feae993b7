// norm.cu -- residual sum, root-mean-square norm and the cast to FP8 blocks
// (include/mla.h, mla_rms_norm_fp8).
//
//   s = x + residual,  v = s / sqrt(mean(s^2) + eps) * weight,
//   per 32 values: e = least with amax 2^-e <= 448, code = e4m3(v 2^-e).
//
// One pass over the data: a thread keeps its pieces of eight elements (as
// fp32 sums) in registers between the reduction and the cast, so each input is
// read once and each output written once.  Four neighbouring lanes hold one
// 32-value block, so its maximum is two shuffles.  Rows of up to 1024 dims
// belong to a warp, longer ones to a block.  Bound by HBM.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;

// Eight consecutive elements <-> fp32.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  }
  __device__ __forceinline__ void put(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
  }
};
template <typename T>
struct Eight16 {
  uint4 w;
  __device__ __forceinline__ void load(const T* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = w; }
};
template <>
struct Eight<__half> : Eight16<__half> {
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const __half2* h = reinterpret_cast<const __half2*>(&w);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = __half22float2(h[k]);
      f[2 * k] = v.x, f[2 * k + 1] = v.y;
    }
  }
  __device__ __forceinline__ void put(const float (&f)[8]) {
    __half2* h = reinterpret_cast<__half2*>(&w);
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
  }
};
template <>
struct Eight<__nv_bfloat16> : Eight16<__nv_bfloat16> {
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(u[k] << 16);
      f[2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void put(const float (&f)[8]) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
  }
};

// kTeam threads share a row; each holds up to kPieces pieces of eight.
template <typename T, int kTeam, int kPieces>
__global__ void __launch_bounds__(kTeam < 256 ? 256 : kTeam) rms_norm_fp8_kernel(const NormParams p) {
  constexpr int kThreads = kTeam < 256 ? 256 : kTeam;
  constexpr int kTeams = kThreads / kTeam;
  __shared__ float partial[kThreads / 32];
  const int team = threadIdx.x / kTeam, tid = threadIdx.x % kTeam;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + team;
  const bool live = row < p.n;
  const int pieces = p.dim / 8;
  float s[kPieces][8];
  float sum = 0.f;
  const T* x = static_cast<const T*>(p.x) + row * p.x_row;
  const T* res = static_cast<const T*>(p.residual);
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int at = tid + i * kTeam;
#pragma unroll
    for (int k = 0; k < 8; ++k) s[i][k] = 0.f;
    if (live && at < pieces) {
      Eight<T> v;
      v.load(x + at * 8);
      v.get(s[i]);
      if (res != nullptr) {
        Eight<T> w;
        float f[8];
        w.load(res + row * p.residual_row + at * 8);
        w.get(f);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[i][k] += f[k];
      }
      if (p.residual_out != nullptr) {
        Eight<T> w;
        w.put(s[i]);
        w.store(static_cast<T*>(p.residual_out) + row * p.residual_out_row + at * 8);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = fmaf(s[i][k], s[i][k], sum);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if constexpr (kTeam > 32) {
    if ((threadIdx.x & 31) == 0) partial[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kTeam / 32; ++w) sum += partial[team * (kTeam / 32) + w];
  }
  const float r = rsqrtf(sum / static_cast<float>(p.dim) + p.eps);
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int at = tid + i * kTeam;
    // The four lanes of a block are all inside the row or all past it.
    const bool in = live && at < pieces;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    float amax = 0.f;
    if (in) {
      Eight<T> w;
      w.load(static_cast<const T*>(p.weight) + at * 8);
      w.get(v);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] *= s[i][k] * r;
        amax = fmaxf(amax, fabsf(v[k]));
      }
    }
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
    if (in) {
      const int e = fp8_block_exponent(amax);
      const float up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, exactly (e is -127 .. 120)
      uint2 c;
      c.x = e4m3x2(v[0] * up, v[1] * up) | (e4m3x2(v[2] * up, v[3] * up) << 16);
      c.y = e4m3x2(v[4] * up, v[5] * up) | (e4m3x2(v[6] * up, v[7] * up) << 16);
      *reinterpret_cast<uint2*>(p.codes + row * p.codes_row + at * 8) = c;
      if ((at & 3) == 0) p.scales[row * p.scales_row + at / 4] = static_cast<uint8_t>(127 + e);
    }
  }
}

template <typename T, int kTeam, int kPieces>
cudaError_t launch(const NormParams& p, cudaStream_t stream) {
  constexpr int kThreads = kTeam < 256 ? 256 : kTeam;
  constexpr int kTeams = kThreads / kTeam;
  const int64_t blocks = (p.n + kTeams - 1) / kTeams;
  rms_norm_fp8_kernel<T, kTeam, kPieces><<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const NormParams& p, cudaStream_t stream) {
  if (p.dim <= 256) return launch<T, 32, 1>(p, stream);
  if (p.dim <= 512) return launch<T, 32, 2>(p, stream);
  if (p.dim <= 1024) return launch<T, 32, 4>(p, stream);
  if (p.dim <= 2048) return launch<T, 128, 2>(p, stream);
  if (p.dim <= 4096) return launch<T, 256, 2>(p, stream);
  if (p.dim <= 8192) return launch<T, 256, 4>(p, stream);
  return launch<T, 512, 4>(p, stream);
}

}  // namespace

cudaError_t launch_rms_norm_fp8(int dtype, const NormParams& p, cudaStream_t stream) {
  if (dtype == MLA_FP32) return launch_typed<float>(p, stream);
  if (dtype == MLA_FP16) return launch_typed<__half>(p, stream);
  return launch_typed<__nv_bfloat16>(p, stream);
}

}  // namespace mla
