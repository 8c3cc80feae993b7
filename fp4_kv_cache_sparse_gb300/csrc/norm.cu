// norm.cu -- residual sum, root-mean-square norm and the cast to FP8 blocks
// (include/mla.h, mla_rms_norm_fp8).
//
//   s = x + residual,  v = s / sqrt(mean(s^2) + eps) * weight,
//   per 32 values: e = least with amax 2^-e <= 448, code = e4m3(v 2^-e).
//
// One pass over the data: each input is read once and each output written
// once, with the row's sums in registers between.  Four neighbouring lanes hold one
// 32-value block, so its maximum is two shuffles.  Rows of up to 512 dims
// belong to a warp, longer ones to as many warps as hold two pieces a thread.
// Bound by HBM.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {

namespace {

constexpr unsigned kFull = 0xFFFFFFFFu;
constexpr int kMaxStages = 8;
constexpr int kNormSmem = 200 * 1024;               // of an SM's shared memory, for the rings of its blocks
constexpr uint64_t kNormWaitNs = 2000000000ull;     // 2 s per wait

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

// 1 / rms is applied with the block's scale: v holds weight * s, the block's
// maximum and its codes take inv once.
__device__ __forceinline__ void store_block(const NormParams& p, int64_t row, int at, bool in, const float (&v)[8],
                                            float inv) {
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(v[k]));
  // Four lanes hold a block; they are all inside the row or all past it.
  amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
  if (!in) return;
  const int e = fp8_block_exponent(amax * inv);
  const float up = inv * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e exactly: e is -127 .. 120
  uint2 c;
  c.x = e4m3x2(v[0] * up, v[1] * up) | (e4m3x2(v[2] * up, v[3] * up) << 16);
  c.y = e4m3x2(v[4] * up, v[5] * up) | (e4m3x2(v[6] * up, v[7] * up) << 16);
  *reinterpret_cast<uint2*>(p.codes + row * p.codes_row + at * 8) = c;
  if ((at & 3) == 0) p.scales[row * p.scales_row + at / 4] = static_cast<uint8_t>(127 + e);
}

template <int kTeam>
constexpr int threads_of() {
  return kTeam < 256 ? 256 : kTeam;
}
template <int kTeam>
constexpr int resident_of() {  // blocks of an SM that the registers are limited for
  return kTeam < 256 ? 4 : 1024 / kTeam;
}

// Sum over a team's threads; two sets of partial sums in turn, so that one
// barrier a row suffices.
template <int kTeam>
__device__ __forceinline__ float team_sum(float sum, float (&partial)[threads_of<kTeam>() / 32], int team) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if constexpr (kTeam > 32) {
    if ((threadIdx.x & 31) == 0) partial[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int k = 0; k < kTeam / 32; ++k) sum += partial[team * (kTeam / 32) + k];
  }
  return sum;
}

// kTeam threads share a row and go on from row to row, `stages` rows ahead of
// themselves: the rows (and the residual's) come by bulk copies into a ring in
// shared memory, so what is in flight costs no registers.  A thread holds two
// pieces of eight of a row as fp32 sums between the reduction and the cast,
// and its piece of the weight for good.
template <typename T, int kTeam, bool kRes>
__global__ void __launch_bounds__(threads_of<kTeam>(), resident_of<kTeam>())
    rms_norm_fp8_kernel(const NormParams p, const int stages) {
  constexpr int kThreads = threads_of<kTeam>(), kTeams = kThreads / kTeam, kPieces = 2;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kTeams * kMaxStages];
  __shared__ float partial[2][kThreads / 32];
  __shared__ int gave_up;
  const int team = threadIdx.x / kTeam, tid = threadIdx.x % kTeam;
  const uint32_t row_bytes = static_cast<uint32_t>(p.dim) * sizeof(T), stage_bytes = row_bytes * (kRes ? 2 : 1);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kTeams * kMaxStages; ++i) mbar_init(&full[i], 1);
    gave_up = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  uint8_t* mine = ring + static_cast<size_t>(team) * stages * stage_bytes;
  uint64_t* bars = full + team * kMaxStages;
  const int pieces = p.dim / 8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kTeams;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + team;
  const auto request = [&](int64_t r, int slot) {
    if (tid != 0 || r >= p.n) return;
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(
                     smem_u32(&bars[slot])),
                 "r"(stage_bytes)
                 : "memory");
    const auto copy = [&](uint8_t* dst, const void* src) {
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                       smem_u32(dst)),
                   "l"(src), "r"(row_bytes), "r"(smem_u32(&bars[slot]))
                   : "memory");
    };
    copy(mine + slot * stage_bytes, static_cast<const T*>(p.x) + r * p.x_row);
    if constexpr (kRes) copy(mine + slot * stage_bytes + row_bytes, static_cast<const T*>(p.residual) + r * p.residual_row);
  };
  for (int i = 0; i < stages; ++i) request(row + i * stride, i);
  Eight<T> w[kPieces];
#pragma unroll
  for (int i = 0; i < kPieces; ++i)
    if (tid + i * kTeam < pieces) w[i].load(static_cast<const T*>(p.weight) + (tid + i * kTeam) * 8);
  const float inv_dim = 1.f / static_cast<float>(p.dim);
  int slot = 0, side = 0;
  uint32_t parity = 0;
  // Every team of a block makes the same number of rounds (the block's barrier).
  for (int64_t first = row - team; first < p.n; first += stride, row += stride, side ^= 1) {
    const bool live = row < p.n;
    if (live) mbar_wait(&bars[slot], parity, &gave_up, nullptr, kNormWaitNs);
    __syncwarp();
    const T* src = reinterpret_cast<const T*>(mine + slot * stage_bytes);
    float s[kPieces][8];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = tid + i * kTeam;
#pragma unroll
      for (int k = 0; k < 8; ++k) s[i][k] = 0.f;
      if (live && at < pieces) {
        Eight<T> x;
        x.load(src + at * 8);
        x.get(s[i]);
        if constexpr (kRes) {
          float f[8];
          x.load(src + p.dim + at * 8);
          x.get(f);
#pragma unroll
          for (int k = 0; k < 8; ++k) s[i][k] += f[k];
        }
        if (p.residual_out != nullptr) {
          x.put(s[i]);
          x.store(static_cast<T*>(p.residual_out) + row * p.residual_out_row + at * 8);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) sum = fmaf(s[i][k], s[i][k], sum);
      }
    }
    sum = team_sum<kTeam>(sum, partial[side], team);
    // The whole team has read the row: its place takes the one `stages` rows on.
    request(row + stages * stride, slot);
    if (++slot == stages) slot = 0, parity ^= 1;
    const float inv = rsqrtf(fmaf(sum, inv_dim, p.eps));
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int at = tid + i * kTeam;
      const bool in = live && at < pieces;
      float v[8];
      w[i].get(v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = in ? v[k] * s[i][k] : 0.f;
      store_block(p, row, at, in, v, inv);
    }
  }
}

// Rows too long for two of them in shared memory: a block each, loaded into
// registers.
template <typename T>
__global__ void __launch_bounds__(512) rms_norm_fp8_long_kernel(const NormParams p) {
  constexpr int kTeam = 512, kPieces = 4;
  __shared__ float partial[kTeam / 32];
  const int tid = threadIdx.x;
  const int pieces = p.dim / 8;
  const int64_t row = blockIdx.x;
  const T* res = static_cast<const T*>(p.residual);
  float s[kPieces][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int at = tid + i * kTeam;
#pragma unroll
    for (int k = 0; k < 8; ++k) s[i][k] = 0.f;
    if (at < pieces) {
      Eight<T> x;
      x.load(static_cast<const T*>(p.x) + row * p.x_row + at * 8);
      x.get(s[i]);
      if (res != nullptr) {
        float f[8];
        x.load(res + row * p.residual_row + at * 8);
        x.get(f);
#pragma unroll
        for (int k = 0; k < 8; ++k) s[i][k] += f[k];
      }
      if (p.residual_out != nullptr) {
        x.put(s[i]);
        x.store(static_cast<T*>(p.residual_out) + row * p.residual_out_row + at * 8);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) sum = fmaf(s[i][k], s[i][k], sum);
    }
  }
  sum = team_sum<kTeam>(sum, partial, 0);
  const float inv = rsqrtf(fmaf(sum, 1.f / static_cast<float>(p.dim), p.eps));
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int at = tid + i * kTeam;
    const bool in = at < pieces;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (in) {
      Eight<T> w;
      w.load(static_cast<const T*>(p.weight) + at * 8);
      w.get(v);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= s[i][k];
    }
    store_block(p, row, at, in, v, inv);
  }
}

template <typename T, int kTeam, bool kRes>
cudaError_t launch_ring(const NormParams& p, cudaStream_t stream) {
  constexpr int kThreads = threads_of<kTeam>(), kTeams = kThreads / kTeam;
  const int round = kTeams * p.dim * static_cast<int>(sizeof(T)) * (kRes ? 2 : 1);  // one stage of every team
  // As many blocks on an SM as leave each two stages at least.
  int per_sm = resident_of<kTeam>();
  while (per_sm > 1 && kNormSmem / per_sm / round < 2) --per_sm;
  int stages = kNormSmem / per_sm / round;
  if (stages > kMaxStages) stages = kMaxStages;
  static std::atomic<uint64_t> configured{0};
  const cudaError_t e = max_dynamic_smem_once(
      configured, reinterpret_cast<const void*>(rms_norm_fp8_kernel<T, kTeam, kRes>), kNormSmem);
  if (e != cudaSuccess) return e;
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int64_t blocks = (p.n + kTeams - 1) / kTeams;
  const int64_t cap = static_cast<int64_t>(sms) * per_sm;
  if (blocks > cap) blocks = cap;
  rms_norm_fp8_kernel<T, kTeam, kRes>
      <<<static_cast<unsigned>(blocks), kThreads, static_cast<size_t>(stages) * round, stream>>>(p, stages);
  return cudaGetLastError();
}

template <typename T, int kTeam>
cudaError_t launch(const NormParams& p, cudaStream_t stream) {
  return p.residual != nullptr ? launch_ring<T, kTeam, true>(p, stream) : launch_ring<T, kTeam, false>(p, stream);
}

template <typename T>
cudaError_t launch_typed(const NormParams& p, cudaStream_t stream) {
  if (p.dim <= 512) return launch<T, 32>(p, stream);
  if (p.dim <= 1024) return launch<T, 64>(p, stream);
  if (p.dim <= 2048) return launch<T, 128>(p, stream);
  if (p.dim <= 4096) return launch<T, 256>(p, stream);
  if (p.dim <= 8192) return launch<T, 512>(p, stream);
  rms_norm_fp8_long_kernel<T><<<static_cast<unsigned>(p.n), 512, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rms_norm_fp8(int dtype, const NormParams& p, cudaStream_t stream) {
  if (dtype == MLA_FP32) return launch_typed<float>(p, stream);
  if (dtype == MLA_FP16) return launch_typed<__half>(p, stream);
  return launch_typed<__nv_bfloat16>(p, stream);
}

}  // namespace mla
