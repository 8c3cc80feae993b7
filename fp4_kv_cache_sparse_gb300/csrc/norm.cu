// norm.cu -- residual sum, root-mean-square norm and the cast to FP8 blocks
// (include/mla.h, mla_rms_norm_fp8).
//
//   s = x + residual,  v = s / sqrt(mean(s^2) + eps) * weight,
//   per 32 values: e = least with amax 2^-e <= 448, code = e4m3(v 2^-e).
//
// One pass over the data: each input is read once and each output written
// once, with the row's sums in registers between.  Two neighbouring lanes hold
// one 32-value block, so its maximum is one shuffle and its exponent is found
// once for sixteen values; products and sums go two values to an instruction.
// Rows of up to 512 dims belong to a warp, longer ones to as many warps as
// give each thread sixteen values.
// Long rows are bound by HBM (8191 x 8192 bf16 with a residual: 83.4 us, 471
// MB, 83 % of a copy's bandwidth); short ones by instructions (200,000 x 512
// fp16: 60.4 us, 311 MB, 76 %).
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
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ void put(const float2 (&f)[4]) {
    a = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    b = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
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
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    const __half2* h = reinterpret_cast<const __half2*>(&w);
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = __half22float2(h[k]);
  }
  __device__ __forceinline__ void put(const float2 (&f)[4]) {
    __half2* h = reinterpret_cast<__half2*>(&w);
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = __float22half2_rn(f[k]);
  }
};
template <>
struct Eight<__nv_bfloat16> : Eight16<__nv_bfloat16> {
  __device__ __forceinline__ void get(float2 (&f)[4]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = make_float2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xFFFF0000u));
  }
  __device__ __forceinline__ void put(const float2 (&f)[4]) {
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&w);
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = __float22bfloat162_rn(f[k]);
  }
};

// Lanes 2 i and 2 i + 1 hold a block of four 8-value pieces, the even one its
// pieces 0 and 2, the odd one 1 and 3: each access of the two is 32 contiguous bytes.
__device__ __forceinline__ int first_of(int at, int i) { return (at >> 1) * 32 + i * 16 + (at & 1) * 8; }

__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Half a block: 16 values of s and their weights.  Lanes 2 i and 2 i + 1 hold a
// block; both are inside the row or both past it.
//
// s / rms lies within sqrt(dim), so in this order only v itself can leave the
// range of 32 bits.  (weight * s can where v does not, and so can 1 / rms with
// the block's scale in one factor, which beside zeros gives NaN; that saved a
// product a value, 57.8 us for 200,000 x 512.)
template <typename T>
__device__ __forceinline__ void store_half_block(const NormParams& p, int64_t row, int at, bool in,
                                                 const float2 (&s)[2][4], const Eight<T> (&weight)[2], float inv) {
  float2 v[2][4];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    weight[i].get(v[i]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[i][k] = __fmul2_rn(__fmul2_rn(s[i][k], make_float2(inv, inv)), v[i][k]);
      amax = max_abs(amax, v[i][k].x, v[i][k].y);
    }
  }
  amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
  if (!in) return;
  const int e = fp8_block_exponent(amax);
  const float up = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e exactly: e is -127 .. 120
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = __fmul2_rn(v[k / 2][k % 2 * 2], make_float2(up, up));
    const float2 b = __fmul2_rn(v[k / 2][k % 2 * 2 + 1], make_float2(up, up));
    c[k] = e4m3x2(a.x, a.y) | (e4m3x2(b.x, b.y) << 16);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<uint2*>(p.codes + row * p.codes_row + first_of(at, i)) = make_uint2(c[2 * i], c[2 * i + 1]);
  if ((at & 1) == 0) p.scales[row * p.scales_row + at / 2] = static_cast<uint8_t>(127 + e);
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
  constexpr int kThreads = threads_of<kTeam>(), kTeams = kThreads / kTeam;
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
  const int at = tid;  // this thread's sixteen values of a row
  const bool inside = at < p.dim / 16;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kTeams;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + team;
  const auto request = [&](int64_t r, int slot) {
    if (tid != 0 || r >= p.n || *static_cast<volatile int*>(&gave_up)) return;
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
    if constexpr (kRes)
      copy(mine + slot * stage_bytes + row_bytes, static_cast<const T*>(p.residual) + r * p.residual_row);
  };
  for (int i = 0; i < stages; ++i) request(row + i * stride, i);
  Eight<T> w[2] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (inside) w[i].load(static_cast<const T*>(p.weight) + first_of(at, i));
  const float inv_dim = 1.f / static_cast<float>(p.dim);
  int slot = 0, side = 0;
  uint32_t parity = 0;
  // Every team of a block makes the same number of rounds (the block's barrier).
  for (int64_t first = row - team; first < p.n; first += stride, row += stride, side ^= 1) {
    const bool live = row < p.n && mbar_wait(&bars[slot], parity, &gave_up, p.d_error, kNormWaitNs);
    __syncwarp();
    const T* src = reinterpret_cast<const T*>(mine + slot * stage_bytes);
    float2 s[2][4], squares = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s[i][k] = make_float2(0.f, 0.f);
      if (live && inside) {
        const int from = first_of(at, i);
        Eight<T> x;
        x.load(src + from);
        x.get(s[i]);
        if constexpr (kRes) {
          float2 f[4];
          x.load(src + p.dim + from);
          x.get(f);
#pragma unroll
          for (int k = 0; k < 4; ++k) s[i][k] = __fadd2_rn(s[i][k], f[k]);
        }
        if (p.residual_out != nullptr) {
          x.put(s[i]);
          x.store(static_cast<T*>(p.residual_out) + row * p.residual_out_row + from);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) squares = __ffma2_rn(s[i][k], s[i][k], squares);
      }
    }
    const float sum = team_sum<kTeam>(squares.x + squares.y, partial[side], team);
    // The whole team has read the row: its place takes the one `stages` rows on.
    request(row + stages * stride, slot);
    if (++slot == stages) slot = 0, parity ^= 1;
    const float inv = rsqrtf(fmaf(sum, inv_dim, p.eps));
    store_half_block(p, row, at, live && inside, s, w, inv);
  }
  // After a wait that gave up: what is still on its way gets another while to land.
  if (gave_up) {
    for (int i = 0; i < stages; ++i) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(&bars[i], i < slot ? parity ^ 1 : parity) && global_timer_ns() - t0 < kNormWaitNs / 8) {
      }
    }
  }
}

// Rows too long for two of them in shared memory (fp32 with a residual, past
// 12800 dims): a block each, loaded into registers, two blocks on an SM.
template <typename T>
__global__ void __launch_bounds__(512) rms_norm_fp8_long_kernel(const NormParams p) {
  constexpr int kTeam = 512, kPieces = 2;
  __shared__ float partial[kTeam / 32];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  const T* res = static_cast<const T*>(p.residual);
  float2 s[kPieces][2][4], squares = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int at = tid + j * kTeam;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s[j][i][k] = make_float2(0.f, 0.f);
      if (at < p.dim / 16) {
        const int from = first_of(at, i);
        Eight<T> x;
        x.load(static_cast<const T*>(p.x) + row * p.x_row + from);
        x.get(s[j][i]);
        if (res != nullptr) {
          float2 f[4];
          x.load(res + row * p.residual_row + from);
          x.get(f);
#pragma unroll
          for (int k = 0; k < 4; ++k) s[j][i][k] = __fadd2_rn(s[j][i][k], f[k]);
        }
        if (p.residual_out != nullptr) {
          x.put(s[j][i]);
          x.store(static_cast<T*>(p.residual_out) + row * p.residual_out_row + from);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) squares = __ffma2_rn(s[j][i][k], s[j][i][k], squares);
      }
    }
  }
  const float sum = team_sum<kTeam>(squares.x + squares.y, partial, 0);
  const float inv = rsqrtf(fmaf(sum, 1.f / static_cast<float>(p.dim), p.eps));
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int at = tid + j * kTeam;
    const bool in = at < p.dim / 16;
    Eight<T> w[2] = {};
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (in) w[i].load(static_cast<const T*>(p.weight) + first_of(at, i));
    store_half_block(p, row, at, in, s[j], w, inv);
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
  // No more stages than rows that a team gets.
  const int64_t rounds = (p.n + blocks * kTeams - 1) / (blocks * kTeams);
  if (stages > rounds) stages = static_cast<int>(rounds);
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
  // (200,000 x 512, one call alone between two events: 63.5 us with a warp a row, 97.0 with two.)
  if (p.dim <= 512) return launch<T, 32>(p, stream);
  if (p.dim <= 1024) return launch<T, 64>(p, stream);
  if (p.dim <= 2048) return launch<T, 128>(p, stream);
  if (p.dim <= 4096) return launch<T, 256>(p, stream);
  if (p.dim <= 8192) return launch<T, 512>(p, stream);
  // A ring that holds one row only copies nothing ahead (2048 x 16384 fp32 with a
  // residual: 104.4 us so, 88.3 by the register kernel); with two rows in it
  // 2048 x 12288 take 62.2 us against 70.4, and 4096 x 16384 fp16 49.2 against 61.7.
  if (2 * p.dim * static_cast<int>(sizeof(T)) * (p.residual != nullptr ? 2 : 1) <= kNormSmem)
    return launch<T, 1024>(p, stream);
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
