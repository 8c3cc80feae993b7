// append.cu -- new tokens into the paged cache with their rotary positions
// applied on the way (include/mla.h, mla_kv_append): what mla_rope and
// mla_kv_write do one after the other, without the rows' way through memory in
// between and with one rounding instead of two.
//
// y = latent, the pairs of dims offset .. offset + rope_dim - 1 turned by the
// phase position * step_j (a 64-bit fraction of a turn, exact; sine and cosine
// in fp32), then the record of y: FP8, per 32 values the least power of two 2^e
// with amax * 2^-e <= 448; FP4, per 16 values amax / 6 rounded to E4M3FN; every
// value rounded to nearest even.
//
// One warp per token, lane l with dims 16 l .. 16 l + 15.  The turned part goes
// through the warp's own row of shared memory, where lane j takes pair j: any
// offset and either layout are the same code, and the 32 pairs of a 64-dim
// tail take one sine and cosine a lane (in registers they would take eight, on
// four lanes).
//
// Bound by bytes where there are many rows: 100000 fp16 rows with 128 turned
// dims to FP8, 156 MB, take 32.4 us, 4.8 TB/s or 72 % of a copy (31.2 with the
// hardware's fast sine and cosine, whose error is one of the whole turn, 35.3
// with sincospif; with the former, at 30.6 then, 34.9 without the next row on its
// way and 31.2 with the steps read from the table each time and eight blocks of
// every SM in the grid instead of the four that are resident).
// 100000 bf16 rows to FP4, 131 MB, take 31.9 (64 turned dims), 60000 fp32 rows to
// FP8, 155 MB, 28.9.  8191 bf16 rows to FP4 take 5.7 us (11 MB, latency), 64 rows
// 2.6, less than the host's call.  (All with L2 written over before.)
#include <cstdint>

#include "mla_device.cuh"
#include "mla_internal.h"
#include "mla_rows.cuh"

namespace mla {

namespace {

constexpr int kWarps = 8;
constexpr double kPi = 3.14159265358979323846;

// Sine and cosine of an angle of at most pi / 4 by their Taylor series (to t^9 and t^10, what follows is below 2^-28 of
// them), each within 2^-23.6 of itself: near 0 too, where a pair that lies in two blocks shows it, as the sine's part of
// a large dim may be all there is of a small one.
__device__ __forceinline__ void sin_cos(float t, float& s, float& c) {
  const float q = t * t;
  s = fmaf(t * q, fmaf(q, fmaf(q, fmaf(q, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), t);
  c = fmaf(q, fmaf(q, fmaf(q, fmaf(q, fmaf(q, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f), -0.5f), 1.f);
}

template <typename T, bool kFp4>
__global__ void __launch_bounds__(kWarps * 32, 4)
    kv_append_kernel(const AppendParams p, const __grid_constant__ mla_rope_table_t table) {
  __shared__ float rows[kWarps][kD];
  __shared__ uint64_t step[MLA_ROPE_MAX_DIM / 2];
  const int lane = threadIdx.x & 31;
  float* row = rows[threadIdx.x >> 5];
  const int pairs = table.rope_dim / 2;  // 0: nothing turns
  const bool half = table.layout == MLA_ROPE_HALF;
  // This lane's 16 dims lie in or across the turned ones.
  const bool touched = pairs > 0 && lane * 16 < p.offset + 2 * pairs && lane * 16 + 16 > p.offset;
  constexpr int kMine = MLA_ROPE_MAX_DIM / 2 / 32;  // pairs of a lane at most
  if (static_cast<int>(threadIdx.x) < pairs) step[threadIdx.x] = table.step[threadIdx.x];
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // The next token is on its way while this one is turned and quantised.
  Row16<T> raw_next;
  int32_t slot_next, pos_next = 0;
  const auto fetch = [&](int64_t t) {
    if (t >= p.n) return;
    raw_next.load(static_cast<const T*>(p.latents) + t * p.row_stride + 16 * lane);
    slot_next = p.slots[t];
    if (pairs > 0) pos_next = p.positions[t];
  };
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps;
  int64_t t = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  fetch(t);
  for (; t < p.n; t += stride) {
    const Row16<T> raw = raw_next;
    const int32_t slot = slot_next;
    const int64_t pos = pos_next;
    fetch(t + stride);
    if (slot < 0 || slot >= p.pool_tokens) {
      if (slot != -1 && lane == 0 && p.d_error) atomicOr(p.d_error, MLA_DEVERR_BAD_INDEX);
      continue;
    }
    float x[16];
    raw.to_float(x);
    if (pairs > 0) {
      float4* mine = reinterpret_cast<float4*>(row + 16 * lane);
      if (touched) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mine[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int j = lane + 32 * i;
        if (j < pairs) {
          // Whole quarters of a turn, and what is left with all of its leading bits.
          const uint64_t phase = static_cast<uint64_t>(pos) * step[j];
          const uint32_t quarters = static_cast<uint32_t>((phase + (uint64_t(1) << 61)) >> 62);
          const int64_t rest = static_cast<int64_t>(phase - (static_cast<uint64_t>(quarters) << 62));
          float s, c;
          sin_cos(static_cast<float>(rest) * static_cast<float>(kPi / 9223372036854775808.0), s, c);  // 2^63 is half a turn
          if (quarters & 1) {
            const float sine = s;
            s = c;
            c = -sine;
          }
          if (quarters & 2) s = -s, c = -c;
          c *= table.factor;
          s *= table.factor;
          float* pa = row + p.offset + (half ? j : 2 * j);
          float* pb = half ? pa + pairs : pa + 1;
          const float a = *pa, b = *pb;
          *pa = fmaf(a, c, -b * s);
          *pb = fmaf(b, c, a * s);
        }
      }
      __syncwarp();
      if (touched) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 v = mine[k];
          x[4 * k] = v.x, x[4 * k + 1] = v.y, x[4 * k + 2] = v.z, x[4 * k + 3] = v.w;
        }
      }
    }
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(x[k]));
    if constexpr (kFp4) {
      const uint32_t sc = e4m3x2(__fdiv_rn(amax, 6.f), 0.f) & 0xFFu;
      const float s = e4m3_to_float(sc);
      uint32_t q[2] = {0u, 0u};
      if (s != 0.f) {
        // x / s by one product with the reciprocal and the remainder's, which
        // leaves a quotient that lies on the border of two codes there (s has 4
        // bits, so x - y s is exact) and others within a step of 2^-23.
        const float inv = __fdiv_rn(1.f, s);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float y[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float v = x[8 * h + k], about = v * inv;
            y[k] = fmaf(fmaf(-about, s, v), inv, about);
          }
          q[h] = e2m1x8(y);
        }
      }
      uint8_t* rec = p.pool + static_cast<int64_t>(slot) * kRecFp4;
      *reinterpret_cast<uint2*>(rec + 8 * lane) = make_uint2(q[0], q[1]);
      // Scale bytes 4m .. 4m+3 gathered by lane m (m < 8).
      uint32_t word = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) word |= __shfl_sync(0xFFFFFFFFu, sc, (4 * lane + k) & 31) << (8 * k);
      if (lane < 8) *reinterpret_cast<uint32_t*>(rec + 256 + 4 * lane) = word;
    } else {
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));  // the 32-value block of lanes 2b, 2b+1
      const int e = fp8_block_exponent(amax);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);  // 2^-e, e in [-127, 120]
      uint32_t q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        q[k] = e4m3x2(x[4 * k] * down, x[4 * k + 1] * down) | (e4m3x2(x[4 * k + 2] * down, x[4 * k + 3] * down) << 16);
      uint8_t* rec = p.pool + static_cast<int64_t>(slot) * kRecFp8;
      *reinterpret_cast<uint4*>(rec + 16 * lane) = make_uint4(q[0], q[1], q[2], q[3]);
      // Scale bytes of blocks 4m .. 4m+3 gathered by lane m (m < 4).
      const uint32_t sb = static_cast<uint32_t>(127 + e);
      uint32_t word = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) word |= __shfl_sync(0xFFFFFFFFu, sb, (8 * lane + 2 * k) & 31) << (8 * k);
      if (lane < 4) *reinterpret_cast<uint32_t*>(rec + kD + 4 * lane) = word;
    }
  }
}

template <typename T>
cudaError_t launch_typed(int kv_format, const AppendParams& p, const mla_rope_table_t& table, cudaStream_t stream) {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int64_t blocks = (p.n + kWarps - 1) / kWarps;
  const int64_t cap = static_cast<int64_t>(sms) * 4;  // as many as are resident
  if (blocks > cap) blocks = cap;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = stream;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kWarps * 32);
  return kv_format == MLA_KV_FP4_288 ? cudaLaunchKernelEx(&cfg, kv_append_kernel<T, true>, p, table)
                                     : cudaLaunchKernelEx(&cfg, kv_append_kernel<T, false>, p, table);
}

}  // namespace

cudaError_t launch_kv_append(int kv_format, int dtype, const AppendParams& p, const mla_rope_table_t& table,
                             cudaStream_t stream) {
  if (dtype == MLA_FP32) return launch_typed<float>(kv_format, p, table, stream);
  if (dtype == MLA_FP16) return launch_typed<__half>(kv_format, p, table, stream);
  return launch_typed<__nv_bfloat16>(kv_format, p, table, stream);
}

}  // namespace mla
