// rope.cu -- rotary positions on strided heads (include/mla.h, mla_rope).
//
// Pair (a, b) of a head at position p turns by the phase p * step_j, a 64-bit
// fraction of a turn: the integer product wraps modulo one turn exactly, so
// the angle at position 2^31 is as good as at 1 and needs no 64-bit floating
// point (of which this GPU has little) and no cosine table in memory.  Its
// upper 32 bits, as a signed fraction in [-1/2, 1/2), go through one fp32
// sine and cosine (of pi x, so no reduction is left): the angle is off by at
// most 2^-32 of a turn, for the bits cut, and 2^-24 of itself.
//
// A thread owns one column -- a 16-byte piece of a head (two in the half
// layout, whose pairs lie rope_dim / 2 apart) -- of one token, computes that
// column's sines once and applies them to a run of heads.  Bound by HBM: 8000
// tokens x 32 heads of 128 dims out of place, fp16 (131 MB), take 24.5 us, 79 %
// of a copy's bandwidth.  Heads or ranges off 16 bytes go element by element:
// 100 dims instead of 128 take 30.8 us, twice what their bytes would.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mla_device.cuh"
#include "mla_internal.h"

namespace mla {

namespace {

constexpr int kRopeThreads = 128;  // (8000 tokens x 32 heads of 128 dims: 24.5 us, 25.9 with 256)
// Heads whose loads are in flight together (8000 tokens x 32 heads of 128 dims:
// 26.6 us with one, 24.5 with two, 23.9 with four; 256 x 128 tails 7.5, 7.8 and 8.0).
constexpr int kAtOnce = 2;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

// VE consecutive elements: one 16-byte access, or element by element.
template <typename T, int VE>
struct alignas(VE * sizeof(T) == 16 ? 16 : sizeof(T)) Piece {
  T v[VE];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VE * sizeof(T) == 16) {
      *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
    } else {
#pragma unroll
      for (int k = 0; k < VE; ++k) v[k] = p[k];
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (VE * sizeof(T) == 16) {
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(v);
    } else {
#pragma unroll
      for (int k = 0; k < VE; ++k) p[k] = v[k];
    }
  }
};

struct RopeGeometry {
  int rot_cols;    // columns of a head that turn
  uint32_t cols;   // all columns of a head (rot_cols when in place)
  uint32_t runs;   // head runs of a token
  int heads_per;   // heads of a run
  int64_t units;   // n * runs
};

template <typename T, int VE, bool kHalf>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p, const RopeGeometry g,
                                                            const __grid_constant__ mla_rope_table_t table) {
  __shared__ uint64_t step[MLA_ROPE_MAX_DIM / 2];
  const int pairs = table.rope_dim / 2;
  for (int j = threadIdx.x; j < pairs; j += kRopeThreads) step[j] = table.step[j];
  __syncthreads();
  constexpr int kPairs = kHalf ? VE : VE / 2;           // pairs of a column
  constexpr int kCopy = VE * sizeof(T) == 16 ? VE : 1;  // elements of a copied column
  constexpr int kParts = kHalf ? 2 : 1;                 // pieces of a column
  const int64_t items = g.units * g.cols;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRopeThreads;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x; it < items; it += stride) {
    int64_t token;
    int col, run;
    if (items < (int64_t(1) << 31)) {
      const uint32_t unit = static_cast<uint32_t>(it) / g.cols, t = unit / g.runs;
      col = static_cast<uint32_t>(it) - unit * g.cols;
      run = unit - t * g.runs;
      token = t;
    } else {
      const int64_t unit = it / g.cols;
      col = static_cast<int>(it - unit * g.cols);
      token = unit / g.runs;
      run = static_cast<int>(unit - token * g.runs);
    }
    const int h0 = run * g.heads_per;
    int left = min(p.heads - h0, g.heads_per);
    const T* x = static_cast<const T*>(p.x) + token * p.x_row + h0 * p.x_head;
    T* y = static_cast<T*>(p.y) + token * p.y_row + h0 * p.y_head;
    if (col >= g.rot_cols) {  // a piece that is only copied
      int e = (col - g.rot_cols) * kCopy;
      if (e >= p.offset) e += table.rope_dim;
      for (; left > 0; --left, x += p.x_head, y += p.y_head) {
        Piece<T, kCopy> v;
        v.load(x + e);
        v.store(y + e);
      }
      continue;
    }
    x += p.offset + col * VE;
    y += p.offset + col * VE;
    // The first heads are on their way while the sines are computed, the next
    // ones while these are turned.
    Piece<T, VE> next[kAtOnce][kParts];
    const auto fetch = [&](const T* from, int n) {
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (u < n) {
          next[u][0].load(from + u * p.x_head);
          if constexpr (kHalf) next[u][1].load(from + u * p.x_head + pairs);
        }
      }
    };
    fetch(x, left);
    const int64_t pos = p.positions[token];
    float cs[kPairs], sn[kPairs];
#pragma unroll
    for (int k = 0; k < kPairs; ++k) {
      const uint64_t phase = static_cast<uint64_t>(pos) * step[col * kPairs + k];
      const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
      float s, c;
      sincospif(half_turns, &s, &c);
      cs[k] = c * table.factor;
      sn[k] = (p.conjugate ? -s : s) * table.factor;
    }
    for (; left > 0; left -= kAtOnce, y += kAtOnce * p.y_head) {
      Piece<T, VE> now[kAtOnce][kParts];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
#pragma unroll
        for (int q = 0; q < kParts; ++q) now[u][q] = next[u][q];
      }
      x += kAtOnce * p.x_head;
      fetch(x, left - kAtOnce);
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (u >= left) break;
        if constexpr (kHalf) {
          Piece<T, VE> &a = now[u][0], &b = now[u][1];
#pragma unroll
          for (int k = 0; k < VE; ++k) {
            const float v = to_f32(a.v[k]), w = to_f32(b.v[k]);
            a.v[k] = from_f32<T>(fmaf(v, cs[k], -w * sn[k]));
            b.v[k] = from_f32<T>(fmaf(w, cs[k], v * sn[k]));
          }
          a.store(y + u * p.y_head);
          b.store(y + u * p.y_head + pairs);
        } else {
          Piece<T, VE>& a = now[u][0];
#pragma unroll
          for (int k = 0; k < kPairs; ++k) {
            const float v = to_f32(a.v[2 * k]), w = to_f32(a.v[2 * k + 1]);
            a.v[2 * k] = from_f32<T>(fmaf(v, cs[k], -w * sn[k]));
            a.v[2 * k + 1] = from_f32<T>(fmaf(w, cs[k], v * sn[k]));
          }
          a.store(y + u * p.y_head);
        }
      }
    }
  }
}

template <typename T, int VE, bool kHalf>
cudaError_t launch(const RopeParams& p, const mla_rope_table_t& table, cudaStream_t stream) {
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  RopeGeometry g{};
  g.rot_cols = table.rope_dim / (kHalf ? 2 * VE : VE);
  g.cols = g.rot_cols + (p.x == p.y ? 0 : (p.head_dim - table.rope_dim) / (VE * sizeof(T) == 16 ? VE : 1));
  // Long head runs spread a column's sines over more heads, short ones keep
  // every SM busy when there are few tokens.  The 64-dim tails of 128 heads in
  // runs of 8 and head by head, one call alone between two events: 1024 tokens
  // 12.4 and 18.9 us, 32 tokens 8.3 and 6.2; 256 tokens 10.2 in runs of 8, 8.2 in
  // runs of 4.
  g.heads_per = 8;
  while (g.heads_per > 1 &&
         p.n * ((p.heads + g.heads_per - 1) / g.heads_per) * g.cols < static_cast<int64_t>(sms) * 384)
    g.heads_per /= 2;
  g.runs = (p.heads + g.heads_per - 1) / g.heads_per;
  g.units = p.n * g.runs;
  int64_t blocks = (g.units * g.cols + kRopeThreads - 1) / kRopeThreads;
  const int64_t cap = static_cast<int64_t>(sms) * 64;
  if (blocks > cap) blocks = cap;
  rope_kernel<T, VE, kHalf><<<static_cast<unsigned>(blocks), kRopeThreads, 0, stream>>>(p, g, table);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_typed(const RopeParams& p, const mla_rope_table_t& table, cudaStream_t stream) {
  constexpr int VE = 16 / static_cast<int>(sizeof(T));
  const bool half = table.layout == MLA_ROPE_HALF;
  const int64_t each[] = {p.x_row, p.x_head, p.y_row, p.y_head, p.offset, p.head_dim,
                          half ? table.rope_dim / 2 : table.rope_dim};
  bool wide = ((reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.y)) & 15u) == 0;
  for (const int64_t v : each) wide = wide && v % VE == 0;
  if (half) return wide ? launch<T, VE, true>(p, table, stream) : launch<T, 1, true>(p, table, stream);
  return wide ? launch<T, VE, false>(p, table, stream) : launch<T, 2, false>(p, table, stream);
}

}  // namespace

cudaError_t launch_rope(int dtype, const RopeParams& p, const mla_rope_table_t& table, cudaStream_t stream) {
  if (dtype == MLA_FP32) return launch_typed<float>(p, table, stream);
  if (dtype == MLA_FP16) return launch_typed<__half>(p, table, stream);
  return launch_typed<__nv_bfloat16>(p, table, stream);
}

}  // namespace mla
