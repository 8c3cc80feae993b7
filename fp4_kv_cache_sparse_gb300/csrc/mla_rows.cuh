// mla_rows.cuh -- what the kernels that turn 16-bit and 32-bit rows into cache
// records share: 16 consecutive values of a row as floats, the e2m1 packing and
// the value of an e4m3 byte.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

namespace mla {

// Eight floats -> eight e2m1 nibbles (x[0] in the low nibble of byte 0).
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// E4M3FN byte -> float, exactly (through f16, which holds every e4m3 value).
__device__ __forceinline__ float e4m3_to_float(uint32_t byte) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(byte)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h2 & 0xFFFFu)));
}

// 16 consecutive values from a 16-byte boundary, as they lie in memory (plain
// loads: a kernel that starts early may run beside the one that writes them).
template <typename T>
struct Row16 {
  static constexpr int kWords = static_cast<int>(16 * sizeof(T) / 16);
  uint4 w[kWords];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int k = 0; k < kWords; ++k) w[k] = reinterpret_cast<const uint4*>(p)[k];
  }
  __device__ __forceinline__ void to_float(float (&x)[16]) const {
    const uint32_t* v = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int k = 0; k < 4 * kWords; ++k) {
      if constexpr (sizeof(T) == 4) {
        x[k] = __uint_as_float(v[k]);
      } else if constexpr (std::is_same<T, __half>::value) {
        x[2 * k] = __half2float(__ushort_as_half(static_cast<unsigned short>(v[k])));
        x[2 * k + 1] = __half2float(__ushort_as_half(static_cast<unsigned short>(v[k] >> 16)));
      } else {
        x[2 * k] = __uint_as_float(v[k] << 16);
        x[2 * k + 1] = __uint_as_float(v[k] & 0xFFFF0000u);
      }
    }
  }
};

}  // namespace mla
