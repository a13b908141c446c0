// Vectors of eight 16-bit values and their fp32 values.
#pragma once

#include "kernel_common.h"

namespace imm {
namespace dev {

typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));

template <int IN>
__device__ __forceinline__ void widen8(const u32x4_t& v, float (&f)[8]) {
  if constexpr (IN == GEMM_F16) {
    const f16x8 h = __builtin_bit_cast(f16x8, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = (float)h[e];
  } else {
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      f[2 * d] = __uint_as_float(v[d] << 16);
      f[2 * d + 1] = __uint_as_float(v[d] & 0xffff0000u);
    }
  }
}

// ... rounded to nearest, ties to even.
template <int IN>
__device__ __forceinline__ u32x4_t narrow8(const float (&f)[8]) {
  if constexpr (IN == GEMM_F16) {
    f16x8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = (_Float16)f[e];
    return __builtin_bit_cast(u32x4_t, h);
  } else {
    bf16x8 h;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = (__bf16)f[e];
    return __builtin_bit_cast(u32x4_t, h);
  }
}

}  // namespace dev
}  // namespace imm
