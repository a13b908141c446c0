// Exchanges between the lanes of a wave.
#pragma once

#include "kernel_common.h"

namespace imm {
namespace dev {

// The value of the lane D lanes apart (lane ^ D), by moves within the vector unit: a
// shuffle through LDS takes ten times as long, and a join of 64 lanes is 6 to 21 of them, each
// waiting for the last.
template <int D>
__device__ __forceinline__ unsigned lane_xor(unsigned v) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int ALL = 0xf;
  if constexpr (D == 1) return __builtin_amdgcn_mov_dpp(v, 0xb1, ALL, ALL, true);        // within four: 1 0 3 2
  else if constexpr (D == 2) return __builtin_amdgcn_mov_dpp(v, 0x4e, ALL, ALL, true);   // 2 3 0 1
  else if constexpr (D == 4)                                                             // eight mirrored, fours mirrored
    return __builtin_amdgcn_mov_dpp(__builtin_amdgcn_mov_dpp(v, 0x141, ALL, ALL, true), 0x1b, ALL, ALL, true);
  else if constexpr (D == 8) return __builtin_amdgcn_mov_dpp(v, 0x128, ALL, ALL, true);  // sixteen turned by 8
  else {
    const auto r = D == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                           : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return threadIdx.x & D ? r[0] : r[1];
  }
#else
  return v;
#endif
}
template <int D>
__device__ __forceinline__ float lane_xor(float v) { return __uint_as_float(lane_xor<D>(__float_as_uint(v))); }
template <int D>
__device__ __forceinline__ uint64_t lane_xor(uint64_t v) {
  return (uint64_t)lane_xor<D>((unsigned)(v >> 32)) << 32 | lane_xor<D>((unsigned)v);
}
// f<1>(), f<2>(), f<4>() ... up to f<32>(), or down
template <int D = 1, class F>
__device__ __forceinline__ void each_up(F&& f) {
  f(std::integral_constant<int, D>{});
  if constexpr (D < 32) each_up<2 * D>(f);
}
template <int D, class F>
__device__ __forceinline__ void each_down(F&& f) {
  f(std::integral_constant<int, D>{});
  if constexpr (D > 1) each_down<D / 2>(f);
}

}  // namespace dev
}  // namespace imm
