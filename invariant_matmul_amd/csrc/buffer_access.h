// Loads through buffer descriptors: bounds-checked, to registers or to LDS.
#pragma once

#include "kernel_common.h"

namespace imm {
namespace dev {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// A buffer of `bytes` (at most 2^31 - 1 count) from base: what lies past it reads as
// zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* base, int64_t bytes) {
  const int n = bytes < 0x7fffffff ? (int)bytes : 0x7fffffff;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, n, 0x00020000);
}
// 16 or 4 bytes at off; zeros past the end.  (All of the offset in the lane's
// operand: the check against the end subtracts a scalar offset from the size,
// which must not pass it.)
__device__ __forceinline__ u32x4 load_b128(__amdgpu_buffer_rsrc_t buf, unsigned off) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, off, 0, 0));
#else
  return u32x4{};
#endif
}
__device__ __forceinline__ unsigned load_b32(__amdgpu_buffer_rsrc_t buf, unsigned off) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_raw_buffer_load_b32(buf, off, 0, 0);
#else
  return 0;
#endif
}

constexpr unsigned OOB = 0x80000000u;  // an offset past every buffer: zeros

// 16 bytes per lane from the buffer's byte off + uni (uni the same for the wave)
// to LDS (lane l at dst + 16 l).  (The host pass, which knows no 16-byte
// transfers, would drop the kernel's stub.)
__device__ __forceinline__ void dma16(__amdgpu_buffer_rsrc_t buf, char* dst, unsigned off, int uni) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, IMM_LDS(dst), 16, off, uni, 0, 0);
#endif
}

}  // namespace dev
}  // namespace imm
