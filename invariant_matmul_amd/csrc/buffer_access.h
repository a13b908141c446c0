// Transfers from a buffer to LDS, zeros for the lanes that ask for them.
#pragma once

#include "kernel_common.h"

namespace imm {
namespace dev {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// The 2^31 - 1 bytes from base.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, 0x7fffffff, 0x00020000);
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

// ... 4 bytes per lane (lane l to dst + 4 l).
__device__ __forceinline__ void dma4(__amdgpu_buffer_rsrc_t buf, char* dst, unsigned off) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, IMM_LDS(dst), 4, off, 0, 0, 0);
#endif
}

}  // namespace dev
}  // namespace imm
