// Buffer descriptors and LDS pointers for the experts' products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {
namespace {

typedef __attribute__((address_space(3))) void* lds_ptr;

// Only the device pass knows buffer descriptors; the host pass needs the
// kernels' names alone.
#ifdef __HIP_DEVICE_COMPILE__
// A buffer descriptor over `bytes` from p: loads then take a 32-bit offset per
// lane, which stays the same from step to step, and the step's in a scalar.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}
#endif

}  // namespace
}  // namespace moe
