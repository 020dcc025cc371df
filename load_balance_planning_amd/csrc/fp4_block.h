// e2m1 values with one power-of-two scale per 32, as the kernels read and write them.
#pragma once

#include "fp8_block.h"

namespace moe {
namespace {

constexpr int kBlk4 = 32;     // columns under one scale
constexpr int kCols4 = 256;   // columns of a 128-byte line, whose 8 scales lie together

// Scale byte of a block whose largest magnitude is amax: the smallest 2^(s - 127)
// with amax <= 6 * 2^(s - 127) -- 6 is 1.5 * 2^2.  127 and 255 as scale_byte.
__device__ __forceinline__ uint32_t scale_byte4(uint32_t amax_bits) {
  if (amax_bits == 0u) return 127u;
  if (amax_bits >= 0x7f800000u) return 255u;
  const int s = (int)(amax_bits >> 23) - 2 + ((amax_bits & 0x7fffffu) > 0x400000u ? 1 : 0);
  return s < 1 ? 1u : (uint32_t)s;
}

// Eight fp32 values of at most 6 to e2m1, to nearest even, the first lowest.
__device__ __forceinline__ uint32_t pack_e2m1(const float* f) {
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, f[0], f[1], 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], 1.0f, 3);
}

// The scale of a byte below 255, exactly (2^-127 is a subnormal).
__device__ __forceinline__ float scale_value(uint32_t s) { return __uint_as_float(s == 0u ? 0x400000u : s << 23); }

}  // namespace
}  // namespace moe
