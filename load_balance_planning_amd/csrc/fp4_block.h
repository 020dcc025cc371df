// e2m1 values with one power-of-two scale per 32, as the kernels read and write them.
#pragma once

#include "fp8_block.h"

namespace moe {
namespace {

constexpr int kBlk4 = 32;     // columns under one scale
constexpr int kCols4 = 256;   // columns of a 128-byte line, whose 8 scales lie together

// The scaled matrix instruction's codes of its operands' formats.
[[maybe_unused]] constexpr int kFp8 = 0, kFp4 = 4;

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

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// A word's pair.  (By value: a bit cast of a vector's element reads element 0.)
__device__ __forceinline__ bf16x2 two_bf16(uint32_t w) { return __builtin_bit_cast(bf16x2, w); }

// Eight bf16 values, divided by the scale of byte s, to e2m1 as above; zeros under
// 255.  (The conversion takes the scale's exponent.)
__device__ __forceinline__ uint32_t pack_e2m1(uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3, uint32_t s) {
  const float by = __uint_as_float(s << 23);
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, two_bf16(x0), by, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, two_bf16(x1), by, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, two_bf16(x2), by, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, two_bf16(x3), by, 3);
  return s == 255u ? 0u : w;
}

// The scale of a byte below 255, exactly (2^-127 is a subnormal).
__device__ __forceinline__ float scale_value(uint32_t s) { return __uint_as_float(s == 0u ? 0x400000u : s << 23); }

}  // namespace
}  // namespace moe
