// bf16 and block-scaled e4m3 values, as the expert-layer kernels read and write them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// The same from any address of a 16-bit type: rows of odd widths begin anywhere,
// and the memory path takes 16 bytes from there in one instruction.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// Operands and results of the matrix instructions.
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// fp32 to bf16, to nearest even, two to a word (the hardware's conversion).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

// Scale byte of a block whose largest magnitude is amax (its NaNs count as
// largest): the smallest 2^(s - 127) with amax <= 448 * 2^(s - 127), from the
// bits -- 448 is 1.75 * 2^8, so s is amax's exponent - 8, one more where its
// mantissa exceeds 1.75.  127 for zeros, 255 for a NaN or an infinity.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits == 0u) return 127u;
  if (amax_bits >= 0x7f800000u) return 255u;
  const int s = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return s < 1 ? 1u : (uint32_t)s;
}

// 2^(127 - s): the factor that brings a block to e4m3's range, exactly.  A
// marked block is multiplied by 0 (its NaNs and infinities become NaN bytes).
__device__ __forceinline__ float inverse_scale(uint32_t s) {
  return s == 255u ? 0.0f : __uint_as_float((254u - s) << 23);
}

// Four fp32 values of at most 448 to e4m3 bytes, to nearest even.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  uint32_t w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, (int)w, true);
}

// Magnitude as ordered bits: a NaN is above every number.
__device__ __forceinline__ uint32_t magnitude(float f) { return __float_as_uint(f) & 0x7fffffffu; }

}  // namespace
}  // namespace moe
