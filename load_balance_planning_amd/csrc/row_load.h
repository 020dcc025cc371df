// Loads of bf16 rows of any width, and the gated activation, for the quantizers.
#pragma once

#include "fp8_block.h"

namespace moe {
namespace {

// Eight bf16 values from element `at` of a tensor.
__device__ __forceinline__ u32x4 load8(const uint16_t* __restrict__ x, int64_t at) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(x + at));
}
// Those of a load that would leave the tensor's `total` elements, one by one;
// zeros outside.
__device__ __forceinline__ u32x4 load8_edge(const uint16_t* __restrict__ x, int64_t at, int64_t total) {
  uint64_t half[2] = {0ull, 0ull};
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll 1
    for (int j = 0; j < 4; ++j)
      if (at + 4 * h + j >= 0 && at + 4 * h + j < total) half[h] |= (uint64_t)x[at + 4 * h + j] << (16 * j);
  return u32x4{(uint32_t)half[0], (uint32_t)(half[0] >> 32), (uint32_t)half[1], (uint32_t)(half[1] >> 32)};
}
__device__ __forceinline__ u32x4 load8(const uint16_t* __restrict__ x, int64_t at, int64_t total) {
  return at >= 0 && at + 8 <= total ? load8(x, at) : load8_edge(x, at, total);
}
__device__ __forceinline__ void widen8(const u32x4& w, float* f) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_low(w[j]);
    f[2 * j + 1] = bf16_high(w[j]);
  }
}
__device__ __forceinline__ void load16(const uint16_t* __restrict__ x, int64_t at, float* f) {
  const u32x4 lo = load8(x, at), hi = load8(x, at + 8);
  widen8(lo, f);
  widen8(hi, f + 8);
}
// The 16 values from element `at` on, `left` of them of the row (what follows is
// the next row's): zeros behind those.
__device__ __forceinline__ void load16(const uint16_t* __restrict__ x, int64_t at, int left, int64_t total, float* f) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    u32x4 w = {0u, 0u, 0u, 0u};
    if (8 * h < left) w = load8(x, at + 8 * h, total);
    widen8(w, f + 8 * h);
  }
  if (left < 16) {
#pragma unroll
    for (int j = 0; j < 16; ++j) f[j] = j < left ? f[j] : 0.0f;
  }
}

// 0 below x = -88.7, where exp(-x) leaves fp32.  exp(x) instead would keep values
// below 2^-128 and costs 5 % (131072 rows of f = 768: 112 -> 118 us).
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }
__device__ __forceinline__ float swiglu(float g, float u) { return g * sigmoid(g) * u; }

}  // namespace
}  // namespace moe
