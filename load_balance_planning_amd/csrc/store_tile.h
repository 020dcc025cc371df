// How a wave of the experts' products writes its part of the result.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_block.h"

namespace moe {
namespace {

typedef float acc16 __attribute__((ext_vector_type(16)));

// acc[i][j] holds, in lane (r, g) = (lane % 32, lane / 32), row 32 j + r, columns
// 32 i + 16 g + 0..15, of a piece of 32 NI columns of a bf16 matrix that begins
// at `out`; rows from rows_left and columns from cols_left on are not written.
//
// A lane's 32 bytes are far from the next lane's (another row), and written as
// they are they reach memory as quarters of its 128-byte lines: the weight
// gradient of 128 experts with hardly a row took 286 us for its 0.8 GB.  So the
// piece goes through LDS (the wave's own part of it) and out in whole rows,
// TURNS times NJ / TURNS of the 32-row parts (2048 NI bytes each).  16-byte place p of row R lies at p ^
// (R % places): eight lanes' writes, one column of eight rows, go to eight places.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
template <int TURNS, int NI, int NJ>
__device__ __forceinline__ void store_wave_tile(const acc16 (&acc)[NI][NJ], unsigned char* lds, uint16_t* out,
                                                int64_t stride, int rows_left, int cols_left, bool vec) {
  constexpr int kPlaces = 4 * NI;  // of a row
  constexpr int kParts = NJ / TURNS;
  static_assert(NJ % TURNS == 0, "whole turns");
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // keeps the addresses below out of registers until here
  const int r = lane & 31, g = lane >> 5;
#pragma unroll
  for (int turn = 0; turn < TURNS; ++turn) {
#pragma unroll
    for (int j = 0; j < kParts; ++j) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const acc16& a = acc[i][turn * kParts + j];
          u32x4 o;
#pragma unroll
          for (int q = 0; q < 4; ++q) o[q] = pack_bf16(a[8 * h + 2 * q], a[8 * h + 2 * q + 1]);
          const int p = 4 * i + 2 * g + h;
          *reinterpret_cast<u32x4*>(lds + ((32 * j + r) * kPlaces + (p ^ (r & (kPlaces - 1)))) * 16) = o;
        }
      }
    }
    wave_sync();
    constexpr int kRowsAtOnce = 64 / kPlaces;
    const int p = lane % kPlaces;
#pragma unroll
    for (int s = 0; s < 32 * kParts / kRowsAtOnce; ++s) {
      const int part_row = s * kRowsAtOnce + lane / kPlaces, row = turn * 32 * kParts + part_row;
      const u32x4 o = *reinterpret_cast<const u32x4*>(lds + (part_row * kPlaces + (p ^ (part_row & (kPlaces - 1)))) * 16);
      if (row >= rows_left || 8 * p >= cols_left) continue;
      uint16_t* dst = out + row * stride + 8 * p;
      if (vec && 8 * p + 8 <= cols_left) {
        *reinterpret_cast<u32x4*>(dst) = o;
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (8 * p + q < cols_left) dst[q] = (uint16_t)(o[q / 2] >> (16 * (q & 1)));
      }
    }
    if (turn + 1 < TURNS) wave_sync();
  }
}

}  // namespace
}  // namespace moe
