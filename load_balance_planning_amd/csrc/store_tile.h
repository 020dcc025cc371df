// How a wave of the experts' products writes its part of the result.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_block.h"
#include "lane_group.h"

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
// piece goes through LDS, the wave's own part of it, and out in whole rows, in
// TI x TJ turns of 32 NI / TI columns by 32 NJ / TJ rows (2048 NI NJ / (TI TJ)
// bytes).  16-byte place p of row R lies at p ^ (R % places): eight lanes'
// writes, one column of eight rows, go to eight places.
template <int TI, int TJ, int NI, int NJ>
__device__ __forceinline__ void store_wave_tile(const acc16 (&acc)[NI][NJ], unsigned char* lds, uint16_t* out,
                                                int64_t stride, int rows_left, int cols_left) {
  static_assert(NI % TI == 0 && NJ % TJ == 0, "whole turns");
  constexpr int kI = NI / TI, kJ = NJ / TJ, kPlaces = 4 * kI, kRowsAtOnce = 64 / kPlaces;
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));  // keeps the addresses below out of registers until here
  const int r = lane & 31, g = lane >> 5, p = lane % kPlaces;
#pragma unroll
  for (int turn = 0; turn < TI * TJ; ++turn) {
    const int ti = turn % TI, tj = turn / TI;
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
#pragma unroll
      for (int i = 0; i < kI; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const acc16& a = acc[ti * kI + i][tj * kJ + j];
          u32x4 o;
#pragma unroll
          for (int q = 0; q < 4; ++q) o[q] = pack_bf16(a[8 * h + 2 * q], a[8 * h + 2 * q + 1]);
          const int at = 4 * i + 2 * g + h;
          *reinterpret_cast<u32x4*>(lds + ((32 * j + r) * kPlaces + (at ^ (r & (kPlaces - 1)))) * 16) = o;
        }
      }
    }
    wave_lds_sync();
#pragma unroll
    for (int s = 0; s < 32 * kJ / kRowsAtOnce; ++s) {
      const int part_row = s * kRowsAtOnce + lane / kPlaces;
      const u32x4 o = *reinterpret_cast<const u32x4*>(lds + (part_row * kPlaces + (p ^ (part_row & (kPlaces - 1)))) * 16);
      const int row = 32 * kJ * tj + part_row, col = 32 * kI * ti + 8 * p;
      if (row >= rows_left || col >= cols_left) continue;
      uint16_t* dst = out + row * stride + col;
      if (col + 8 <= cols_left) {
        *reinterpret_cast<u32x4_any*>(dst) = o;
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (col + q < cols_left) dst[q] = (uint16_t)(o[q / 2] >> (16 * (q & 1)));
      }
    }
    if (turn + 1 < TI * TJ) wave_lds_sync();
  }
}

}  // namespace
}  // namespace moe
