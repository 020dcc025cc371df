// What the experts' products in tiles share: where rows lie in LDS, the barrier that
// waits for loads into it, and the row tiles of a plan's instances.
#pragma once

#include "instances.h"

namespace moe {
namespace {

// LDS rows are 128 bytes, eight 16-byte pieces.  A direct load writes its
// lanes' pieces one after the other, so the placement is chosen on the memory
// side: the piece of linear place L belongs to row pair L / 16, and within the
// pair's 256 bytes piece p of row R lies at place (8 (R % 2) + p) ^ s(R).  The
// 16 lanes of a read then find their pieces in 16 different places of 256
// bytes: s takes three bits in which the rows of 16 lanes differ and which do
// not change from one instruction tile to the next (one address serves all
// reads of a step, the rest are immediate offsets) -- bits 1, 2, 3 of R for
// the rows operand, and 1, 2, 4 for the channels.
template <bool CHANNELS>
__device__ __forceinline__ int piece_swizzle(int pair) {  // pair = R / 2
  return CHANNELS ? (pair & 3) | ((pair >> 1) & 4) : pair & 7;
}
template <bool CHANNELS>
__device__ __forceinline__ int piece_at(int row, int p) {
  return (row >> 1) * 256 + ((((row & 1) << 3) | p) ^ piece_swizzle<CHANNELS>(row >> 1)) * 16;
}

// Barrier after which every wave sees every wave's loads into LDS, and has its
// own reads.  A barrier alone does not wait for the loads: to the compiler they
// are loads, which a workgroup fence need not order (and where it does, it waits
// for all of them).
// NEWER of the wave's last loads may still be under way (loads end in order).
template <int NEWER = 0>
[[maybe_unused]] __device__ __forceinline__ void sync_with_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(NEWER) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The row tiles of the instances: pre[i] of them before instance i, as many as
// the rows need (a bad instance has none).  All threads of a workgroup of 256.
// Instances that lie one behind the other need at most rows / ROWS + 1 each, in
// all row_tile_ids; offsets that fall may repeat rows without end, and get none.
[[maybe_unused]] __device__ __forceinline__ int count_row_tiles(const Instances& in, int rows, int32_t* pre, int32_t* sums) {
  const int n = instance_count(in), per = (n + 255) / 256;
  const int first = threadIdx.x * per;
  Span sp;
  int64_t mine = 0;
  for (int i = first; i < min(first + per, n); ++i)
    if (instance_span(in, i, &sp)) mine += (sp.end - sp.begin + rows - 1) / rows;
  // a sum that passes the bound stays past it, and within 32 bits
  const int most = (int)row_tile_ids(in, rows);
  const int own = (int)min(mine, (int64_t)most + 1);
  int incl = own;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(incl, off);
    incl = min(incl + ((threadIdx.x & 63) >= off ? o : 0), most + 1);
  }
  if ((threadIdx.x & 63) == 63) sums[threadIdx.x >> 6] = incl;
  __syncthreads();
  const int total = sums[0] + sums[1] + sums[2] + sums[3];
  if (total > most) return 0;
  int before = incl - own;
  for (int q = 0; q < (int)(threadIdx.x >> 6); ++q) before += sums[q];
  for (int i = first; i < min(first + per, n); ++i) {
    pre[i] = before;
    if (instance_span(in, i, &sp)) before += (int)((sp.end - sp.begin + rows - 1) / rows);
  }
  if (threadIdx.x == 0) pre[n] = total;
  __syncthreads();
  return total;
}

// The instance of row tile t < pre[n]: the last with pre[i] <= t.  One wave, two rounds of 64.
[[maybe_unused]] __device__ __forceinline__ int instance_of(const int32_t* pre, int n, int t) {
  const int lane = threadIdx.x & 63, stride = (n + 63) / 64;
  const uint64_t coarse = __ballot(lane * stride < n && pre[min(lane * stride, n)] <= t);
  const int first = (__popcll(coarse) - 1) * stride;
  const uint64_t fine = __ballot(lane < stride && first + lane < n && pre[min(first + lane, n)] <= t);
  return first + __popcll(fine) - 1;
}

}  // namespace
}  // namespace moe
