// What the experts' products in tiles share: where rows lie in LDS, the barrier that
// waits for loads into it, the row tiles of a plan's instances, and which tiles a
// workgroup takes.
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

// The tiles of a workgroup: from *tile on every (gridDim.x / 8)-th below *last.
// Workgroups go to the eight XCDs in turn: each XCD takes a run of consecutive
// tiles (below 2^24 in all), four row tiles by all channel tiles at a time, so that
// the tiles that it works on at once share their operands in its L2.
[[maybe_unused]] __device__ __forceinline__ void xcd_run(int total, int* tile, int* last) {
  const int xcd = blockIdx.x & 7;
  *last = (int)((int64_t)total * (xcd + 1) / 8);
  *tile = (int)((int64_t)total * xcd / 8) + (blockIdx.x >> 3);
}

// A tile: its rows, channels, expert.
struct Tile {
  int r0, rows, c0, chans, expert, rt;
};
template <int BC, int BT>
[[maybe_unused]] __device__ __forceinline__ Tile locate_tile(const Instances& in, const int32_t* pre, int n_inst,
                                                             int row_tiles, int nct, int n, int t) {
  const int band = t / (4 * nct), in_band = t - band * 4 * nct;
  const int band_rows = min(4, row_tiles - band * 4);
  const int rt = band * 4 + in_band % band_rows;
  const int i = instance_of(pre, n_inst, rt);
  Tile o;
  o.c0 = __builtin_amdgcn_readfirstlane(in_band / band_rows * BC);
  o.chans = min(BC, n - o.c0);
  o.r0 = __builtin_amdgcn_readfirstlane(in.offset[i] + (rt - pre[i]) * BT);
  o.rows = min(BT, __builtin_amdgcn_readfirstlane(in.offset[i + 1]) - o.r0);
  o.expert = __builtin_amdgcn_readfirstlane(in.expert[i]);
  o.rt = rt;
  return o;
}

}  // namespace
}  // namespace moe
