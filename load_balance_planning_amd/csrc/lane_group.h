// Reductions, scans and sorts over aligned groups of P lanes (P a power of two
// up to 64), for kernels that give each token a group of lanes of one wave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {
namespace {

// Order key of IEEE bits u: the IEEE total order as unsigned integers.
__device__ __forceinline__ uint32_t order_key(uint32_t u) {
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// Inverse of the order key u ^ (sign ? 0xffffffff : 0x80000000) of IEEE bits u.
__device__ __forceinline__ uint32_t float_from_order_key(uint32_t k) {
  return (k & 0x80000000u) ? (k & 0x7fffffffu) : ~k;
}

__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ uint64_t shfl_xor_u64(uint64_t v, int m) {
  int lo = (int)(uint32_t)v, hi = (int)(uint32_t)(v >> 32);
  lo = __shfl_xor(lo, m);
  hi = __shfl_xor(hi, m);
  return ((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo;
}

// DPP lane moves inside a row of 16 lanes (controls: quad_perm [1,0,3,2] = 0xB1,
// quad_perm [2,3,0,1] = 0x4E, row_half_mirror = 0x141, row_mirror = 0x140).
template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
  const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, 0xf, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, 0xf, 0xf, false);
  return ((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo;
}

__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// Max over each aligned group of P lanes, result in every lane of the group.
// Within a 16-lane row the butterfly uses DPP (quad swaps, then the half-row
// and row mirrors, which pair every lane with one of the other half); wider
// groups finish with two cross-row exchanges.
template <int P>
__device__ __forceinline__ uint64_t group_max_u64(uint64_t v) {
  if (P >= 2) v = max_u64(v, dpp_u64<0xB1>(v));
  if (P >= 4) v = max_u64(v, dpp_u64<0x4E>(v));
  if (P >= 8) v = max_u64(v, dpp_u64<0x141>(v));
  if (P >= 16) v = max_u64(v, dpp_u64<0x140>(v));
  if (P >= 32) v = max_u64(v, shfl_xor_u64(v, 16));
  if (P >= 64) v = max_u64(v, shfl_xor_u64(v, 32));
  return v;
}

// Exchange with lane (l ^ J) of the same aligned group of 2J lanes, all
// inside the DPP unit for J <= 8: quad permutes for J = 1, 2; for J = 4 a
// row shift left or right by 4 (selected by bit 2 of the lane); for J = 8 a
// row rotate by 8 (inside a row of 16 lanes that is l ^ 8).  J = 16 uses the
// swizzle unit (xor mask mode), J = 32 the LDS crossbar.
template <int J>
__device__ __forceinline__ uint32_t xor_lane_u32(uint32_t v, int lig) {
  if (J == 1) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, false);
  if (J == 2) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, false);
  if (J == 4) {
    const uint32_t up = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x104, 0xf, 0xf, false);  // row_shl:4
    const uint32_t dn = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false);  // row_shr:4
    return (lig & 4) ? dn : up;
  }
  if (J == 8) return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false);
  if (J == 16) return (uint32_t)__builtin_amdgcn_ds_swizzle((int)v, (16 << 10) | 0x1F);
  return (uint32_t)__shfl_xor((int)v, J);
}

// Inclusive sum over the lanes 0..lig of each aligned group of P lanes: a DPP
// row scan (row shifts by 1, 2, 4, 8, masked at group borders), then row
// broadcasts for groups wider than a row.
template <int P>
__device__ __forceinline__ int group_incl_scan(int v, int lig) {
  int o;
  if (P >= 2) { o = __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false); v += (lig & 15) >= 1 ? o : 0; }
  if (P >= 4) { o = __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false); v += (lig & 15) >= 2 ? o : 0; }
  if (P >= 8) { o = __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false); v += (lig & 15) >= 4 ? o : 0; }
  if (P >= 16) { o = __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false); v += (lig & 15) >= 8 ? o : 0; }
  if (P >= 32) { o = __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false); v += o; }  // row_bcast:15 into rows 1, 3
  if (P >= 64) { o = __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false); v += o; }  // row_bcast:31 into rows 2, 3
  return v;
}

// Value of the last lane of each aligned group of P lanes, in every lane.
template <int P>
__device__ __forceinline__ int group_last(int v) {
  if (P == 64) return __builtin_amdgcn_readlane(v, 63);
  return __builtin_amdgcn_ds_swizzle(v, ((0x1F & ~(P - 1)) << 0) | ((P - 1) << 5));
}

template <int SIZE, int J>
__device__ __forceinline__ uint32_t bitonic_step_u32(uint32_t v, int lig) {
  const uint32_t o = xor_lane_u32<J>(v, lig);
  const bool desc = (lig & SIZE) == 0;  // in the last stage every lane sorts descending
  const bool keep_max = ((lig & J) == 0) == desc;
  return keep_max ? max(o, v) : min(o, v);
}

// Bitonic sort of one 32-bit key per lane over aligned groups of P lanes,
// descending: afterwards lane l of a group holds the group's (l+1)-th largest.
template <int P>
__device__ __forceinline__ uint32_t group_sort_desc_u32(uint32_t v, int lig) {
#define MOE_BSTEP(S, J) if (P >= (S)) v = bitonic_step_u32<((S) >= P ? P : (S)), J>(v, lig);
  MOE_BSTEP(2, 1)
  MOE_BSTEP(4, 2) MOE_BSTEP(4, 1)
  MOE_BSTEP(8, 4) MOE_BSTEP(8, 2) MOE_BSTEP(8, 1)
  MOE_BSTEP(16, 8) MOE_BSTEP(16, 4) MOE_BSTEP(16, 2) MOE_BSTEP(16, 1)
  MOE_BSTEP(32, 16) MOE_BSTEP(32, 8) MOE_BSTEP(32, 4) MOE_BSTEP(32, 2) MOE_BSTEP(32, 1)
  MOE_BSTEP(64, 32) MOE_BSTEP(64, 16) MOE_BSTEP(64, 8) MOE_BSTEP(64, 4) MOE_BSTEP(64, 2) MOE_BSTEP(64, 1)
#undef MOE_BSTEP
  return v;
}

// Sort of a bitonic sequence (the last stage of the sort above), descending.
template <int P>
__device__ __forceinline__ uint32_t group_merge_desc_u32(uint32_t v, int lig) {
  if (P >= 64) v = bitonic_step_u32<P, 32>(v, lig);
  if (P >= 32) v = bitonic_step_u32<P, 16>(v, lig);
  if (P >= 16) v = bitonic_step_u32<P, 8>(v, lig);
  if (P >= 8) v = bitonic_step_u32<P, 4>(v, lig);
  if (P >= 4) v = bitonic_step_u32<P, 2>(v, lig);
  return bitonic_step_u32<P, 1>(v, lig);
}

}  // namespace
}  // namespace moe
