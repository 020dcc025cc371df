// Which rows a plan's instances hold, as the experts' products read them.
#pragma once

#include "experts.h"

namespace moe {
namespace {

// Rows [begin, end) of instance i and its expert; an instance that breaks the
// contract (moex_matmul) has none.
struct Span {
  int64_t begin, end;
  int expert;
};

__device__ __forceinline__ int instance_count(const Instances& in) {
  const int n = *in.n_inst;
  return n < 0 || n > in.cap ? 0 : n;
}

__device__ __forceinline__ bool instance_span(const Instances& in, int i, Span* s) {
  const int64_t a = in.offset[i], b = in.offset[i + 1];
  const int e = in.expert[i];
  s->begin = a;
  s->end = b;
  s->expert = e;
  return a >= 0 && a <= b && b <= in.rows && (unsigned)e < (unsigned)in.E;
}

// Reports a bad count or instance in the status word; one workgroup calls it.
__device__ __forceinline__ void check_instances(const Instances& in, int32_t* status) {
  const int n = *in.n_inst;
  bool bad = n < 0 || n > in.cap;
  if (!bad) {
    Span s;
    for (int i = threadIdx.x; i < n; i += blockDim.x) bad |= !instance_span(in, i, &s);
  }
  if (bad) atomicOr(status, MOE_STATUS_PLAN_CHECK);
}

// Row tiles of ROWS rows.  Instance i owns the tile ids from offset[i] / ROWS + i
// on: offset[i+1] / ROWS - offset[i] / ROWS + 1 ids, at least as many as its
// rows need, so ids rise with i, need no prefix sum, and there are at most
// rows / ROWS + n_inst of them.  The instance of an id is found by one wave
// in two loads of 64 offsets each (cap <= 3072).  Every lane of the wave calls
// this and gets the same answer; false: no rows under this id.
template <int ROWS>
__device__ __forceinline__ bool find_row_tile(const Instances& in, int n_inst, int64_t id, Span* span, int64_t* row) {
  const int lane = threadIdx.x & 63;
  const int stride = (n_inst + 63) / 64;
  auto at_or_before = [&](int i) { return i < n_inst && (int64_t)in.offset[i] / ROWS + i <= id; };
  const uint64_t coarse = __ballot(at_or_before(lane * stride));
  if (coarse == 0ull) return false;
  const int first = (__popcll(coarse) - 1) * stride;
  const uint64_t fine = __ballot(lane < stride && at_or_before(first + lane));
  if (fine == 0ull) return false;
  const int i = first + __popcll(fine) - 1;
  if (i >= n_inst || !instance_span(in, i, span)) return false;
  *row = span->begin + (id - (span->begin / ROWS + i)) * ROWS;
  return *row >= span->begin && *row < span->end;
}

// The same tile in scalar registers (rows < 2^31): every lane holds the same
// values, which the compiler cannot see.
__device__ __forceinline__ void keep_in_scalars(Span* s, int64_t* row) {
  s->begin = __builtin_amdgcn_readfirstlane((int)s->begin);
  s->end = __builtin_amdgcn_readfirstlane((int)s->end);
  s->expert = __builtin_amdgcn_readfirstlane(s->expert);
  *row = __builtin_amdgcn_readfirstlane((int)*row);
}

// Upper bound of the tile ids.
inline int64_t row_tile_ids(const Instances& in, int rows) { return in.rows / rows + in.cap; }

}  // namespace
}  // namespace moe
