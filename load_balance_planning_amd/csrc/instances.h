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
// rows / ROWS + n_inst of them.  The instance of an id is found by one wave in
// two rounds of loads, 64 instances each (cap <= 64 * 64; the count arrives with
// the first, the instance's rows and expert with the second).  Every lane of
// the wave calls this and gets the same answer, in scalars (rows < 2^31);
// false: no rows under this id.
template <int ROWS>
__device__ __forceinline__ bool find_row_tile(const Instances& in, int64_t id, Span* span, int64_t* row) {
  const int lane = threadIdx.x & 63;
  const int stride = (in.cap + 63) / 64;
  const int probe = min(lane * stride, in.cap);  // offset has cap + 1 entries
  const int at_probe = in.offset[probe];
  const int n_inst = instance_count(in);
  const uint64_t coarse = __ballot(lane * stride < n_inst && (int64_t)at_probe / ROWS + lane * stride <= id);
  if (coarse == 0ull) return false;
  const int first = (__popcll(coarse) - 1) * stride;
  const int i = min(first + lane, in.cap - 1);
  const int begin = in.offset[i], end = in.offset[i + 1], expert = in.expert[i];
  const uint64_t fine = __ballot(lane < stride && first + lane < n_inst && (int64_t)begin / ROWS + first + lane <= id);
  if (fine == 0ull) return false;
  const int who = __popcll(fine) - 1;  // lane of the instance
  span->begin = __builtin_amdgcn_readlane(begin, who);
  span->end = __builtin_amdgcn_readlane(end, who);
  span->expert = __builtin_amdgcn_readlane(expert, who);
  const int64_t r = span->begin + (id - (span->begin / ROWS + first + who)) * ROWS;
  *row = __builtin_amdgcn_readfirstlane((int)r);
  return span->begin >= 0 && span->begin <= span->end && span->end <= in.rows &&
         (unsigned)span->expert < (unsigned)in.E && r >= span->begin && r < span->end;
}

// Upper bound of the tile ids.
__host__ __device__ inline int64_t row_tile_ids(const Instances& in, int rows) { return in.rows / rows + in.cap; }

}  // namespace
}  // namespace moe
