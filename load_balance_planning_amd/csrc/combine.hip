// Gate-weighted combine on gfx950: the return path of the dispatch.
//
// [TopoEP] section 2.1, Fig. 1: after the experts, each token's k expert
// outputs come back and are summed.  The gate weights are the softmax of the
// token's k selected logits (the maximum taken out before exp):
//   w[t][j]   = exp(v[t][j] - max) / sum_j' exp(v[t][j'] - max)
//   out[t][:] = bf16( sum over j = 0..k-1 of w[t][j] * expert_out[slot_pos[t*k+j]][:] )
// accumulated in fp32 in slot order and rounded once to bf16 (nearest even).
//
// One workgroup per token: the first wave computes the weights and reads the
// k row positions into LDS; every thread then owns 32 columns (four 16-byte
// vectors) and streams the k rows through them, eight rows' loads in flight.
// HBM traffic is k rows read and one written per token -- the mirror of the
// gather.  The expert rows are read once, with non-temporal loads (measured
// on MI355X: DeepSeek-V3-shaped layer 798 -> 777 us, Kimi-K2-shaped 757 ->
// 712 us).
//
// The same sum with given weights (moex_combine; no weights: all 1, the
// gradient of the dispatch) and its gradient:
//   grad_expert_out[slot_pos[t*k+j]][:] = bf16( w[t][j] * g[t][:] )
//   grad_weight[t][j] = sum over c of g[t][c] * expert_out[slot_pos[t*k+j]][c]
// One workgroup per token again: g's row stays in registers while the k rows
// stream through, each row read once and its gradient's row written once.
#include "experts.h"
#include "fp8_block.h"

namespace moe {
namespace {

constexpr int kCombThreads = 256;
constexpr int kRowsInFlight = 8;
// Fewer tokens than this do not fill 256 CUs with a workgroup each.  64 tokens
// of 8 rows of 7168: 11 -> 4.5 us, their gradient 8 -> 4.5 us.
constexpr int kFewTokens = 512;
// A row of H >= 8 values is read and written in ceil(H / 8) vectors of 16 bytes
// from any address of a 16-bit type; the last begins at H - 8, so where H is no
// multiple of 8 it has values of the one before again (value by value, such
// rows took two to eight times as long: 8192 tokens of 8 rows of 7167, 553 us and 218;
// 64 tokens of 8 rows of 7001, 39 and 5).
__device__ __forceinline__ int vector_at(int v, int H) { return min(8 * v, H - 8); }

// acc[0..7] += w * (8 bf16 values of v), each an fp32 FMA.
__device__ __forceinline__ void fma_row(float* acc, float w, const u32x4& v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] = fmaf(w, bf16_low(v[i]), acc[2 * i]);
    acc[2 * i + 1] = fmaf(w, bf16_high(v[i]), acc[2 * i + 1]);
  }
}

// The 8 sums, each rounded once.  Gives the bits of pack_bf16 for every fp32
// value, in integer arithmetic: with the conversion instruction the four-vector
// kernel took longer (32768 tokens of 8 rows of 7168, given weights: 776 and
// 802 us; one vector a thread, 4096 tokens of rows of 2055: 32.6 and 32.1).
__device__ __forceinline__ u32x4 rounded(const float* acc) {
  auto bits = [](float f) {
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return (u >> 16) | 0x40u;  // NaN stays a quiet NaN
    return (u + 0x7fffu + ((u >> 16) & 1u)) >> 16;
  };
  u32x4 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = bits(acc[2 * i]) | (bits(acc[2 * i + 1]) << 16);
  return y;
}

// Weights and row positions of token t into LDS (first wave).  GIVEN: topk_val
// holds the weights themselves (null: all 1); otherwise the selected logits,
// whose softmax they are.  A non-finite selected logit or a position outside
// the dispatch buffer is recorded in the status word; such a position is
// stored as -1 and its slot skipped.
template <bool GIVEN>
__device__ __forceinline__ void gate_weights(const Dims& d, int64_t t, const float* __restrict__ topk_val,
                                             const int32_t* __restrict__ slot_pos, float* w_s, int32_t* p_s,
                                             int32_t* status) {
  const int lane = threadIdx.x;
  if (lane < 64) {
    const bool on = lane < d.k;
    float w;
    if (GIVEN) {
      w = on && topk_val ? topk_val[t * d.k + lane] : 1.0f;
    } else {
      const float v = on ? topk_val[t * d.k + lane] : -INFINITY;
      if (on && !__builtin_isfinite(v)) atomicOr(status, MOE_STATUS_NAN_LOGIT);
      float m = v;
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
      const float e = on ? expf(v - m) : 0.0f;
      float s = e;
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off);
      w = e / s;
    }
    int32_t p = on ? slot_pos[t * d.k + lane] : 0;
    // Both have arrived before the branch: a load still under way on the path
    // around it had every row's load below wait for all loads before it.
    asm volatile("" : "+v"(w), "+v"(p));
    if (on) {
      w_s[lane] = w;
      const int64_t N = (int64_t)d.T * d.k;
      if (p < 0 || p >= N) {
        atomicOr(status, MOE_STATUS_PLAN_CHECK);
        p = -1;
      }
      p_s[lane] = p;
    }
  }
  __syncthreads();
}

template <int VPT, bool GIVEN>
__global__ __launch_bounds__(kCombThreads) void combine_vec_kernel(Dims d, const float* __restrict__ topk_val,
                                                                   const int32_t* __restrict__ slot_pos,
                                                                   const uint16_t* __restrict__ expert_out,
                                                                   uint16_t* __restrict__ out,
                                                                   int32_t* __restrict__ status) {
  __shared__ float w_s[kMaxK];
  __shared__ int32_t p_s[kMaxK];
  const int64_t t = blockIdx.x;
  gate_weights<GIVEN>(d, t, topk_val, slot_pos, w_s, p_s, status);
  const int vpr = (d.H + 7) / 8;
  // a row's columns in gridDim.y parts (few tokens), each of the same work
  for (int base = blockIdx.y * kCombThreads * VPT; base < vpr; base += gridDim.y * kCombThreads * VPT) {
    float acc[VPT][8];
#pragma unroll
    for (int u = 0; u < VPT; ++u)
#pragma unroll
      for (int q = 0; q < 8; ++q) acc[u][q] = 0.0f;
    // kRowsInFlight rows loaded per batch (measured on MI355X: 8 beats 2 and 4
    // by ~5 %, more rows cost occupancy); the sums still go j = 0, 1, 2, ... in order
    for (int j = 0; j < d.k; j += kRowsInFlight) {
      int pj[kRowsInFlight];
      float wj[kRowsInFlight];
#pragma unroll
      for (int q = 0; q < kRowsInFlight; ++q) {
        pj[q] = j + q < d.k ? p_s[j + q] : -1;
        wj[q] = pj[q] >= 0 ? w_s[j + q] : 0.0f;
      }
      u32x4 x[kRowsInFlight][VPT];
#pragma unroll
      for (int q = 0; q < kRowsInFlight; ++q) {
        const uint16_t* row = expert_out + (int64_t)(pj[q] >= 0 ? pj[q] : 0) * d.H;
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
          const int c = base + threadIdx.x + u * kCombThreads;
          u32x4 y = {0, 0, 0, 0};  // a skipped slot adds 0 * 0
          if (c < vpr && pj[q] >= 0)
            y = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(row + vector_at(c, d.H)));
          x[q][u] = y;
        }
      }
#pragma unroll
      for (int q = 0; q < kRowsInFlight; ++q)
        if (j + q < d.k)
#pragma unroll
          for (int u = 0; u < VPT; ++u) fma_row(acc[u], wj[q], x[q][u]);
    }
    uint16_t* dst = out + t * d.H;
#pragma unroll
    for (int u = 0; u < VPT; ++u) {
      const int c = base + threadIdx.x + u * kCombThreads;
      if (c < vpr) *reinterpret_cast<u32x4_any*>(dst + vector_at(c, d.H)) = rounded(acc[u]);
    }
  }
}

// H < 8: one bf16 element per thread.
template <bool GIVEN>
__global__ __launch_bounds__(kCombThreads) void combine_u16_kernel(Dims d, const float* __restrict__ topk_val,
                                                                   const int32_t* __restrict__ slot_pos,
                                                                   const uint16_t* __restrict__ expert_out,
                                                                   uint16_t* __restrict__ out,
                                                                   int32_t* __restrict__ status) {
  __shared__ float w_s[kMaxK];
  __shared__ int32_t p_s[kMaxK];
  const int64_t t = blockIdx.x;
  gate_weights<GIVEN>(d, t, topk_val, slot_pos, w_s, p_s, status);
  for (int c = threadIdx.x; c < d.H; c += kCombThreads) {
    float acc = 0.0f;
    for (int j = 0; j < d.k; ++j) {
      const int p = p_s[j];
      if (p >= 0) acc = fmaf(w_s[j], bf16_low(expert_out[(int64_t)p * d.H + c]), acc);
    }
    out[t * d.H + c] = (uint16_t)pack_bf16(acc, 0.0f);
  }
}

// Sum over the wave, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// dot += 8 products of bf16 values, each an fp32 FMA.
__device__ __forceinline__ void dot_row(float* dot, const u32x4& g, const u32x4& x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    *dot = fmaf(bf16_low(g[i]), bf16_low(x[i]), *dot);
    *dot = fmaf(bf16_high(g[i]), bf16_high(x[i]), *dot);
  }
}

// 8 bf16 values with zeros for the first `count` of them.
__device__ __forceinline__ u32x4 without(u32x4 x, int count) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] &= (2 * i >= count ? 0xffffu : 0u) | (2 * i + 1 >= count ? 0xffff0000u : 0u);
  return x;
}

// w times 8 bf16 values, rounded once.
__device__ __forceinline__ u32x4 scaled_row(float w, const u32x4& g) {
  u32x4 y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = pack_bf16(w * bf16_low(g[i]), w * bf16_high(g[i]));
  return y;
}

// ROWS of a token's k rows per workgroup; a token's workgroups are neighbours,
// so that they find its gradient row in the caches.
template <int VPT, int ROWS>
__global__ __launch_bounds__(kCombThreads) void combine_grad_vec_kernel(
    Dims d, const float* __restrict__ weight, const int32_t* __restrict__ slot_pos,
    const uint16_t* __restrict__ expert_out, const uint16_t* __restrict__ grad_out,
    uint16_t* __restrict__ grad_rows, float* __restrict__ grad_weight, int32_t* __restrict__ status) {
  __shared__ float w_s[kMaxK];
  __shared__ int32_t p_s[kMaxK];
  __shared__ float dot_s[kCombThreads / 64][ROWS];
  const int groups = (d.k + ROWS - 1) / ROWS;
  const int vpr = (d.H + 7) / 8;
  const int64_t blocks = (int64_t)d.T * groups;
  for (int64_t block = blockIdx.x; block < blocks; block += gridDim.x) {  // once, below 2^23 blocks
    const int64_t t = block / groups;
    const int j0 = (int)(block - t * groups) * ROWS;
    __syncthreads();  // the last round's weights and sums have been read
    gate_weights<true>(d, t, weight, slot_pos, w_s, p_s, status);
    const uint16_t* __restrict__ g_row = grad_out + t * d.H;
    float dot[ROWS];
#pragma unroll
    for (int q = 0; q < ROWS; ++q) dot[q] = 0.0f;
    for (int base = 0; base < vpr; base += kCombThreads * VPT) {
      u32x4 g[VPT];
#pragma unroll
      for (int u = 0; u < VPT; ++u) {
        const int c = base + threadIdx.x + u * kCombThreads;
        g[u] = c < vpr ? *reinterpret_cast<const u32x4_any*>(g_row + vector_at(c, d.H)) : u32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int q = 0; q < ROWS; ++q) {
        const int p = j0 + q < d.k ? p_s[j0 + q] : -1;
        if (p < 0) continue;  // the same for the whole workgroup
        const uint16_t* x_row = expert_out + (int64_t)p * d.H;
        uint16_t* y_row = grad_rows + (int64_t)p * d.H;
        const float w = w_s[j0 + q];
        u32x4 x[VPT];
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
          const int c = base + threadIdx.x + u * kCombThreads;
          const u32x4_any* at = reinterpret_cast<const u32x4_any*>(x_row + vector_at(c, d.H));
          x[u] = c < vpr ? __builtin_nontemporal_load(at) : u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int u = 0; u < VPT; ++u) {
          const int c = base + threadIdx.x + u * kCombThreads;
          if (c < vpr)
            __builtin_nontemporal_store(scaled_row(w, g[u]), reinterpret_cast<u32x4_any*>(y_row + vector_at(c, d.H)));
          const int again = 8 * c - (d.H - 8);  // values that the vector before has counted
          if (again > 0 && c < vpr)
            dot_row(&dot[q], without(g[u], again), without(x[u], again));
          else
            dot_row(&dot[q], g[u], x[u]);
        }
      }
    }
#pragma unroll
    for (int q = 0; q < ROWS; ++q) {
      const float s = wave_sum(dot[q]);
      if ((threadIdx.x & 63) == 0) dot_s[threadIdx.x >> 6][q] = s;
    }
    __syncthreads();
    if (threadIdx.x < ROWS && j0 + (int)threadIdx.x < d.k) {
      const int q = threadIdx.x;
      grad_weight[t * d.k + j0 + q] = dot_s[0][q] + dot_s[1][q] + dot_s[2][q] + dot_s[3][q];
    }
  }
}

// Many tokens with rows of at most 64 vectors and given weights: P lanes (a power
// of two) hold a token's row, a vector each, so a workgroup has 256 / P tokens
// (8192 tokens of 8 rows of 512: 17 us with a token to a workgroup and 14 so, the
// gradient 55 and 28; rows of 148: 15 and 6.5, 45 and 14; but 64 tokens of rows of
// 512: 3.5 and 3.9, 3.2 and 7.5, whose gradient is split by rows there).
constexpr int kNarrow = 64;
inline bool narrow_rows(const Dims& d) { return d.H >= 8 && d.H <= 8 * kNarrow && d.T >= kFewTokens; }
inline int narrow_lanes(int H) {
  int P = 1;
  while (8 * P < H) P *= 2;
  return P;
}
// Row of slot j of token t and its weight; -1 and 0 past the k slots and for a
// position outside the dispatch buffer, which is reported.
__device__ __forceinline__ int narrow_slot(const Dims& d, int64_t t, int j, const float* __restrict__ weight,
                                           const int32_t* __restrict__ slot_pos, float* w, int32_t* status) {
  *w = 0.0f;
  if (j >= d.k) return -1;
  const int p = slot_pos[t * d.k + j];
  if (p < 0 || p >= (int64_t)d.T * d.k) {
    atomicOr(status, MOE_STATUS_PLAN_CHECK);
    return -1;
  }
  *w = weight ? weight[t * d.k + j] : 1.0f;
  return p;
}

__global__ __launch_bounds__(kCombThreads) void combine_narrow_kernel(Dims d, int P, const float* __restrict__ weight,
                                                                      const int32_t* __restrict__ slot_pos,
                                                                      const uint16_t* __restrict__ expert_out,
                                                                      uint16_t* __restrict__ out,
                                                                      int32_t* __restrict__ status) {
  const int lane = threadIdx.x & (P - 1);
  const int64_t t = (int64_t)blockIdx.x * (kCombThreads / P) + threadIdx.x / P;
  if (t >= d.T) return;
  const bool on = 8 * lane < d.H;
  const int at = vector_at(lane, d.H);
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  for (int j = 0; j < d.k; j += kRowsInFlight) {
    int p[kRowsInFlight];
    float w[kRowsInFlight];
    u32x4 x[kRowsInFlight];
#pragma unroll
    for (int q = 0; q < kRowsInFlight; ++q) p[q] = narrow_slot(d, t, j + q, weight, slot_pos, &w[q], status);
#pragma unroll
    for (int q = 0; q < kRowsInFlight; ++q) {
      x[q] = u32x4{0, 0, 0, 0};
      if (on && p[q] >= 0)
        x[q] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(expert_out + (int64_t)p[q] * d.H + at));
    }
#pragma unroll
    for (int q = 0; q < kRowsInFlight; ++q)
      if (j + q < d.k) fma_row(acc, w[q], x[q]);
  }
  if (!on) return;
  *reinterpret_cast<u32x4_any*>(out + t * d.H + at) = rounded(acc);
}

__global__ __launch_bounds__(kCombThreads) void combine_grad_narrow_kernel(
    Dims d, int P, const float* __restrict__ weight, const int32_t* __restrict__ slot_pos,
    const uint16_t* __restrict__ expert_out, const uint16_t* __restrict__ grad_out,
    uint16_t* __restrict__ grad_rows, float* __restrict__ grad_weight, int32_t* __restrict__ status) {
  constexpr int kRows = 4;
  const int lane = threadIdx.x & (P - 1);
  const int64_t t = (int64_t)blockIdx.x * (kCombThreads / P) + threadIdx.x / P;
  if (t >= d.T) return;  // whole tokens: the sums below stay within one
  const bool on = 8 * lane < d.H;
  const int at = vector_at(lane, d.H);
  const int again = 8 * lane - (d.H - 8);  // values that the vector before has counted
  u32x4 g = {0, 0, 0, 0};
  if (on) g = *reinterpret_cast<const u32x4_any*>(grad_out + t * d.H + at);
  for (int j = 0; j < d.k; j += kRows) {
    int p[kRows];
    float w[kRows];
    u32x4 x[kRows];
#pragma unroll
    for (int q = 0; q < kRows; ++q) p[q] = narrow_slot(d, t, j + q, weight, slot_pos, &w[q], status);
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      x[q] = u32x4{0, 0, 0, 0};
      if (on && p[q] >= 0)
        x[q] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(expert_out + (int64_t)p[q] * d.H + at));
    }
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      if (on && p[q] >= 0)
        __builtin_nontemporal_store(scaled_row(w[q], g),
                                    reinterpret_cast<u32x4_any*>(grad_rows + (int64_t)p[q] * d.H + at));
      float dot = 0.0f;
      if (on && p[q] >= 0) dot_row(&dot, without(g, again), without(x[q], again));
      for (int off = P / 2; off >= 1; off >>= 1) dot += __shfl_xor(dot, off);
      if (lane == 0 && j + q < d.k) grad_weight[t * d.k + j + q] = dot;
    }
  }
}

// H < 8: one bf16 element per thread.
__global__ __launch_bounds__(kCombThreads) void combine_grad_u16_kernel(
    Dims d, const float* __restrict__ weight, const int32_t* __restrict__ slot_pos,
    const uint16_t* __restrict__ expert_out, const uint16_t* __restrict__ grad_out,
    uint16_t* __restrict__ grad_rows, float* __restrict__ grad_weight, int32_t* __restrict__ status) {
  __shared__ float w_s[kMaxK];
  __shared__ int32_t p_s[kMaxK];
  __shared__ float dot_s[kCombThreads / 64];
  const int64_t t = blockIdx.x;
  gate_weights<true>(d, t, weight, slot_pos, w_s, p_s, status);
  for (int j = 0; j < d.k; ++j) {
    const int p = p_s[j];
    float dot = 0.0f;
    if (p >= 0) {
      for (int c = threadIdx.x; c < d.H; c += kCombThreads) {
        const float g = bf16_low(grad_out[t * d.H + c]);
        dot = fmaf(g, bf16_low(expert_out[(int64_t)p * d.H + c]), dot);
        grad_rows[(int64_t)p * d.H + c] = (uint16_t)pack_bf16(w_s[j] * g, 0.0f);
      }
    }
    const float s = wave_sum(dot);
    if ((threadIdx.x & 63) == 0) dot_s[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0) grad_weight[t * d.k + j] = dot_s[0] + dot_s[1] + dot_s[2] + dot_s[3];
    __syncthreads();
  }
}

template <bool GIVEN>
hipError_t launch_sum(const Dims& d, const float* topk_val, const int32_t* slot_pos, const uint16_t* expert_out,
                      uint16_t* out, int32_t* status, hipStream_t st) {
  if (d.T == 0) return hipSuccess;
  if (GIVEN && narrow_rows(d)) {
    const int P = narrow_lanes(d.H), tokens = kCombThreads / P;
    hipLaunchKernelGGL(combine_narrow_kernel, dim3((unsigned)((d.T + tokens - 1) / tokens)), dim3(kCombThreads), 0, st,
                       d, P, topk_val, slot_pos, expert_out, out, status);
    return hipGetLastError();
  }
  if (d.H >= 8) {
    // One vector a thread and round, or four.  Four read a row in one go, which
    // pays where the rows are spread over more than some 2 GB and four fill the
    // threads (rows of 7168, eight a token: 32768 tokens 791 us against 839, 24000
    // tokens 580 against 609, 16384 tokens 385 against 378, 2048 tokens 52 against
    // 51; 131072 tokens of rows of 2056: 1310 against 983).  Tokens too few for the
    // chip give each round a workgroup of its own.
    const int vpr = (d.H + 7) / 8, rounds = (vpr + kCombThreads - 1) / kCombThreads;
    const bool few = d.T < kFewTokens;
    const bool wide = (int64_t)d.T * d.k * d.H >= (int64_t)1 << 30;
    const bool one = few || !wide || (rounds & 3) == 1 || (rounds & 3) == 2;
    if (!one)
      hipLaunchKernelGGL((combine_vec_kernel<4, GIVEN>), dim3(d.T), dim3(kCombThreads), 0, st, d, topk_val, slot_pos,
                         expert_out, out, status);
    if (one)
      hipLaunchKernelGGL((combine_vec_kernel<1, GIVEN>), dim3(d.T, few ? rounds : 1), dim3(kCombThreads), 0, st, d,
                         topk_val, slot_pos, expert_out, out, status);
  } else {
    hipLaunchKernelGGL((combine_u16_kernel<GIVEN>), dim3(d.T), dim3(kCombThreads), 0, st, d, topk_val, slot_pos, expert_out,
                       out, status);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_combine(const Dims& d, const float* topk_val, const int32_t* slot_pos, const uint16_t* expert_out,
                          uint16_t* out, int32_t* status, hipStream_t st) {
  return launch_sum<false>(d, topk_val, slot_pos, expert_out, out, status, st);
}

hipError_t launch_combine_weighted(const Dims& d, const float* weight, const int32_t* slot_pos,
                                   const uint16_t* expert_out, uint16_t* out, int32_t* status, hipStream_t st) {
  return launch_sum<true>(d, weight, slot_pos, expert_out, out, status, st);
}

namespace {

template <int VPT, int ROWS>
void launch_combine_grad_rows(const Dims& d, const float* weight, const int32_t* slot_pos, const uint16_t* expert_out,
                              const uint16_t* grad_out, uint16_t* grad_expert_out, float* grad_weight,
                              int32_t* status, hipStream_t st) {
  const int64_t blocks = (int64_t)d.T * ((d.k + ROWS - 1) / ROWS);
  const int64_t most = 1 << 23;  // a launch holds fewer than 2^32 work-items
  hipLaunchKernelGGL((combine_grad_vec_kernel<VPT, ROWS>), dim3((unsigned)(blocks < most ? blocks : most)),
                     dim3(kCombThreads), 0, st, d, weight, slot_pos, expert_out, grad_out, grad_expert_out,
                     grad_weight, status);
}

}  // namespace

hipError_t launch_combine_grad(const Dims& d, const float* weight, const int32_t* slot_pos,
                               const uint16_t* expert_out, const uint16_t* grad_out, uint16_t* grad_expert_out,
                               float* grad_weight, int32_t* status, hipStream_t st) {
  if (d.T == 0) return hipSuccess;
  if (narrow_rows(d)) {
    const int P = narrow_lanes(d.H), tokens = kCombThreads / P;
    hipLaunchKernelGGL(combine_grad_narrow_kernel, dim3((unsigned)((d.T + tokens - 1) / tokens)), dim3(kCombThreads), 0,
                       st, d, P, weight, slot_pos, expert_out, grad_out, grad_expert_out, grad_weight, status);
    return hipGetLastError();
  }
  // Four rows to a workgroup (one, two and eight measured within 3 % of it), or
  // one where tokens are few; a row in one round of the threads or four vectors each.
  const bool narrow = (d.H + 7) / 8 <= kCombThreads;
  const bool few = d.T < kFewTokens;
  auto launch = few ? (narrow ? launch_combine_grad_rows<1, 1> : launch_combine_grad_rows<4, 1>)
                    : (narrow ? launch_combine_grad_rows<1, 4> : launch_combine_grad_rows<4, 4>);
  if (d.H < 8)
    hipLaunchKernelGGL(combine_grad_u16_kernel, dim3(d.T), dim3(kCombThreads), 0, st, d, weight, slot_pos, expert_out,
                       grad_out, grad_expert_out, grad_weight, status);
  else
    launch(d, weight, slot_pos, expert_out, grad_out, grad_expert_out, grad_weight, status, st);
  return hipGetLastError();
}

}  // namespace moe
