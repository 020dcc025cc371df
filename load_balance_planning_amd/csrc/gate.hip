// Router scores, selection, weights and their gradient on gfx950.
//
//   score[e]  = softmax over the logits, or 1 / (1 + exp(-x[e]))
//   choice[e] = score[e] + bias[e]
//   groups    of consecutive experts rank by the sum of their one or two
//             largest choices; experts outside the best ones rank as -infinity
//   top-k     by choice (by logit where there is no bias), ties to the lower
//             expert;  weight[j] = scale * s_j  or  scale * s_j / (sum s + 1e-20)
//
// P lanes hold a token, V consecutive logits each, so a row is read once into
// registers.  The selection is route.hip's: tau, the k-th largest of the lane
// maxima, admits about k candidates; up to 2 P of them go to LDS and each one's
// rank among them is its output position.  (With room for P candidates alone,
// 4 % of the tokens of a 256-expert top-8 router had too many, and a decoding
// step waited 40 us for them.)
//
// Choices are compared as in 64 bits without computing them in 64 bits: the
// fp32 choice of an expert is off by at most half of `margin`, so two that
// differ by more are in the right order, and equal inputs are a tie.  Where two
// candidates, or two groups across the cut, lie closer (about one token in a
// hundred), the token's lanes evaluate only those candidates, or the group
// values, in 64 bits.  Where there are more candidates (long ties: a row of
// equal or of masked logits), the token takes rounds of a maximum, first over
// the fp32 choices, and over 64-bit ones if two picks, or the last pick and an
// expert left over, lie too close.
#include <math.h>

#include "experts.h"
#include "lane_group.h"

namespace moe {
namespace {

constexpr float kTiny = 1e-20f;  // added to the sum of the selected scores

// Tokens per workgroup: route.hip's rule (slices of at least 8 bits of a mask), or,
// where one workgroup takes ALL tokens, up to 32 and 1024 threads.
template <int P, bool ALL>
constexpr int gate_tpw() {
  return ALL ? (1024 / P < 32 ? 1024 / P : 32) : 256 / P < 8 ? 8 : 256 / P;
}

template <int P>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int off = P / 2; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  return v;
}
template <int P, typename F>
__device__ __forceinline__ F group_sum(F v) {
#pragma unroll
  for (int off = P / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

// Score of a logit; m and inv are the row's maximum and 1 / sum of exp(x - m)
// (softmax).  -infinity scores 0 in either form.  Far below zero a sigmoid is
// exp(x) to within fp32, where exp(-x) would leave it (at -89).
__device__ __forceinline__ float score32(bool softmax, float x, float m, float inv) {
  if (x == -INFINITY) return 0.0f;
  const bool far = x < -80.0f;
  const float e = expf(softmax ? x - m : far ? x : -x);
  return softmax ? e * inv : far ? e : 1.0f / (1.0f + e);
}
__device__ __forceinline__ double score64(bool softmax, float x, float m, double sum) {
  if (x == -INFINITY) return 0.0;
  return softmax ? exp((double)x - (double)m) / sum : 1.0 / (1.0 + exp(-(double)x));
}

// Whether a group of `per` experts is a power of two of lanes of V experts:
// its value then comes from registers, otherwise from a row of choices in LDS.
template <int V>
__host__ __device__ inline bool groups_of_lanes(int per) {
  const int lanes = per / V;
  return per % V == 0 && (lanes & (lanes - 1)) == 0;
}

// LDS of gate_kernel: presence masks; the bias, zeros up to P V; per token 2 P candidates
// (64-bit choice, choice, expert) and P selected experts; with groups their
// values and, unless they are whole lanes, a row of choices (8 words apart, for
// other banks).
__host__ __device__ inline int choice_stride(int E) { return E + 8; }
struct GateLds {
  size_t bias, cand, chosen, group, choice, total;
};
template <int P, int V, bool ALL>
__host__ __device__ inline GateLds gate_lds(int E, int n_group, bool prev, bool biased) {
  constexpr size_t TPW = gate_tpw<P, ALL>();
  GateLds l;
  l.bias = sizeof(uint64_t) * (size_t)E * (prev ? 2 : 1);
  l.cand = l.bias + (biased ? (size_t)P * V * sizeof(float) : 0);
  l.chosen = l.cand + TPW * 2 * P * 16;
  l.group = l.chosen + TPW * P * 4;
  l.choice = l.group + (n_group > 1 ? TPW * n_group * sizeof(double) : 0);
  const bool rows = n_group > 1 && !groups_of_lanes<V>(E / n_group);
  l.total = l.choice + (rows ? TPW * choice_stride(E) * sizeof(float) : 0);
  return l;
}

constexpr float kLog2e = 1.44269504f;
constexpr float kUlp = 5.9604645e-8f;  // 2^-24

// The two largest (a >= b) of a pair and a value: the median of three is the second.
__device__ __forceinline__ void push_top2(float* a, float* b, float v) {
  *b = __builtin_amdgcn_fmed3f(*a, *b, v);
  *a = fmaxf(*a, v);
}
// The two largest of two pairs (a >= b, oa >= ob).
__device__ __forceinline__ void merge_top2(float* a, float* b, float oa, float ob) {
  *b = fmaxf(fminf(*a, oa), fmaxf(*b, ob));
  *a = fmaxf(*a, oa);
}

// ALL: one workgroup, which writes omega and count itself; else the tiles' masks,
// from which a second launch counts.
template <int P, int V, bool ALL>
__global__ __launch_bounds__((gate_tpw<P, ALL>() * P)) void gate_kernel(
    Dims d, moex_gate_config g, bool vec, const float* __restrict__ logits, const float* __restrict__ bias,
    const int32_t* __restrict__ prev_topk, int32_t* __restrict__ topk_idx, float* __restrict__ topk_val,
    float* __restrict__ weight, uint64_t* __restrict__ tile_mask, uint64_t* __restrict__ prev_mask,
    int32_t* __restrict__ omega, int32_t* __restrict__ count, int32_t* __restrict__ status) {
  constexpr int TPW = gate_tpw<P, ALL>();
  constexpr int SLICES = 64 / TPW;
  extern __shared__ __align__(16) unsigned char smem_gate[];
  const bool want_prev = prev_topk != nullptr;
  const GateLds lay = gate_lds<P, V, ALL>(d.E, g.n_group, want_prev, bias != nullptr);
  unsigned long long* smask = reinterpret_cast<unsigned long long*>(smem_gate);
  unsigned long long* pmask = smask + d.E;
  float* bias_s = reinterpret_cast<float*>(smem_gate + lay.bias);
  const int x_tile = blockIdx.x / SLICES, h = blockIdx.x - x_tile * SLICES;
  const int s = x_tile / d.C, c = x_tile - s * d.C;
  const int64_t t0 = ALL ? 0 : (int64_t)s * d.Tr + (int64_t)c * kTile + h * TPW;
  const int nt = ALL ? d.T : max(0, min(TPW, d.Tr - c * kTile - h * TPW));
  const int tid = threadIdx.x, nthr = blockDim.x;
  bool bad = false;
  for (int e = tid; e < d.E; e += nthr) {
    smask[e] = 0ull;
    if (want_prev) pmask[e] = 0ull;
  }
  if (bias) {
    for (int e = tid; e < P * V; e += nthr) {
      const float b = e < d.E ? bias[e] : 0.0f;
      const bool wrong = b != b || b == INFINITY;
      bad |= wrong;
      bias_s[e] = wrong ? 0.0f : b;
    }
  }
  __syncthreads();

  const int lane = tid % P;
  const int grp_base = (tid & 63) - lane;
  const uint64_t grp_bits = (P == 64 ? ~0ull : ((1ull << P) - 1ull)) << grp_base;
  const int i = tid / P;
  // this token's candidates, [2 P] of each, and its selected experts
  double* cand64 = reinterpret_cast<double*>(smem_gate + lay.cand) + (size_t)i * 2 * P;
  float* cand_c = reinterpret_cast<float*>(smem_gate + lay.cand + (size_t)TPW * 2 * P * 8) + (size_t)i * 2 * P;
  int* cand_e = reinterpret_cast<int*>(smem_gate + lay.cand + (size_t)TPW * 2 * P * 12) + (size_t)i * 2 * P;
  int* chosen_e = reinterpret_cast<int*>(smem_gate + lay.chosen) + (size_t)i * P;
  const bool softmax = g.score == MOEX_SOFTMAX;
  const int k = d.k;
  if (i < nt) {
    const int64_t t = t0 + i;
    const float* __restrict__ row = logits + t * d.E;
    const int e0 = lane * V;
    const bool full = P * V == d.E;  // every slot holds an expert
    float x[V], o32[V];              // logits; what the experts are ordered by
    if (V >= 4 && vec) {
      // E a multiple of 4: a vector is inside the row as a whole
#pragma unroll
      for (int w = 0; w < V / 4; ++w) {
        const bool in = full || e0 + 4 * w < d.E;
        const float4 f = in ? *reinterpret_cast<const float4*>(row + e0 + 4 * w)
                            : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        x[4 * w + 0] = f.x;
        x[4 * w + 1] = f.y;
        x[4 * w + 2] = f.z;
        x[4 * w + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = e0 + v < d.E ? row[e0 + v] : -INFINITY;
    }
    float xmax = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      bad |= v % 2 == 0 && __builtin_isunordered(x[v], x[V > 1 ? v + 1 : v]);
      x[v] = fmaxf(x[v], -INFINITY);  // a NaN becomes -infinity
      xmax = fmaxf(xmax, x[v]);
    }
    float m = 0.0f, inv = 0.0f;
    if (softmax) {
      m = group_max<P>(xmax);
      if (m == INFINITY) {
        bad = true;
        xmax = -INFINITY;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          x[v] = x[v] == INFINITY ? -INFINITY : x[v];
          xmax = fmaxf(xmax, x[v]);
        }
        m = group_max<P>(xmax);
      }
      m = m == -INFINITY ? 0.0f : m;  // nothing but -infinity: every exponential is 0
    }
    // Choices in fp32, by the hardware's exponential and reciprocal (each good
    // to one unit).  The argument of an exponential is off by 2^-24 of itself,
    // which costs at most 2^-24 of 0.3 in a sigmoid and 0.6 in a softmax share;
    // with the other roundings, the sum of a softmax (V terms per lane, log2 P
    // levels) and the addition of the bias, a choice is off by less than
    // margin / 2 (1 + |choice|), where margin = 16 units, or 2 V + 32 of them.
    const bool scored = bias != nullptr || g.n_group > 1;  // choices are needed, not the logits' order alone
    const float margin = (softmax ? 2.0f * V + 32.0f : 16.0f) * kUlp;
    if (softmax) {
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        o32[v] = __builtin_amdgcn_exp2f((x[v] - m) * kLog2e);
        sum += o32[v];
      }
      sum = group_sum<P>(sum);
      inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    }
    if (scored) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        o32[v] = softmax ? o32[v] * inv : __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x[v] * -kLog2e));
      if (bias) {
#pragma unroll
        for (int v = 0; v < V; ++v) o32[v] += bias_s[e0 + v];
      }
    }
    // in 64 bits, where a comparison needs it
    double sum64 = 1.0;
    bool have64 = !softmax;
    auto logit = [&](int e) {
      const float xe = row[e];
      return xe != xe || (softmax && xe == INFINITY) ? -INFINITY : xe;
    };
    auto need64 = [&]() {
      if (have64) return;
      double a = 0.0;
#pragma unroll 1
      for (int e = e0; e < min(e0 + V, d.E); ++e) a += score64(true, logit(e), m, 1.0);
      sum64 = group_sum<P>(a);
      have64 = true;
    };
    auto choice64 = [&](int e) { return score64(softmax, logit(e), m, sum64) + (bias ? (double)bias_s[e] : 0.0); };
    auto same_inputs = [&](int a, int b) { return logit(a) == logit(b) && bias_s[a] == bias_s[b]; };

    uint64_t kept = ~0ull;  // groups a token may choose from
    const int per = d.E / g.n_group;
    if (g.n_group > 1) {
      // a group's value in 64 bits; before, in fp32, with what it may be off by
      double* gv64 = reinterpret_cast<double*>(smem_gate + lay.group) + (size_t)i * g.n_group;
      float2* gv = reinterpret_cast<float2*>(gv64);
      // Either term may be off by margin / 2 (1 + |term|), however small their sum
      // is (biases of opposite sign), and the addition by 2^-24 of the sum, margin
      // / 16 of it at most.  A term of -infinity makes the value exact; a sum that
      // leaves fp32 is off without bound.
      auto group_value = [&](float a, float b) {
        if (g.group_top != 2) b = 0.0f;
        const float y = a + b, size = fabsf(a) + fabsf(b);
        return make_float2(y, fminf(a, b) == -INFINITY ? 0.0f : margin * (1.25f + 0.625f * size));
      };
      // where a group's experts are not whole lanes', or are evaluated again, this
      // many lanes take a group: all of them, as far as there are groups
      int L = 1;
      while (2 * L * g.n_group <= P) L *= 2;
      const int part = lane & (L - 1);
      if (groups_of_lanes<V>(per)) {
        // the two largest of this lane's choices, then of the group's lanes
        const int lanes = per / V;
        float a = o32[0], b = -INFINITY;
#pragma unroll
        for (int v = 1; v < V; ++v) push_top2(&a, &b, o32[v]);
        for (int off = 1; off < lanes; off <<= 1) merge_top2(&a, &b, __shfl_xor(a, off), __shfl_xor(b, off));
        if ((lane & (lanes - 1)) == 0 && e0 < d.E) gv[e0 / per] = group_value(a, b);
      } else {
        float* ch = reinterpret_cast<float*>(smem_gate + lay.choice) + (size_t)i * choice_stride(d.E);
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (e0 + v < d.E) ch[e0 + v] = o32[v];
        wave_lds_sync();
        for (int q0 = 0; q0 < g.n_group; q0 += P / L) {
          const int q = q0 + lane / L;
          float a = -INFINITY, b = -INFINITY;
          if (q < g.n_group) {
#pragma unroll 4
            for (int j = part; j < per; j += L) push_top2(&a, &b, ch[q * per + j]);
          }
          for (int off = 1; off < L; off <<= 1) merge_top2(&a, &b, __shfl_xor(a, off), __shfl_xor(b, off));
          if (part == 0 && q < g.n_group) gv[q] = group_value(a, b);
        }
      }
      wave_lds_sync();
      bool unsure = false;
      uint64_t mask = 0ull;
      for (int q0 = 0; q0 < g.n_group; q0 += P) {
        const int q = q0 + lane;
        bool in = false;
        if (q < g.n_group) {
          const float2 y = gv[q];
          int ahead = 0, near = 0;
#pragma unroll 4
          for (int o = 0; o < g.n_group; ++o) {
            const float2 z = gv[o];
            const float room = y.y + z.y;
            ahead += z.x - y.x > room ? 1 : 0;
            near += y.x - z.x > room ? 0 : 1;  // itself, and what a NaN or an infinite room leaves open, among them
          }
          in = near <= g.topk_group;
          unsure |= !in && ahead < g.topk_group;
        }
        mask |= ((__ballot(in) & grp_bits) >> grp_base) << q0;
      }
      if ((__ballot(unsure) & grp_bits) != 0ull) {
        need64();
        wave_lds_sync();
        for (int q0 = 0; q0 < g.n_group; q0 += P / L) {
          const int q = q0 + lane / L;
          double a = -INFINITY, b = -INFINITY;
          if (q < g.n_group) {
#pragma unroll 1
            for (int j = part; j < per; j += L) {
              const double y = choice64(q * per + j);
              b = fmax(b, fmin(a, y));
              a = fmax(a, y);
            }
          }
          for (int off = 1; off < L; off <<= 1) {
            const double oa = __shfl_xor(a, off), ob = __shfl_xor(b, off);
            b = fmax(fmin(a, oa), fmax(b, ob));
            a = fmax(a, oa);
          }
          if (part == 0 && q < g.n_group) gv64[q] = g.group_top == 2 ? a + b : a;
        }
        wave_lds_sync();
        mask = 0ull;
        for (int q0 = 0; q0 < g.n_group; q0 += P) {
          const int q = q0 + lane;
          bool in = false;
          if (q < g.n_group) {
            int ahead = 0;
            for (int o = 0; o < g.n_group; ++o) ahead += gv64[o] > gv64[q] || (gv64[o] == gv64[q] && o < q) ? 1 : 0;
            in = ahead < g.topk_group;
          }
          mask |= ((__ballot(in) & grp_bits) >> grp_base) << q0;
        }
      }
      kept = mask;
    }

    // What the k experts are ordered by: choices, or the logits themselves
    // (-0 as +0).  Past the row's end and outside the kept groups: -infinity.
    if (!bias) {
#pragma unroll
      for (int v = 0; v < V; ++v) o32[v] = x[v] + 0.0f;
    }
    if (g.n_group > 1) {
      int q = e0 / per;
      if (per % V == 0) {
        const bool in = ((kept >> (q & 63)) & 1ull) != 0ull;  // the lane's experts are of one group
#pragma unroll
        for (int v = 0; v < V; ++v) o32[v] = in ? o32[v] : -INFINITY;
      } else {
        int left = (q + 1) * per - e0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          o32[v] = ((kept >> (q & 63)) & 1ull) != 0ull ? o32[v] : -INFINITY;
          if (--left == 0) {
            ++q;
            left = per;
          }
        }
      }
    }
    if (!full) {
#pragma unroll
      for (int v = 0; v < V; ++v) o32[v] = e0 + v < d.E ? o32[v] : -INFINITY;
    }
    uint32_t sorted;
    if (g.n_group > 1) {
      // Kept groups leave some lanes without a choice, and the k-th largest
      // maximum of the others admits too much: take each lane's two largest.
      // The larger of the i-th maximum and the i-th smallest second are the P
      // largest of them all, in bitonic order.
      float a = o32[0], b = -INFINITY;
#pragma unroll
      for (int v = 1; v < V; ++v) push_top2(&a, &b, o32[v]);
      sorted = group_sort_desc_u32<P>(order_key(__float_as_uint(a)), lane);
      const uint32_t seconds = group_sort_desc_u32<P>(order_key(__float_as_uint(b)), lane);
      sorted = group_merge_desc_u32<P>(max(sorted, (uint32_t)__shfl_xor((int)seconds, P - 1)), lane);
    } else {
      float a = o32[0];
#pragma unroll
      for (int v = 1; v < V; ++v) a = fmaxf(a, o32[v]);
      sorted = group_sort_desc_u32<P>(order_key(__float_as_uint(a)), lane);
    }
    const float kth = __uint_as_float(float_from_order_key((uint32_t)__shfl((int)sorted, grp_base + k - 1)));
    const float tau = bias ? kth - margin * (1.0f + fabsf(kth)) : kth;
    const int valid = full ? V : d.E - e0;  // slots past the row's end count for nothing
    int mine = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) mine += (int)(o32[v] >= tau) & (int)(v < valid);
    const int incl = group_incl_scan<P>(mine, lane);
    const int total = group_last<P>(incl);
    if (total <= 2 * P) {
      int w = incl - mine;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if ((int)(o32[v] >= tau) & (int)(v < valid)) {
          cand_c[w] = o32[v];
          cand_e[w] = e0 + v;
          ++w;
        }
      }
      wave_lds_sync();
      bool unsure = false;
      for (int at = lane; at < total; at += P) {  // once, but for the few tokens with more than P
        const float my_c = cand_c[at];
        // a choice this near is not told from this one (-infinity is sure)
        const float room = bias && my_c != -INFINITY ? margin * (1.0f + fabsf(my_c)) : -1.0f;
        int rank = 0, near = 0;
#pragma unroll 4
        for (int j = 0; j < total; ++j) {
          const float cj = cand_c[j];
          rank += cj > my_c || (cj == my_c && j < at) ? 1 : 0;  // candidates are in expert order
          near += fabsf(cj - my_c) <= room ? 1 : 0;             // itself among them
        }
        const int e = cand_e[at];
        if (near > 1)
          for (int j = 0; j < total; ++j)
            if (fabsf(cand_c[j] - my_c) <= room) unsure |= !same_inputs(cand_e[j], e);
        if (rank < k) chosen_e[rank] = e;
      }
      if ((__ballot(unsure) & grp_bits) != 0ull) {
        need64();
        for (int at = lane; at < total; at += P)  // -infinity stays: outside the kept groups, or its bias
          cand64[at] = cand_c[at] == -INFINITY ? -INFINITY : choice64(cand_e[at]);
        wave_lds_sync();
        for (int at = lane; at < total; at += P) {
          const double y = cand64[at];
          int rank = 0;
          for (int j = 0; j < total; ++j) rank += cand64[j] > y || (cand64[j] == y && j < at) ? 1 : 0;
          if (rank < k) chosen_e[rank] = cand_e[at];
        }
      }
    } else {
      // Rounds, each the largest left, ties to the lower expert.  Taken experts' bits: V <= 32.
      uint32_t taken = 0u;
      bool unsure = false;
      float last_c = 0.0f;
      int last_e = -1;
      for (int j = 0; j < k; ++j) {
        uint64_t best = 0ull;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const uint64_t key = ((uint64_t)order_key(__float_as_uint(o32[v])) << 32) | (uint32_t)(0x7fffffff - (e0 + v));
          best = e0 + v < d.E && ((taken >> v) & 1u) == 0u && key > best ? key : best;
        }
        const uint64_t top = group_max_u64<P>(best);
        const int e = 0x7fffffff - (int)(uint32_t)top;
        if (e >= e0 && e < e0 + V) taken |= 1u << (e - e0);
        const float ce = __uint_as_float(float_from_order_key((uint32_t)(top >> 32)));
        if (lane == 0) chosen_e[j] = e;
        if (bias) {
          if (last_e >= 0 && fabsf(ce - last_c) <= margin * (1.0f + fmaxf(fabsf(ce), fabsf(last_c))))
            unsure |= !same_inputs(e, last_e);
          last_c = ce;
          last_e = e;
        }
      }
      if (bias) {
        // Neighbouring picks are now either of the same inputs or surely in order.
        // An expert left over may belong before some of them if it is this near to
        // the last one and has other inputs.
        const float room = margin * (1.0f + fabsf(last_c));
        uint32_t close = 0u;
#pragma unroll
        for (int v = 0; v < V; ++v)
          close |= e0 + v < d.E && last_c - o32[v] <= room ? 1u << v : 0u;  // (-infinity is sure: NaN or infinity here)
        for (close &= ~taken; close != 0u; close &= close - 1u) unsure |= !same_inputs(e0 + __ffs((int)close) - 1, last_e);
      }
      if ((__ballot(unsure) & grp_bits) != 0ull) {
        need64();
        taken = 0u;
        for (int j = 0; j < k; ++j) {
          double best = -INFINITY;
          int at = d.E;  // none
#pragma unroll 1
          for (int v = 0; v < V; ++v) {
            const int e = e0 + v;
            if (e >= d.E || ((taken >> v) & 1u) != 0u) continue;
            const bool in = g.n_group == 1 || ((kept >> ((e / per) & 63)) & 1ull) != 0ull;
            const double y = in ? choice64(e) : -INFINITY;
            if (y > best || at == d.E) {
              best = y;
              at = e;
            }
          }
#pragma unroll
          for (int off = P / 2; off >= 1; off >>= 1) {
            const double ob = __shfl_xor(best, off);
            const int oa = __shfl_xor(at, off);
            if (oa < d.E && (at == d.E || ob > best || (ob == best && oa < at))) {
              best = ob;
              at = oa;
            }
          }
          if (at >= e0 && at < e0 + V) taken |= 1u << (at - e0);
          if (lane == 0) chosen_e[j] = at;
        }
      }
    }
    wave_lds_sync();
    // lane j: the j-th expert
    const bool chosen = lane < k;
    const int e = chosen ? chosen_e[lane] : 0;
    const float raw = chosen ? row[e] : 0.0f;
    float xe = fmaxf(raw, -INFINITY);
    if (softmax && xe == INFINITY) xe = -INFINITY;
    const float sc = chosen ? score32(softmax, xe, m, inv) : 0.0f;
    float factor = g.scale;
    if (g.renorm) factor = g.scale / (group_sum<P>(sc) + kTiny);
    if (chosen) {
      topk_idx[t * k + lane] = e;
      if (topk_val) topk_val[t * k + lane] = raw;
      weight[t * k + lane] = sc * factor;
      atomicOr(&smask[e], 1ull << i);
    }
  }
  if (want_prev) {
    for (int q = tid; q < nt * k; q += nthr) {
      const int ip = q / k;
      const int e = prev_topk[(t0 + ip) * k + (q - ip * k)];
      if ((unsigned)e < (unsigned)d.E) {
        const unsigned long long old = atomicOr(&pmask[e], 1ull << ip);
        if (old & (1ull << ip)) atomicOr(status, MOE_STATUS_BAD_TOPK);
      } else {
        atomicOr(status, MOE_STATUS_BAD_TOPK);
      }
    }
  }
  if (bad) atomicOr(status, MOE_STATUS_NAN_LOGIT);
  __syncthreads();
  if (ALL) {
    for (int e = tid; e < d.E; e += nthr) {
      const unsigned long long mk = smask[e];
      count[e] = __popcll(mk);
      for (int r = 0; r < d.R; ++r) omega[r * d.E + e] = __popcll((mk >> (r * d.Tr)) & ((1ull << d.Tr) - 1ull));
    }
    return;
  }
  // This workgroup's TPW-bit slice of every mask word of the tile.
  auto store = [&](uint64_t* word, unsigned long long mk) {
    if (TPW == 32) reinterpret_cast<uint32_t*>(word)[h] = (uint32_t)mk;
    else if (TPW == 16) reinterpret_cast<uint16_t*>(word)[h] = (uint16_t)mk;
    else reinterpret_cast<uint8_t*>(word)[h] = (uint8_t)mk;
  };
  for (int e = tid; e < d.E; e += nthr) {
    store(tile_mask + (int64_t)x_tile * d.E + e, smask[e]);
    if (want_prev) store(prev_mask + (int64_t)x_tile * d.E + e, pmask[e]);
  }
}

template <int P, int V, bool ALL>
hipError_t launch_gate_pv(const Dims& d, const moex_gate_config& g, bool vec, const float* logits, const float* bias,
                          const int32_t* prev_topk, int32_t* topk_idx, float* topk_val, float* weight,
                          uint64_t* tile_mask, uint64_t* prev_mask, int32_t* omega, int32_t* count, int32_t* status,
                          hipStream_t st) {
  constexpr int TPW = gate_tpw<P, ALL>();
  const size_t lds = gate_lds<P, V, ALL>(d.E, g.n_group, prev_topk != nullptr, bias != nullptr).total;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(gate_kernel<P, V, ALL>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  // all tokens: as many threads as they need, and at least a full workgroup's for the experts' loops
  const int threads = ALL ? (d.T * P > 256 ? (d.T * P + 63) / 64 * 64 : 256) : TPW * P;
  hipLaunchKernelGGL((gate_kernel<P, V, ALL>), dim3((unsigned)(ALL ? 1 : d.NT * (64 / TPW))), dim3(threads), lds, st, d,
                     g, vec, logits, bias, prev_topk, topk_idx, topk_val, weight, tile_mask, prev_mask, omega, count,
                     status);
  return hipGetLastError();
}

// ---- gradient ----------------------------------------------------------------

// P lanes (a power of two, at least k) hold a token's row, NV 16-byte vectors
// (or 4 NV single logits) each.  The k scores and their gradients sit one to a
// lane; the sums over them are butterflies, and the row is written once, the
// selected experts' terms read from a row of LDS.
template <int NV, bool VEC>
__global__ __launch_bounds__(256) void gate_grad_kernel(Dims d, moex_gate_config g, int P,
                                                        const float* __restrict__ logits,
                                                        const int32_t* __restrict__ topk_idx,
                                                        const float* __restrict__ grad_weight,
                                                        float* __restrict__ grad_logits, int32_t* __restrict__ status) {
  extern __shared__ __align__(16) float smem_grad[];
  const int lane = threadIdx.x & (P - 1), i = threadIdx.x / P;
  const int64_t t = (int64_t)blockIdx.x * (256 / P) + i;
  if (t >= d.T) return;  // whole lane groups; no barrier below
  const int row_words = (d.E + 3) / 4 * 4;
  float* ds_row = smem_grad + (size_t)i * row_words;
  const bool softmax = g.score == MOEX_SOFTMAX;
  const float* __restrict__ row = logits + t * d.E;
  auto gmax = [&](float v) {
    for (int off = P / 2; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
    return v;
  };
  auto gsum = [&](float v) {
    for (int off = P / 2; off >= 1; off >>= 1) v += __shfl_xor(v, off);
    return v;
  };
  auto expert = [&](int w, int q) { return VEC ? 4 * (lane + P * w) + q : lane + P * (4 * w + q); };
  float x[4 * NV];
  bool bad = false;
#pragma unroll
  for (int w = 0; w < NV; ++w) {
    if (VEC) {
      if (expert(w, 0) < d.E) *reinterpret_cast<float4*>(ds_row + expert(w, 0)) = make_float4(0, 0, 0, 0);
      if (softmax) {
        const float4 f = expert(w, 0) < d.E ? *reinterpret_cast<const float4*>(row + expert(w, 0))
                                            : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        x[4 * w] = f.x;
        x[4 * w + 1] = f.y;
        x[4 * w + 2] = f.z;
        x[4 * w + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int e = expert(w, q);
        if (e < d.E) ds_row[e] = 0.0f;
        if (softmax) x[4 * w + q] = e < d.E ? row[e] : -INFINITY;
      }
    }
  }
  float m = 0.0f, inv = 0.0f;
  if (softmax) {
    float top = -INFINITY;
#pragma unroll
    for (int v = 0; v < 4 * NV; ++v) {
      const bool wrong = x[v] != x[v] || x[v] == INFINITY;
      bad |= wrong;
      x[v] = wrong ? -INFINITY : x[v];
      top = fmaxf(top, x[v]);
    }
    m = gmax(top);
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < 4 * NV; ++v) {
      x[v] = x[v] == -INFINITY ? 0.0f : expf(x[v] - m);
      sum += x[v];
    }
    sum = gsum(sum);
    inv = sum > 0.0f ? 1.0f / sum : 0.0f;
  }
  // the selected experts, one to a lane
  int e = -1;
  float gw = 0.0f, s = 0.0f, one_minus = 0.0f;
  if (lane < d.k) {
    e = topk_idx[t * d.k + lane];
    gw = grad_weight[t * d.k + lane];
    if ((unsigned)e >= (unsigned)d.E) {
      atomicOr(status, MOE_STATUS_BAD_TOPK);
      e = -1;
      gw = 0.0f;
    } else {
      float xe = row[e];
      if (xe != xe || (softmax && xe == INFINITY)) {
        bad = true;
        xe = -INFINITY;
      }
      s = score32(softmax, xe, m, inv);
      one_minus = 1.0f / (1.0f + expf(xe));  // sigmoid: 1 - s without cancellation
    }
  }
  const int base = (threadIdx.x & 63) - lane;
  bool twice = false;
  for (int j = 0; j < d.k; ++j) twice |= __shfl(e, base + j) == e && j < lane;
  if (e >= 0 && twice) {
    atomicOr(status, MOE_STATUS_BAD_TOPK);
    e = -1;
  }
  float ds = g.scale * gw;
  if (g.renorm) {
    const float r = 1.0f / (gsum(s) + kTiny);
    ds = g.scale * r * (gw - gsum(gw * s) * r);
  }
  const float dot = softmax ? gsum(e >= 0 ? s * ds : 0.0f) : 0.0f;
  wave_lds_sync();
  if (e >= 0) ds_row[e] = softmax ? ds : ds * s * one_minus;
  wave_lds_sync();
  float* __restrict__ out = grad_logits + t * d.E;
#pragma unroll
  for (int w = 0; w < NV; ++w) {
    if (VEC) {
      if (expert(w, 0) < d.E) {
        float4 y = *reinterpret_cast<const float4*>(ds_row + expert(w, 0));
        if (softmax) {
          y.x = x[4 * w] * inv * (y.x - dot);
          y.y = x[4 * w + 1] * inv * (y.y - dot);
          y.z = x[4 * w + 2] * inv * (y.z - dot);
          y.w = x[4 * w + 3] * inv * (y.w - dot);
        }
        *reinterpret_cast<float4*>(out + expert(w, 0)) = y;
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int o = expert(w, q);
        if (o < d.E) out[o] = softmax ? x[4 * w + q] * inv * (ds_row[o] - dot) : ds_row[o];
      }
    }
  }
  if (bad) atomicOr(status, MOE_STATUS_NAN_LOGIT);
}

}  // namespace

// Lanes per token P: at least 2k where it can be, so that the candidates rarely
// outgrow the lanes, and at most 16 logits a lane (512 experts, top 8, 16384
// tokens: 30.5 us with 32 a lane, 25.7 with 16, 31 with 8).  Few tokens leave
// the chip idle, and a shorter row per lane is a shorter wait: 8 a lane, 4 up to
// 32 lanes (256 experts, top 8 of 4 of 8 groups: 9.9 -> 9.0 us for 64 tokens,
// 12.1 -> 11.6 for 4096, 20.7 -> 21.7 for 8192; 128 experts, 2048 tokens: 9.1 ->
// 7.9; each with the histograms' 3 us).
hipError_t launch_gate(const Dims& d, const moex_gate_config& g, const float* logits, const float* bias,
                       const int32_t* prev_topk, int32_t* topk_idx, float* topk_val, float* weight,
                       uint64_t* tile_mask, uint64_t* prev_mask, bool masks_wanted, int32_t* omega, int32_t* count,
                       bool* counted, int32_t* status, hipStream_t st) {
  *counted = false;
  if (d.NT == 0) return hipSuccess;
  const bool vec = (d.E % 4) == 0 && ((uintptr_t)logits % 16) == 0;
  int P = 8;
  while (P < 64 && (P < 2 * d.k || P * (d.T > 4096 ? 16 : P < 32 ? 4 : 8) < d.E)) P *= 2;
  int V = 1;
  while (P * V < d.E) V *= 2;
  // Few tokens and no need of masks: one workgroup, and no second launch (256
  // experts, 4 of 8 groups: 4 tokens 8.7 us -> 5.9, 16 tokens 8.7 -> 6.5, 32 tokens
  // 8.9 -> 8.2, and called from Python 9.1 -> 6.5, 9.4 -> 6.4, 9.5 -> 7.9; 64 tokens
  // would take 10.7 in one).  Groups of more than 1024 experts may need rows of
  // choices that, for 16 tokens, outgrow the CU's LDS.
  *counted = !masks_wanted && d.T <= 32 && d.T * P <= 1024 && (g.n_group == 1 || d.E <= 1024);
#define MOE_GATE_CASE(P_, V_)                                                                                         \
  if (P == (P_) && V == (V_))                                                                                         \
    return *counted ? launch_gate_pv<P_, V_, true>(d, g, vec, logits, bias, prev_topk, topk_idx, topk_val, weight,    \
                                                   tile_mask, prev_mask, omega, count, status, st)                    \
                    : launch_gate_pv<P_, V_, false>(d, g, vec, logits, bias, prev_topk, topk_idx, topk_val, weight,   \
                                                    tile_mask, prev_mask, omega, count, status, st);
#define MOE_GATE_P(P_) \
  MOE_GATE_CASE(P_, 1) MOE_GATE_CASE(P_, 2) MOE_GATE_CASE(P_, 4) MOE_GATE_CASE(P_, 8) MOE_GATE_CASE(P_, 16)
  MOE_GATE_P(8)
  MOE_GATE_P(16)
  MOE_GATE_P(32)
  MOE_GATE_P(64)
  MOE_GATE_CASE(64, 32)
#undef MOE_GATE_P
#undef MOE_GATE_CASE
  return hipErrorInvalidValue;
}

hipError_t launch_gate_grad(const Dims& d, const moex_gate_config& g, const float* logits, const int32_t* topk_idx,
                            const float* grad_weight, float* grad_logits, int32_t* status, hipStream_t st) {
  if (d.T == 0) return hipSuccess;
  const bool vec = (d.E % 4) == 0 && ((uintptr_t)logits % 16) == 0 && ((uintptr_t)grad_logits % 16) == 0;
  int P = 8;
  while (P < 64 && (P < d.k || P * 4 < d.E)) P *= 2;
  const int nv = (d.E + 4 * P - 1) / (4 * P);  // at most 8: E <= 2048
  const size_t lds = sizeof(float) * (size_t)(256 / P) * ((d.E + 3) / 4 * 4);
  const dim3 grid((unsigned)((d.T + 256 / P - 1) / (256 / P)));
#define MOE_GRAD_CASE(NV_, VEC_)                                                                                    \
  if (nv <= (NV_) && vec == (VEC_)) {                                                                               \
    hipLaunchKernelGGL((gate_grad_kernel<NV_, VEC_>), grid, dim3(256), lds, st, d, g, P, logits, topk_idx,          \
                       grad_weight, grad_logits, status);                                                           \
    return hipGetLastError();                                                                                       \
  }
  MOE_GRAD_CASE(1, true) MOE_GRAD_CASE(2, true) MOE_GRAD_CASE(4, true) MOE_GRAD_CASE(8, true)
  MOE_GRAD_CASE(1, false) MOE_GRAD_CASE(2, false) MOE_GRAD_CASE(4, false) MOE_GRAD_CASE(8, false)
#undef MOE_GRAD_CASE
  return hipErrorInvalidValue;
}

}  // namespace moe
