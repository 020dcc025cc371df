// A layer's experts for at most 64 tokens in two launches on gfx950.
//
//   up    (g, u) = W1[e] Q(hidden[t]),  a = Q(g sigmoid(g) u)   per slot (t, j)
//   down  out[t] = sum_j weight[t][j] W2[e_tj] a_tj
//
// Q rounds to e4m3 with a power-of-two scale per 32.  What bounds both launches
// is the matrices' bytes, once each, so the tokens of an expert are one operand
// of the matrix instruction (16 columns of it, mostly empty) and an expert's
// rows go straight from memory to registers.  With a scale per 32 of the summed
// axis a workgroup of 32 channels quantizes its activations by itself; the
// instruction takes such scales as they are.
//
// Which tokens an expert has is found by every workgroup from the top-k (at most
// 2048 numbers): a 64-bit mask of tokens per expert, in LDS.
#include "experts4.h"
#include "fp4_block.h"
#include "lane_group.h"
#include "row_load.h"

namespace moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kFp8 = 0, kFp4 = 4;  // the instruction's format codes
constexpr int kColsF = 16;         // tokens of a tile

__device__ __forceinline__ v4i load16b(const uint8_t* p) { return *reinterpret_cast<const v4i*>(p); }

// Experts that have tokens, ascending, and the slots t * k + j of each, tokens
// ascending.  In dynamic LDS: masks u64 [E], first int32 [cap + 1], expert and
// slot uint16 [cap], [T * k]; cap = min(E, T * k).
struct Chosen {
  uint64_t* mask;
  int32_t* first;    // slots of experts before this one; entry n: all
  uint16_t* expert;
  uint16_t* slot;
  int n;
};
__host__ __device__ inline int chosen_cap(const Dims& d) { return d.E < d.T * d.k ? d.E : d.T * d.k; }
__host__ __device__ inline size_t chosen_lds(const Dims& d) {
  return ((size_t)8 * d.E + 4 * (chosen_cap(d) + 1) + 2 * chosen_cap(d) + 2 * d.T * d.k + 15) / 16 * 16;
}

template <int THREADS>
__device__ __forceinline__ Chosen collect(const Dims& d, const int32_t* __restrict__ topk, unsigned char* lds,
                                          int32_t* status) {
  __shared__ int32_t sums[THREADS / 64];
  const int slots = d.T * d.k, cap = chosen_cap(d);
  Chosen c;
  c.mask = reinterpret_cast<uint64_t*>(lds);
  c.first = reinterpret_cast<int32_t*>(lds + 8 * d.E);
  c.expert = reinterpret_cast<uint16_t*>(c.first + cap + 1);
  c.slot = c.expert + cap;
  constexpr int kPer = 2048 / THREADS;  // slots of a thread at most, and experts
  int e[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = threadIdx.x + i * THREADS;
    e[i] = s < slots ? topk[s] : -1;
  }
  for (int i = threadIdx.x; i < d.E; i += THREADS) c.mask[i] = 0ull;
  __syncthreads();
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = threadIdx.x + i * THREADS;
    if (s >= slots) continue;
    if ((unsigned)e[i] >= (unsigned)d.E) {
      bad = true;
      continue;
    }
    const uint64_t bit = 1ull << (s / d.k);
    bad |= (atomicOr(reinterpret_cast<unsigned long long*>(c.mask + e[i]), (unsigned long long)bit) & bit) != 0ull;
  }
  if (bad && status && blockIdx.x == 0) atomicOr(status, MOE_STATUS_BAD_TOPK);
  __syncthreads();
  // experts with tokens and their slots, counted together: 16 bits each
  const int per = (d.E + THREADS - 1) / THREADS, from = threadIdx.x * per;
  int mine = 0;
  for (int i = from; i < min(from + per, d.E); ++i) {
    const int m = __popcll(c.mask[i]);
    mine += m ? 0x10000 + m : 0;
  }
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(incl, off);
    incl += (threadIdx.x & 63) >= off ? o : 0;
  }
  if ((threadIdx.x & 63) == 63) sums[threadIdx.x >> 6] = incl;
  __syncthreads();
  int before = incl - mine, all = 0;
#pragma unroll
  for (int q = 0; q < THREADS / 64; ++q) {
    before += q < (int)(threadIdx.x >> 6) ? sums[q] : 0;
    all += sums[q];
  }
  c.n = all >> 16;
  for (int i = from; i < min(from + per, d.E); ++i) {
    const uint64_t set = c.mask[i];
    if (!set) continue;
    const int m = __popcll(set);
    c.expert[before >> 16] = (uint16_t)i;
    c.first[before >> 16] = before & 0xffff;
    // the slots' places need the mask no more than the place: it holds the tokens still
    before += 0x10000 + m;
  }
  if (threadIdx.x == 0) c.first[c.n] = all & 0xffff;
  __syncthreads();
  // each slot to its expert's list: the expert's index by bisection
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = threadIdx.x + i * THREADS;
    if (s >= slots || (unsigned)e[i] >= (unsigned)d.E) continue;
    int lo = 0, hi = c.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (c.expert[mid] < e[i])
        lo = mid + 1;
      else
        hi = mid;
    }
    c.slot[c.first[lo] + __popcll(c.mask[e[i]] & ((1ull << (s / d.k)) - 1ull))] = (uint16_t)s;
  }
  __syncthreads();
  return c;
}

// 16 values of a row from column c on, packed; zeros from column `cols` on.
__device__ __forceinline__ void load16_packed(const uint16_t* __restrict__ x, int64_t row_at, int c, int cols,
                                              int64_t total, uint32_t* w) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int o = c + 8 * h;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (o + 8 <= cols) {
      v = *reinterpret_cast<const u32x4_any*>(x + row_at + o);
    } else if (o < cols) {
      v = row_at + o + 8 <= total ? (u32x4) * reinterpret_cast<const u32x4_any*>(x + row_at + o)
                                  : load8_edge(x, row_at + o, total);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] &= (o + 2 * i < cols ? 0xffffu : 0u) | (o + 2 * i + 1 < cols ? 0xffff0000u : 0u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[4 * h + i] = v[i];
  }
}

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// Four words of bf16 pairs over the scale 2^(s - 127) to eight e4m3 bytes.
__device__ __forceinline__ uint32_t pack4_e4m3(uint32_t a, uint32_t b, float scale) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  s16x2 o = {0, 0};
  o = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, __builtin_bit_cast(bf16x2, a), scale, false);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(o, __builtin_bit_cast(bf16x2, b), scale, true);
  return __builtin_bit_cast(uint32_t, o);
}

// A 128-step of 16 tokens' rows as the instruction's second operand: this lane's
// 16 values from column c + 16 g on and 16 from c + 64 + 16 g on, which are
// halves of blocks g / 2 and 2 + g / 2 of 32; and block g's scale.
__device__ __forceinline__ v8i quantize_step(const uint32_t* lo, const uint32_t* hi, int lane, int* scale) {
  uint32_t ml = 0, mh = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    ml = pk_max(ml, lo[i] & 0x7fff7fffu);
    mh = pk_max(mh, hi[i] & 0x7fff7fffu);
  }
  uint32_t top = max(ml & 0xffffu, ml >> 16) | max(mh & 0xffffu, mh >> 16) << 16;  // one of each half
  top = pk_max(top, (uint32_t)__builtin_amdgcn_ds_swizzle((int)top, (16 << 10) | 0x1F));  // with lane ^ 16
  const uint32_t sl = scale_byte(top << 16), sh = scale_byte(top & 0xffff0000u);
  const float fl = sl == 255u ? 1.0f : scale_value(sl), fh = sh == 255u ? 1.0f : scale_value(sh);
  v8i o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i] = (int)pack4_e4m3(lo[2 * i], lo[2 * i + 1], fl);
    o[4 + i] = (int)pack4_e4m3(hi[2 * i], hi[2 * i + 1], fh);
  }
  // groups 1 and 2 hold one another's scales
  const int g = lane >> 4;
  const uint32_t both = sl | sh << 8;
  const uint32_t from = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (g == 1 || g == 2 ? lane ^ 48 : lane), (int)both);
  *scale = (int)(g < 2 ? from : from >> 8);
  return o;
}

// One instruction's share (16 rows by 128 columns) of matrices in WB bits: from
// line b, half h.  `row` is the lane's row of the expert's matrix of `rows` rows.
template <int WB>
struct Matrix {
  const uint8_t* q;
  const uint8_t* s;
  int64_t row_bytes, scale_step;
};
template <int WB>
__device__ __forceinline__ Matrix<WB> matrix_row(const uint8_t* __restrict__ w, const uint8_t* __restrict__ ws,
                                                 int expert, int rows, int row, int cols, int g) {
  Matrix<WB> m;
  if (WB == 4) {
    const int nb = (cols + kCols4 - 1) / kCols4;
    m.row_bytes = (int64_t)nb * (kCols4 / 2);
    m.q = w + ((int64_t)expert * rows + row) * m.row_bytes + 16 * g;
    m.s = ws + ((int64_t)expert * nb * rows + row) * 8;
    m.scale_step = (int64_t)rows * 8;
  } else {
    const int nb = (cols + kBlk - 1) / kBlk, ns = (nb + 3) / 4 * 4;
    m.row_bytes = (int64_t)nb * kBlk;
    m.q = w + ((int64_t)expert * rows + row) * m.row_bytes + 16 * g;
    m.s = ws + ((int64_t)expert * ((rows + kBlk - 1) / kBlk) + row / kBlk) * ns;
    m.scale_step = 2;
  }
  return m;
}
// The operands of a line: both halves (8 bits: the second only if it is there).
template <int WB>
struct Line {
  v8i v[2];
  uint32_t s[2];
};
template <int WB>
__device__ __forceinline__ Line<WB> load_line(const Matrix<WB>& m, int b, bool second, int g) {
  Line<WB> l;
  if (WB == 4) {
    const u32x2 s = *reinterpret_cast<const u32x2*>(m.s + b * m.scale_step);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const v4i v = load16b(m.q + (int64_t)b * (kCols4 / 2) + 64 * h);
      l.v[h] = v8i{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
      l.s[h] = s[h] >> (8 * g);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = 2 * b + (second ? h : 0);
      const v4i lo = load16b(m.q + (int64_t)at * kBlk), hi = load16b(m.q + (int64_t)at * kBlk + 64);
      l.v[h] = v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      l.s[h] = m.s[at];
    }
  }
  return l;
}
template <int WB>
__device__ __forceinline__ v4f multiply(const Line<WB>& l, int h, const v8i& x, int sx, const v4f& acc) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(l.v[h], x, acc, WB == 4 ? kFp4 : kFp8, kFp8, 0, (int)l.s[h],
                                                          0, sx);
}

// 32 gate and 32 up channels of one expert per unit; the four waves take every
// fourth line of the long axis each and add their sums in LDS.
constexpr int kUpThreads = 256, kChan = 32;
template <int WB>
__global__ __launch_bounds__(kUpThreads) void experts_up_kernel(Dims d, const uint16_t* __restrict__ hidden,
                                                                const int32_t* __restrict__ topk,
                                                                const uint8_t* __restrict__ w,
                                                                const uint8_t* __restrict__ ws, int f,
                                                                uint8_t* __restrict__ act,
                                                                uint8_t* __restrict__ act_scale,
                                                                int32_t* __restrict__ status) {
  extern __shared__ __align__(16) unsigned char lds[];
  __shared__ float part[4][kColsF][2 * kChan + 4];
  const Chosen ch = collect<kUpThreads>(d, topk, lds, status);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int chunks = (f + kChan - 1) / kChan, units = ch.n * chunks;
  const int fp = (int)padded_cols4(f), steps = (d.H + kBlk - 1) / kBlk, lines = (steps + 1) / 2;
  const int64_t total = (int64_t)d.T * d.H;
  for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int a = unit / chunks, chunk = unit - a * chunks, c0 = chunk * kChan;
    const int expert = ch.expert[a], first = ch.first[a], count = ch.first[a + 1] - first;
    Matrix<WB> m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m[i] = matrix_row<WB>(w, ws, expert, 2 * f, (i >> 1) * f + min(c0 + 16 * (i & 1) + r, f - 1), d.H, g);
    for (int t0 = 0; t0 < count; t0 += kColsF) {
      const int slot = t0 + r < count ? ch.slot[first + t0 + r] : -1;
      const int64_t row_at = (int64_t)(max(slot, 0) / d.k) * d.H;
      v4f acc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = v4f{0, 0, 0, 0};
      for (int b = wave; b < lines; b += 4) {
        const bool second = 2 * b + 1 < steps;
        Line<WB> l[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) l[i] = load_line<WB>(m[i], b, second, g);
        uint32_t x[2][2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int p = 0; p < 2; ++p) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[h][p][i] = 0u;
            if (slot >= 0)
              load16_packed(hidden, row_at, (2 * b + h) * kBlk + 64 * p + 16 * g, d.H, total, x[h][p]);
          }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && !second) break;
          int sx;
          const v8i xv = quantize_step(x[h][0], x[h][1], lane, &sx);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = multiply<WB>(l[i], h, xv, sx, acc[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<v4f*>(&part[wave][r][16 * i + 4 * g]) = acc[i];
      __syncthreads();
      {
        const int row = threadIdx.x >> 4, c = 2 * (threadIdx.x & 15);
        float v[2];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float gate = part[0][row][c + j], up = part[0][row][kChan + c + j];
#pragma unroll
          for (int q = 1; q < 4; ++q) {
            gate += part[q][row][c + j];
            up += part[q][row][kChan + c + j];
          }
          v[j] = c0 + c + j < f ? swiglu(gate, up) : 0.0f;
          top = max(top, magnitude(v[j]));
        }
        top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xf, 0xf, false));
        top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xf, 0xf, false));
        top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x141, 0xf, 0xf, false));
        top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x140, 0xf, 0xf, false));
        if (t0 + row < count) {
          const uint32_t s = scale_byte(top);
          const float inv = inverse_scale(s);
          const int64_t at = ch.slot[first + t0 + row];
          uint8_t* dst = act + at * fp + c0 + c;
          *reinterpret_cast<uint16_t*>(dst) = (uint16_t)pack_e4m3(v[0] * inv, v[1] * inv, 0.0f, 0.0f);
          uint8_t* sc = act_scale + at * (fp / kBlk4) + chunk;
          if (c == 0) *sc = (uint8_t)s;
          if (chunk == chunks - 1)  // zeros up to the line's end
            for (int z = 1; c0 + z * kChan < fp; ++z) {
              *reinterpret_cast<uint16_t*>(dst + z * kChan) = 0;
              if (c == 0) sc[z] = 127;
            }
        }
      }
      __syncthreads();
    }
  }
}

// 16 channels of the result per workgroup, over all experts with tokens: its
// waves take pieces of experts' long axes in turn and add them, times the slots'
// weights, to sums of their own in LDS.
constexpr int kDownThreads = 512, kDownWaves = kDownThreads / 64, kOut = 16;
template <int WB>
__global__ __launch_bounds__(kDownThreads) void experts_down_kernel(Dims d, const int32_t* __restrict__ topk,
                                                                    const float* __restrict__ weight,
                                                                    const uint8_t* __restrict__ w,
                                                                    const uint8_t* __restrict__ ws, int f,
                                                                    const uint8_t* __restrict__ act,
                                                                    const uint8_t* __restrict__ act_scale,
                                                                    uint16_t* __restrict__ out) {
  extern __shared__ __align__(16) unsigned char lds[];
  const Chosen ch = collect<kDownThreads>(d, topk, lds, nullptr);
  float* sums = reinterpret_cast<float*>(lds + chosen_lds(d));  // [waves][T][kOut]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  for (int i = threadIdx.x; i < kDownWaves * d.T * kOut; i += kDownThreads) sums[i] = 0.0f;
  __syncthreads();
  float* mine = sums + wave * d.T * kOut;
  const int c0 = blockIdx.x * kOut, row = min(c0 + r, d.H - 1);
  const int fp = (int)padded_cols4(f), steps = (f + kBlk - 1) / kBlk, lines = fp / kCols4;
  // as long pieces as leave every wave one, up to four lines
  const int piece = max(1, min(4, ch.n * lines / kDownWaves)), pieces = (lines + piece - 1) / piece;
  for (int item = wave; item < ch.n * pieces; item += kDownWaves) {
    const int a = item / pieces, b0 = (item - a * pieces) * piece, b1 = min(b0 + piece, lines);
    const int expert = ch.expert[a], first = ch.first[a], count = ch.first[a + 1] - first;
    const Matrix<WB> m = matrix_row<WB>(w, ws, expert, d.H, row, f, g);
    for (int t0 = 0; t0 < count; t0 += kColsF) {
      const int slot = t0 + r < count ? ch.slot[first + t0 + r] : -1;
      const float by = slot >= 0 ? weight[slot] : 0.0f;
      const uint8_t* xq = act + (int64_t)max(slot, 0) * fp + 16 * g;
      const uint8_t* xs = act_scale + (int64_t)max(slot, 0) * (fp / kBlk4);
      v4f acc = {0, 0, 0, 0};
      for (int b = b0; b < b1; ++b) {
        const bool second = 2 * b + 1 < steps;
        const Line<WB> l = load_line<WB>(m, b, second, g);
        const u32x2 s = *reinterpret_cast<const u32x2*>(xs + 8 * b);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && !second) break;
          const v4i lo = load16b(xq + b * kCols4 + 128 * h), hi = load16b(xq + b * kCols4 + 128 * h + 64);
          acc = multiply<WB>(l, h, v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]},
                             (int)(s[h] >> (8 * g)), acc);
        }
      }
      if (slot >= 0) {
        v4f* to = reinterpret_cast<v4f*>(mine + (slot / d.k) * kOut + 4 * g);
        v4f v = *to;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += by * acc[j];
        *to = v;
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < d.T * kOut; i += kDownThreads) {
    const int t = i / kOut, c = c0 + i % kOut;
    float v = sums[i];
#pragma unroll
    for (int q = 1; q < kDownWaves; ++q) v += sums[q * d.T * kOut + i];
    if (c < d.H) out[(int64_t)t * d.H + c] = (uint16_t)pack_bf16(v, 0.0f);
  }
}

template <int WB>
hipError_t launch(const Dims& d, const uint16_t* hidden, const int32_t* topk_idx, const float* weight, int32_t f,
                  const uint8_t* w1, const uint8_t* w1s, const uint8_t* w2, const uint8_t* w2s, uint8_t* act,
                  uint8_t* act_scale, uint16_t* out, int32_t* status, hipStream_t st) {
  const int64_t units = (int64_t)chosen_cap(d) * ((f + kChan - 1) / kChan);
  const size_t lds = chosen_lds(d), sums = (size_t)kDownWaves * d.T * kOut * sizeof(float);
  hipLaunchKernelGGL((experts_up_kernel<WB>), dim3((unsigned)(units < 1024 ? units : 1024)), dim3(kUpThreads), lds, st,
                     d, hidden, topk_idx, w1, w1s, f, act, act_scale, status);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (lds + sums > 64 * 1024) {
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(experts_down_kernel<WB>),
                            hipFuncAttributeMaxDynamicSharedMemorySize, (int)(lds + sums));
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((experts_down_kernel<WB>), dim3((unsigned)((d.H + kOut - 1) / kOut)), dim3(kDownThreads),
                     lds + sums, st, d, topk_idx, weight, w2, w2s, f, act, act_scale, out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_experts(const Dims& d, const uint16_t* hidden, const int32_t* topk_idx, const float* weight,
                          int32_t w_bits, int32_t f, const uint8_t* w1, const uint8_t* w1s, const uint8_t* w2,
                          const uint8_t* w2s, uint8_t* act, uint8_t* act_scale, uint16_t* out, int32_t* status,
                          hipStream_t st) {
  if (d.T == 0) return hipSuccess;
  return w_bits == 4
             ? launch<4>(d, hidden, topk_idx, weight, f, w1, w1s, w2, w2s, act, act_scale, out, status, st)
             : launch<8>(d, hidden, topk_idx, weight, f, w1, w1s, w2, w2s, act, act_scale, out, status, st);
}

}  // namespace moe
