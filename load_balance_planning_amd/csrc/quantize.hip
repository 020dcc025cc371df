// Block quantization to e4m3 on gfx950: rows (one scale per 1 x 128), expert
// matrices (one per 128 x 128, both layouts), and the gated activation and its
// gradient fused with the row form.
//
//   s = smallest power of two with max|x| <= 448 s,  q = e4m3(x / s)
//
// The scale is a power of two because the matrix unit multiplies by one for
// free (E8M0), x / s and q * s are then exact, and e4m3 being a floating type,
// a scale between two powers of two would not make the values more exact.
//
// All of these move bytes once: 2 read and 1 written per value (activation: 4
// and 1, gradient: 6 and 2).  Eight lanes hold a 1 x 128 block, 16 values (32
// bytes in, 16 out) each, and find its largest magnitude with three DPP steps;
// a matrix block is held by a workgroup, 8 x 8 values to a thread, which
// transposes its bytes in registers and the block's in LDS.
#include "experts.h"
#include "fp8_block.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kLanesPerBlock = 8;
constexpr int kPerLane = kBlk / kLanesPerBlock;  // 16
constexpr int64_t kMaxGrid = 1 << 20;

enum Kind { kPlain, kSwiglu, kSwigluGrad };

// Largest of the eight lanes of an aligned group, in all of them: quad swaps,
// then the mirror of half a row, which pairs a lane with one of the other quad.
__device__ __forceinline__ uint32_t max_of_8(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, false));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, false));
}

// Eight bf16 values from element `at` of a tensor.
__device__ __forceinline__ u32x4 load8(const uint16_t* __restrict__ x, int64_t at) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(x + at));
}
// Those of a load that would leave the tensor's `total` elements, one by one;
// zeros outside.
__device__ __forceinline__ u32x4 load8_edge(const uint16_t* __restrict__ x, int64_t at, int64_t total) {
  uint64_t half[2] = {0ull, 0ull};
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll 1
    for (int j = 0; j < 4; ++j)
      if (at + 4 * h + j >= 0 && at + 4 * h + j < total) half[h] |= (uint64_t)x[at + 4 * h + j] << (16 * j);
  return u32x4{(uint32_t)half[0], (uint32_t)(half[0] >> 32), (uint32_t)half[1], (uint32_t)(half[1] >> 32)};
}
__device__ __forceinline__ u32x4 load8(const uint16_t* __restrict__ x, int64_t at, int64_t total) {
  return at >= 0 && at + 8 <= total ? load8(x, at) : load8_edge(x, at, total);
}
__device__ __forceinline__ void widen8(const u32x4& w, float* f) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_low(w[j]);
    f[2 * j + 1] = bf16_high(w[j]);
  }
}
__device__ __forceinline__ void load16(const uint16_t* __restrict__ x, int64_t at, float* f) {
  const u32x4 lo = load8(x, at), hi = load8(x, at + 8);
  widen8(lo, f);
  widen8(hi, f + 8);
}
// The 16 values from element `at` on, `left` of them of the row (what follows is
// the next row's): zeros behind those.
__device__ __forceinline__ void load16(const uint16_t* __restrict__ x, int64_t at, int left, int64_t total, float* f) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    u32x4 w = {0u, 0u, 0u, 0u};
    if (8 * h < left) w = load8(x, at + 8 * h, total);
    widen8(w, f + 8 * h);
  }
  if (left < 16) {
#pragma unroll
    for (int j = 0; j < 16; ++j) f[j] = j < left ? f[j] : 0.0f;
  }
}

// Quantizes the 16 values of each of a block's lanes and stores them.
__device__ __forceinline__ void store_block(const float* f, uint8_t* __restrict__ q, uint8_t* __restrict__ scale,
                                            int lane8, int pad_scales) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < kPerLane; ++j) top = max(top, magnitude(f[j]));
  const uint32_t s = scale_byte(max_of_8(top));
  const float inv = inverse_scale(s);
  u32x4 w;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = pack_e4m3(f[4 * j] * inv, f[4 * j + 1] * inv, f[4 * j + 2] * inv, f[4 * j + 3] * inv);
  *reinterpret_cast<u32x4*>(q + 16 * lane8) = w;
  // the row's last block also writes the scales that fill up the row
  if (lane8 <= pad_scales) scale[lane8] = lane8 == 0 ? (uint8_t)s : (uint8_t)127;
}

// 0 below x = -88.7, where exp(-x) leaves fp32.  exp(x) instead would keep values
// below 2^-128 and costs 5 % (131072 rows of f = 768: 112 -> 118 us).
__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }
__device__ __forceinline__ float swiglu(float g, float u) { return g * sigmoid(g) * u; }
// KIND kPlain: x [rows][cols].  kSwiglu: x [rows][2 cols] (gate, up), cols = f.
// kSwigluGrad: x [rows][cols] (gate, up) and grad [rows][cols / 2], cols = 2 f.
// A block of 128 output columns per eight lanes.  Rows of any width are read 16
// bytes at a time (element by element, widths that are no multiple of 8 took four
// times as long: 27672 rows of f = 2690, 324 us and 84 so; its gradient, 20000
// rows, 495 and 149).
template <int KIND>
__global__ __launch_bounds__(kThreads) void quantize_rows_kernel(const uint16_t* __restrict__ x,
                                                                 const uint16_t* __restrict__ grad, int64_t rows,
                                                                 int cols, uint8_t* __restrict__ q,
                                                                 uint8_t* __restrict__ scale) {
  const int nb = (cols + kBlk - 1) / kBlk, ns = (nb + 3) / 4 * 4;
  const int lane8 = threadIdx.x % kLanesPerBlock;
  const int64_t blocks = rows * nb, step = (int64_t)gridDim.x * (kThreads / kLanesPerBlock);
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / kLanesPerBlock) + threadIdx.x / kLanesPerBlock; i < blocks;
       i += step) {
    const int64_t r = i / nb;
    const int b = (int)(i - r * nb);
    const int c = b * kBlk + lane8 * kPerLane;
    float f[kPerLane];
    if (KIND == kPlain) {
      if (c + kPerLane <= cols)
        load16(x, r * cols + c, f);
      else
        load16(x, r * cols + c, cols - c, rows * cols, f);
    } else if (KIND == kSwiglu) {
      float u[kPerLane];
      const int64_t at = r * 2 * cols + c;
      if (c + kPerLane <= cols) {
        load16(x, at, f);
        load16(x, at + cols, u);
      } else {
        load16(x, at, cols - c, rows * 2 * cols, f);
        load16(x, at + cols, cols - c, rows * 2 * cols, u);
      }
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) f[j] = c + j < cols ? swiglu(f[j], u[j]) : 0.0f;
    } else {
      // Columns [0, half) are the gate's, [half, 2 half) the up's; 16 columns may
      // cross from one to the other.  The up's columns need gate and gradient
      // from `half` columns before: for those, that many elements earlier.
      const int half = cols / 2;
      float u[kPerLane], da[kPerLane];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int o = c + 8 * h;
        u32x4 g0 = {0u, 0u, 0u, 0u}, d0 = g0, u0 = g0, g1 = g0, d1 = g0;
        if (o < half) {
          g0 = load8(x, r * cols + o, rows * cols);
          u0 = load8(x, r * cols + half + o, rows * cols);
          d0 = load8(grad, r * half + o, rows * half);
        }
        if (o + 8 > half && o < cols) {
          g1 = load8(x, r * cols + o - half, rows * cols);
          d1 = load8(grad, r * half + o - half, rows * half);
        }
        float fg0[8], fg1[8], fd0[8], fd1[8];
        widen8(g0, fg0);
        widen8(g1, fg1);
        widen8(d0, fd0);
        widen8(d1, fd1);
        widen8(u0, u + 8 * h);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          f[8 * h + j] = o + j < half ? fg0[j] : fg1[j];
          da[8 * h + j] = o + j < half ? fd0[j] : fd1[j];
        }
      }
#pragma unroll
      for (int j = 0; j < kPerLane; ++j) {
        const int o = c + j;
        const float g = f[j], s = sigmoid(g);
        const float v = o < half ? da[j] * u[j] * (s * (1.0f + g * (1.0f - s))) : da[j] * (g * s);
        f[j] = o < cols ? v : 0.0f;
      }
    }
    store_block(f, q + (r * nb + b) * kBlk, scale + r * ns + b, lane8, b == nb - 1 ? ns - nb : 0);
  }
}

// The gradient where f is whole blocks: gate's and up's block in one pass over y.
__global__ __launch_bounds__(kThreads) void swiglu_grad_kernel(const uint16_t* __restrict__ y,
                                                               const uint16_t* __restrict__ grad, int64_t rows, int f,
                                                               uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  const int nb = f / kBlk, ns = (2 * nb + 3) / 4 * 4;
  const int lane8 = threadIdx.x % kLanesPerBlock;
  const int64_t blocks = rows * nb, step = (int64_t)gridDim.x * (kThreads / kLanesPerBlock);
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / kLanesPerBlock) + threadIdx.x / kLanesPerBlock; i < blocks;
       i += step) {
    const int64_t r = i / nb;
    const int b = (int)(i - r * nb);
    const int c = b * kBlk + lane8 * kPerLane;
    float g[kPerLane], u[kPerLane], da[kPerLane];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      widen8(load8(y, r * 2 * f + c + 8 * h), g + 8 * h);
      widen8(load8(y, r * 2 * f + f + c + 8 * h), u + 8 * h);
      widen8(load8(grad, r * f + c + 8 * h), da + 8 * h);
    }
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const float s = sigmoid(g[j]);
      const float dg = da[j] * u[j] * (s * (1.0f + g[j] * (1.0f - s)));
      u[j] = da[j] * (g[j] * s);
      g[j] = dg;
    }
    uint8_t* qr = q + r * 2 * f;
    store_block(g, qr + b * kBlk, scale + r * ns + b, lane8, 0);
    store_block(u, qr + f + b * kBlk, scale + r * ns + nb + b, lane8, b == nb - 1 ? ns - 2 * nb : 0);
  }
}

// One 128 x 128 block of a matrix per workgroup.  Thread (g, c8): rows 8g ..
// 8g+7, columns 8 c8 .. 8 c8+7, so a wave loads whole 256-byte row pieces and
// every thread can transpose its 8 x 8 bytes itself.
constexpr int kTransStride = kBlk + 16;  // LDS bytes of a row of the transposed block
__global__ __launch_bounds__(kThreads) void quantize_weights_kernel(const uint16_t* __restrict__ w, int experts,
                                                                    int n, int k, int nbn, int nbk,
                                                                    uint8_t* __restrict__ q,
                                                                    uint8_t* __restrict__ scale,
                                                                    uint8_t* __restrict__ qt,
                                                                    uint8_t* __restrict__ scale_t) {
  __shared__ __align__(16) uint8_t tr[kBlk * kTransStride];
  __shared__ uint32_t top_s[kThreads / 64];
  const int bk = blockIdx.x % nbk;
  const int rest = blockIdx.x / nbk;
  const int bn = rest % nbn, e = rest / nbn;
  const int c8 = threadIdx.x % 16, rg = threadIdx.x / 16;
  const int c = bk * kBlk + 8 * c8, r0 = bn * kBlk + 8 * rg;
  const uint16_t* __restrict__ base = w + (int64_t)e * n * k;
  u32x4 v[8];
  const int rows = c < k ? min(8, n - r0) : 0;  // this thread's, possibly none
  if (rows == 8 && c + 8 <= k) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = load8(base, (int64_t)(r0 + j) * k + c);
  } else {
    const int64_t total = (int64_t)(experts - e) * n * k;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t at = (int64_t)(r0 + (j < rows ? j : 0)) * k + c;
      v[j] = u32x4{0u, 0u, 0u, 0u};
      if (j < rows) v[j] = at + 8 <= total ? load8(base, at) : load8_edge(base, at, total);
#pragma unroll
      for (int i = 0; i < 4; ++i)  // columns from k on are the next row's
        v[j][i] &= (c + 2 * i < k ? 0xffffu : 0u) | (c + 2 * i + 1 < k ? 0xffff0000u : 0u);
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(v[j][i] & 0x7fff0000u, (v[j][i] << 16) & 0x7fff0000u));
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off));
  if ((threadIdx.x & 63) == 0) top_s[threadIdx.x >> 6] = top;
  __syncthreads();
  top = max(max(top_s[0], top_s[1]), max(top_s[2], top_s[3]));
  const uint32_t s = scale_byte(top);
  const float inv = inverse_scale(s);
  const int nsk = (nbk + 3) / 4 * 4, nsn = (nbn + 3) / 4 * 4;
  const int kp = nbk * kBlk, np = nbn * kBlk;
  u32x2 b[8];  // bytes of columns 0..3 and 4..7 of each row
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    b[j][0] = pack_e4m3(bf16_low(v[j][0]) * inv, bf16_high(v[j][0]) * inv, bf16_low(v[j][1]) * inv,
                        bf16_high(v[j][1]) * inv);
    b[j][1] = pack_e4m3(bf16_low(v[j][2]) * inv, bf16_high(v[j][2]) * inv, bf16_low(v[j][3]) * inv,
                        bf16_high(v[j][3]) * inv);
    if (r0 + j < n) *reinterpret_cast<u32x2*>(q + ((int64_t)e * n + r0 + j) * kp + c) = b[j];
  }
  if (threadIdx.x < 4) {
    const int i = threadIdx.x;  // the last block of a row of scales fills it up
    if (i == 0 || (bk == nbk - 1 && bk + i < nsk))
      scale[((int64_t)e * nbn + bn) * nsk + bk + i] = i == 0 ? (uint8_t)s : (uint8_t)127;
    if (qt && (i == 0 || (bn == nbn - 1 && bn + i < nsn)))
      scale_t[((int64_t)e * nbk + bk) * nsn + bn + i] = i == 0 ? (uint8_t)s : (uint8_t)127;
  }
  if (!qt) return;
  // 4 x 4 byte transposes: first pairs of rows, then pairs of pairs
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    u32x2 t[4];  // column 4h + i, rows 8rg .. 8rg+7
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t a0 = b[4 * p][h], a1 = b[4 * p + 1][h], a2 = b[4 * p + 2][h], a3 = b[4 * p + 3][h];
      // selector bytes 0..3 pick from the second operand, 4..7 from the first
      const uint32_t lo01 = __builtin_amdgcn_perm(a1, a0, 0x05010400u), hi01 = __builtin_amdgcn_perm(a1, a0, 0x07030602u);
      const uint32_t lo23 = __builtin_amdgcn_perm(a3, a2, 0x05010400u), hi23 = __builtin_amdgcn_perm(a3, a2, 0x07030602u);
      t[0][p] = __builtin_amdgcn_perm(lo23, lo01, 0x05040100u);
      t[1][p] = __builtin_amdgcn_perm(lo23, lo01, 0x07060302u);
      t[2][p] = __builtin_amdgcn_perm(hi23, hi01, 0x05040100u);
      t[3][p] = __builtin_amdgcn_perm(hi23, hi01, 0x07060302u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<u32x2*>(tr + (8 * c8 + 4 * h + i) * kTransStride + 8 * rg) = t[i];
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int i = threadIdx.x + p * kThreads;  // 16-byte piece: row i / 8 of the transposed block
    const int row = bk * kBlk + i / 8;
    if (row < k)
      *reinterpret_cast<u32x4*>(qt + ((int64_t)e * k + row) * np + bn * kBlk + 16 * (i % 8)) =
          *reinterpret_cast<const u32x4*>(tr + (i / 8) * kTransStride + 16 * (i % 8));
  }
}

unsigned grid_of(int64_t blocks) {
  const int64_t g = (blocks + kThreads / kLanesPerBlock - 1) / (kThreads / kLanesPerBlock);
  return (unsigned)(g < kMaxGrid ? g : kMaxGrid);
}

template <int KIND>
hipError_t launch_rows(const uint16_t* x, const uint16_t* grad, int64_t rows, int cols, uint8_t* q, uint8_t* scale,
                       hipStream_t st) {
  if (rows == 0) return hipSuccess;
  hipLaunchKernelGGL((quantize_rows_kernel<KIND>), dim3(grid_of(rows * (padded_cols(cols) / kBlk))), dim3(kThreads), 0,
                     st, x, grad, rows, cols, q, scale);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize(const uint16_t* x, int64_t rows, int32_t cols, uint8_t* q, uint8_t* scale, hipStream_t st) {
  return launch_rows<kPlain>(x, nullptr, rows, cols, q, scale, st);
}

hipError_t launch_swiglu(const uint16_t* y, int64_t rows, int32_t f, uint8_t* q, uint8_t* scale, hipStream_t st) {
  return launch_rows<kSwiglu>(y, nullptr, rows, f, q, scale, st);
}

hipError_t launch_swiglu_grad(const uint16_t* y, const uint16_t* grad, int64_t rows, int32_t f, uint8_t* q,
                              uint8_t* scale, hipStream_t st) {
  if (f % kBlk != 0) return launch_rows<kSwigluGrad>(y, grad, rows, 2 * f, q, scale, st);
  if (rows == 0) return hipSuccess;
  hipLaunchKernelGGL(swiglu_grad_kernel, dim3(grid_of(rows * (f / kBlk))), dim3(kThreads), 0, st, y, grad, rows, f, q,
                     scale);
  return hipGetLastError();
}

hipError_t launch_quantize_weights(const uint16_t* w, int32_t experts, int32_t n, int32_t k, uint8_t* q,
                                   uint8_t* scale, uint8_t* qt, uint8_t* scale_t, hipStream_t st) {
  const int nbn = (int)(padded_cols(n) / kBlk), nbk = (int)(padded_cols(k) / kBlk);
  const int64_t blocks = (int64_t)experts * nbn * nbk;
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(quantize_weights_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, st, w, experts, n, k, nbn,
                     nbk, q, scale, qt, scale_t);
  return hipGetLastError();
}

}  // namespace moe
