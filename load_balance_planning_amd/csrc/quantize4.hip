// Block quantization to e2m1 on gfx950: rows (one scale per 1 x 32), expert
// matrices in both layouts, the gated activation fused with the row form, and
// the values back.
//
//   s = smallest power of two with max|x| <= 6 s,  q = e2m1(x / s)
//
// All of these move bytes once: 2 read and 0.53 written per value (matrices in
// both layouts 2 and 1.06, activation 4 and 0.53, values 0.53 and 2).  A copy of
// 2 GiB moves 4.8 TB/s here, and reads alone 6.1.
#include "experts4.h"
#include "fp4_block.h"
#include "row_load.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxGrid = 1 << 20;

// Largest of an aligned pair, or of four, of lanes.
__device__ __forceinline__ uint32_t max_of_2(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, false));
}
__device__ __forceinline__ uint32_t max_of_4(uint32_t v) {
  v = max_of_2(v);
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, false));
}

// g sigmoid(g) u to 2^-20, in a dozen instructions: the exponential as 2^t with what t
// = -g log2(e) lost to rounding, 1 / (1 + e) as a reciprocal of a quarter of it, which
// stays a normal number.  As with expf and a division, 0 below g = -88.7.
__device__ __forceinline__ float swiglu_near(float g, float u) {
  const float x = __builtin_amdgcn_fmed3f(g, -128.0f, 128.0f);  // past these 0 and 1; g itself brings its NaN
  const float t = x * -1.44269502f;
  const float lost = fmaf(x, -1.44269502f, -t) + x * -1.92596303e-8f;
  const float e = __builtin_amdgcn_exp2f(t) * fmaf(lost, 0.693147182f, 1.0f);
  return g * (0.25f * __builtin_amdgcn_rcpf(fmaf(0.25f, e, 0.25f))) * u;
}

// Sixteen rows by 256 columns per workgroup, 16 values to a thread: whole
// 128-byte lines of results, and their scales are one line too.  Memory-bound:
// 131072 rows of 2048 117 us (5.8 TB/s).  SWIGLU: x [rows][2 cols], gate and up;
// 32768 rows of 2688 75 us (5.3 TB/s; with expf and a division, 40 vector
// instructions a value in all, 92).
constexpr int kTileRows = 16;
template <bool SWIGLU>
__global__ __launch_bounds__(kThreads) void quantize4_rows_kernel(const uint16_t* __restrict__ x, int64_t rows,
                                                                  int cols, uint8_t* __restrict__ q,
                                                                  uint8_t* __restrict__ scale) {
  const int nb = (cols + kCols4 - 1) / kCols4;
  const int64_t tiles = (rows + kTileRows - 1) / kTileRows * nb;
  const int lane16 = threadIdx.x & 15;
  const int64_t width = SWIGLU ? 2 * (int64_t)cols : cols;
  for (int64_t i = blockIdx.x; i < tiles; i += gridDim.x) {
    const int64_t rt = i / nb;
    const int b = (int)(i - rt * nb);
    const int64_t r = rt * kTileRows + (threadIdx.x >> 4);
    if (r >= rows) continue;  // whole groups of 16 lanes
    const int c = b * kCols4 + lane16 * 16;
    float f[16], u[16];
    if (c + 16 <= cols) {
      load16(x, r * width + c, f);
      if (SWIGLU) load16(x, r * width + cols + c, u);
    } else {
      load16(x, r * width + c, cols - c, rows * width, f);
      if (SWIGLU) load16(x, r * width + cols + c, cols - c, rows * width, u);
    }
    if (SWIGLU) {
#pragma unroll
      for (int j = 0; j < 16; ++j) f[j] = c + j < cols ? swiglu_near(f[j], u[j]) : 0.0f;
    }
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) top = max(top, magnitude(f[j]));
    const uint32_t s = scale_byte4(max_of_2(top));
    const float inv = inverse_scale(s);
#pragma unroll
    for (int j = 0; j < 16; ++j) f[j] *= inv;
    u32x2 w = {pack_e2m1(f), pack_e2m1(f + 8)};
    if (s == 255u) w = u32x2{0u, 0u};
    *reinterpret_cast<u32x2*>(q + (r * nb + b) * (kCols4 / 2) + 8 * lane16) = w;
    if ((lane16 & 1) == 0) scale[((int64_t)b * rows + r) * 8 + (lane16 >> 1)] = (uint8_t)s;
  }
}

// One 128 x 128 piece of a matrix per workgroup.  Thread (g, c8): rows 8g ..
// 8g+7, columns 8 c8 .. 8 c8+7, so a wave loads whole 256-byte row pieces.  A
// block of 32 columns is four neighbouring threads', one of 32 rows those of a
// wave with the same columns; the transposed bytes pass through LDS.
//
// Values stay bf16 pairs: the conversion divides by the scale, and magnitudes
// compare as integers.  Memory-bound: 128 matrices of 1536 x 2048 in both layouts
// 200 us (6.1 TB/s) where values4_kernel reads the results next, 267 (4.6) one such
// launch right behind the other, in one layout 164 (6.2) so; 8 of 4096 x 7168 in
// both 124 (5.8).  In fp32, the pieces dealt to the XCDs one by one, and with 8-way
// conflicts in LDS, one behind the other: 296 and 154.
constexpr int kTransStride4 = kBlk / 2 + 16;  // LDS bytes of a row of the transposed piece
// Its 16-byte pieces are exchanged so that eight rows' lie in different banks.
__device__ __forceinline__ int trans_place(int row, int piece) { return 16 * (piece ^ ((row >> 4) & 3)); }
__global__ __launch_bounds__(kThreads) void quantize4_weights_kernel(const uint16_t* __restrict__ w, int experts,
                                                                     int n, int k, int pn, int pk,
                                                                     uint8_t* __restrict__ q,
                                                                     uint8_t* __restrict__ scale,
                                                                     uint8_t* __restrict__ qt,
                                                                     uint8_t* __restrict__ scale_t) {
  __shared__ __align__(16) uint8_t tr[kBlk * kTransStride4];
  __shared__ uint32_t s_row[kBlk], s_col[kBlk];  // four scales each
  // Every XCD takes a run of pieces: two side by side write a 128-byte line together,
  // in one L2 then.
  const int id = (int)(blockIdx.x & 7) * (int)(gridDim.x >> 3) + (int)(blockIdx.x >> 3);
  const int rest = id / pk, bk = id - rest * pk, e = rest / pn, bn = rest - e * pn;
  if (e >= experts) return;
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
  const int nbk = pk / 2, nbn = pn / 2;  // lines of 256 values
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t top = v[j][0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 4; ++i) top = pk_max(top, v[j][i] & 0x7fff7fffu);
    const uint32_t s = scale_byte4(max_of_4(max(top << 16, top & 0xffff0000u)));
    const uint32_t o = pack_e2m1(v[j][0], v[j][1], v[j][2], v[j][3], s);
    if (r0 + j < n)
      *reinterpret_cast<uint32_t*>(q + (((int64_t)e * n + r0 + j) * pk + bk) * (kBlk / 2) + 4 * c8) = o;
    if ((c8 & 3) == 0) reinterpret_cast<uint8_t*>(s_row)[(8 * rg + j) * 4 + (c8 >> 2)] = (uint8_t)s;
  }
  if (qt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // two columns
      uint32_t top = v[0][i] & 0x7fff7fffu;
#pragma unroll
      for (int j = 1; j < 8; ++j) top = pk_max(top, v[j][i] & 0x7fff7fffu);
      top = pk_max(top, (uint32_t)__shfl_xor((int)top, 16));
      top = pk_max(top, (uint32_t)__shfl_xor((int)top, 32));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[j] = __builtin_amdgcn_perm(v[2 * j + 1][i], v[2 * j][i], h ? 0x07060302u : 0x05040100u);
        const uint32_t s = scale_byte4(h ? top & 0xffff0000u : top << 16);
        const int col = 8 * c8 + 2 * i + h;
        *reinterpret_cast<uint32_t*>(tr + col * kTransStride4 + trans_place(col, rg >> 2) + 4 * (rg & 3)) =
            pack_e2m1(x[0], x[1], x[2], x[3], s);
        if ((rg & 3) == 0) reinterpret_cast<uint8_t*>(s_col)[col * 4 + (rg >> 2)] = (uint8_t)s;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < kBlk) {
    const int r = bn * kBlk + threadIdx.x;
    if (r < n)
      *reinterpret_cast<uint32_t*>(scale + (((int64_t)e * nbk + bk / 2) * n + r) * 8 + 4 * (bk & 1)) =
          s_row[threadIdx.x];
  } else if (qt) {
    const int i = threadIdx.x - kBlk, r = bk * kBlk + i;
    if (r < k)
      *reinterpret_cast<uint32_t*>(scale_t + (((int64_t)e * nbn + bn / 2) * k + r) * 8 + 4 * (bn & 1)) = s_col[i];
  }
  if (!qt) return;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int i = threadIdx.x + p * kThreads;  // 16-byte piece: row i / 4 of the transposed piece
    const int row = bk * kBlk + i / 4;
    if (row < k)
      *reinterpret_cast<u32x4*>(qt + (((int64_t)e * k + row) * pn + bn) * (kBlk / 2) + 16 * (i % 4)) =
          *reinterpret_cast<const u32x4*>(tr + (i / 4) * kTransStride4 + trans_place(i / 4, i % 4));
  }
}

// 32 rows by 256 columns per workgroup, 8 values of four rows to a thread: four
// loads under way each.  128 matrices of 1536 x 2048 176 us (5.8 TB/s).
constexpr int kValueRows = 32;
__global__ __launch_bounds__(kThreads) void values4_kernel(const uint8_t* __restrict__ q,
                                                           const uint8_t* __restrict__ scale, int matrices,
                                                           int64_t rows, int cols, uint16_t* __restrict__ x) {
  const int nb = (cols + kCols4 - 1) / kCols4;
  const int64_t row_tiles = (rows + kValueRows - 1) / kValueRows, tiles = matrices * row_tiles * nb;
  const int lane32 = threadIdx.x & 31;
  for (int64_t i = blockIdx.x; i < tiles; i += gridDim.x) {
    const int64_t mr = i / nb, m = mr / row_tiles;
    const int b = (int)(i - mr * nb);
    const int64_t r0 = (mr - m * row_tiles) * kValueRows + (threadIdx.x >> 5);
    const int c = b * kCols4 + lane32 * 8;
    uint32_t w[4], s[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = min(r0 + 8 * j, rows - 1);
      w[j] = __builtin_nontemporal_load(
          reinterpret_cast<const uint32_t*>(q + ((m * rows + r) * nb + b) * (kCols4 / 2) + 4 * lane32));
      s[j] = scale[((m * nb + b) * rows + r) * 8 + (lane32 >> 2)];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t r = r0 + 8 * j;
      if (r >= rows || c >= cols) continue;
      const float by = scale_value(s[j]);
      u32x4 o;
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      const f32x2 v[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], 1.0f, 0),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], 1.0f, 1),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], 1.0f, 2),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[j], 1.0f, 3)};
#pragma unroll
      for (int h = 0; h < 4; ++h) o[h] = s[j] == 255u ? 0x7fc07fc0u : pack_bf16(v[h][0] * by, v[h][1] * by);
      uint16_t* dst = x + (m * rows + r) * cols + c;
      if (c + 8 <= cols) {
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4_any*>(dst));
      } else {
#pragma unroll
        for (int h = 0; h < 8; ++h)
          if (c + h < cols) dst[h] = (uint16_t)(o[h / 2] >> (16 * (h & 1)));
      }
    }
  }
}

unsigned grid_of(int64_t tiles) { return (unsigned)(tiles < kMaxGrid ? tiles : kMaxGrid); }

template <bool SWIGLU>
hipError_t launch_rows(const uint16_t* x, int64_t rows, int cols, uint8_t* q, uint8_t* scale, hipStream_t st) {
  if (rows == 0) return hipSuccess;
  hipLaunchKernelGGL((quantize4_rows_kernel<SWIGLU>),
                     dim3(grid_of((rows + kTileRows - 1) / kTileRows * (padded_cols4(cols) / kCols4))), dim3(kThreads),
                     0, st, x, rows, cols, q, scale);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize4(const uint16_t* x, int64_t rows, int32_t cols, uint8_t* q, uint8_t* scale, hipStream_t st) {
  return launch_rows<false>(x, rows, cols, q, scale, st);
}

hipError_t launch_swiglu4(const uint16_t* y, int64_t rows, int32_t f, uint8_t* q, uint8_t* scale, hipStream_t st) {
  return launch_rows<true>(y, rows, f, q, scale, st);
}

hipError_t launch_quantize_weights4(const uint16_t* w, int32_t experts, int32_t n, int32_t k, uint8_t* q,
                                    uint8_t* scale, uint8_t* qt, uint8_t* scale_t, hipStream_t st) {
  // pieces of 128 x 128, in whole lines of 256 values along both axes
  const int pn = (int)(padded_cols4(n) / kBlk), pk = (int)(padded_cols4(k) / kBlk);
  const int64_t pieces = (int64_t)experts * pn * pk;
  if (pieces == 0) return hipSuccess;
  hipLaunchKernelGGL(quantize4_weights_kernel, dim3((unsigned)((pieces + 7) / 8 * 8)), dim3(kThreads), 0, st, w,
                     experts, n, k, pn, pk, q, scale, qt, scale_t);
  return hipGetLastError();
}

hipError_t launch_values4(const uint8_t* q, const uint8_t* scale, int32_t matrices, int64_t rows, int32_t cols,
                          uint16_t* x, hipStream_t st) {
  const int64_t tiles = matrices * ((rows + kValueRows - 1) / kValueRows) * (padded_cols4(cols) / kCols4);
  if (tiles == 0) return hipSuccess;
  hipLaunchKernelGGL(values4_kernel, dim3(grid_of(tiles)), dim3(kThreads), 0, st, q, scale, matrices, rows, cols, x);
  return hipGetLastError();
}

}  // namespace moe
