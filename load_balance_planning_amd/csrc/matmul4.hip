// The experts' products with matrices in 4 bits on gfx950: y[r][c] = sum_j
// x[r][j] w[e(r)][c][j], w e2m1 values with a power-of-two scale per 32 along j,
// x the same or e4m3 with a scale per 128.
//
// The scaled matrix instruction takes each operand in a format of its own and
// multiplies by both scales.  Its blocks of 32 along the summed axis are, for
// 4-bit operands, one lane's 16 bytes, whose scale that lane gives.  8-bit
// operands hold a block in two lanes, 16 bytes each: of 16x16x128, lane group g
// has bytes 16 g on and 64 + 16 g on, with 32x32x64 bytes 16 g on and 32 + 16 g
// on.  As in the 8-bit products the matrices are the first operand, so a lane's
// results are channels of one row.
#include "buffers.h"
#include "experts4.h"
#include "fp4_block.h"
#include "instances.h"
#include "product_tiles.h"
#include "store_tile.h"

namespace moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// The instruction's operand of 16 bytes of 4-bit values; it reads no more.
__device__ __forceinline__ v8i operand4(v4i v) { return v8i{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }
__device__ __forceinline__ v8i operand8(v4i lo, v4i hi) {
  return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}
__device__ __forceinline__ v4i load16b(const uint8_t* p) { return *reinterpret_cast<const v4i*>(p); }

constexpr int kFp8 = 0, kFp4 = 4;  // the instruction's format codes

// 16 rows x 64 channels per workgroup; its four waves take every fourth line of
// the long axis each (256 values: two instructions), straight from memory to
// registers, and add their sums in LDS.
constexpr int kRowsS = 16, kChanS = 64;
template <int XB>
__global__ __launch_bounds__(256) void matmul4_rows16_kernel(Instances in, const uint8_t* __restrict__ x,
                                                             const uint8_t* __restrict__ xs,
                                                             const uint8_t* __restrict__ w,
                                                             const uint8_t* __restrict__ ws, int n, int k,
                                                             int64_t tiles, uint16_t* __restrict__ y,
                                                             int32_t* __restrict__ status) {
  __shared__ float part[4][kRowsS][kChanS + 4];
  if (blockIdx.x == 0) check_instances(in, status);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int nb = (k + kCols4 - 1) / kCols4;                             // lines of a 4-bit row
  const int nb8 = (k + kBlk - 1) / kBlk, ns8 = (nb8 + 3) / 4 * 4;      // blocks of an 8-bit row
  const int64_t line = kCols4 / 2;
  const int nct = (n + kChanS - 1) / kChanS;
  for (int64_t id = blockIdx.x; id < tiles; id += gridDim.x) {
    const int64_t rt = id / nct;
    const int c0 = (int)(id - rt * nct) * kChanS;
    Span sp;
    int64_t r0;
    if (!find_row_tile<kRowsS>(in, rt, &sp, &r0)) continue;  // the same for all waves
    const int64_t row = min(r0 + r, sp.end - 1);
    const uint8_t* wp[4];
    const uint8_t* wsp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = min(c0 + 16 * (r >> 2) + 4 * i + (r & 3), n - 1);
      wp[i] = w + ((int64_t)sp.expert * n + c) * nb * line + 16 * g;
      wsp[i] = ws + ((int64_t)sp.expert * nb * n + c) * 8;
    }
    v4f acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = v4f{0, 0, 0, 0};
    for (int b = wave; b < nb; b += 4) {
      v8i xv[2];
      uint32_t sx[2];
      if (XB == 4) {
        const uint8_t* xp = x + (row * nb + b) * line + 16 * g;
        const u32x2 s = *reinterpret_cast<const u32x2*>(xs + ((int64_t)b * in.rows + row) * 8);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          xv[h] = operand4(load16b(xp + 64 * h));
          sx[h] = s[h] >> (8 * g);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // past the last block the matrices' values are zeros: any block will do
          const int b8 = min(2 * b + h, nb8 - 1);
          const uint8_t* xp = x + (row * nb8 + b8) * kBlk + 16 * g;
          xv[h] = operand8(load16b(xp), load16b(xp + 64));
          sx[h] = xs[row * ns8 + b8];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x2 s = *reinterpret_cast<const u32x2*>(wsp[i] + (int64_t)b * n * 8);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand4(load16b(wp[i] + b * line + 64 * h)), xv[h],
                                                                    acc[i], kFp4, XB == 4 ? kFp4 : kFp8, 0,
                                                                    (int)(s[h] >> (8 * g)), 0, (int)sx[h]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<v4f*>(&part[wave][r][16 * g + 4 * i]) = acc[i];
    __syncthreads();
    const int orow = threadIdx.x >> 4, oc = 4 * (threadIdx.x & 15);
    v4f sum = *reinterpret_cast<const v4f*>(&part[0][orow][oc]);
#pragma unroll
    for (int q = 1; q < 4; ++q) sum += *reinterpret_cast<const v4f*>(&part[q][orow][oc]);
    if (r0 + orow < sp.end) {
      uint16_t* dst = y + (r0 + orow) * n + c0 + oc;
      const uint32_t lo = pack_bf16(sum[0], sum[1]), hi = pack_bf16(sum[2], sum[3]);
      if (c0 + oc + 3 < n) {
        typedef u32x2 u32x2_any __attribute__((aligned(2)));
        *reinterpret_cast<u32x2_any*>(dst) = u32x2{lo, hi};
      } else {
        if (c0 + oc < n) dst[0] = (uint16_t)lo;
        if (c0 + oc + 1 < n) dst[1] = (uint16_t)(lo >> 16);
        if (c0 + oc + 2 < n) dst[2] = (uint16_t)hi;
        if (c0 + oc + 3 < n) dst[3] = (uint16_t)(hi >> 16);
      }
    }
    __syncthreads();
  }
}

template <int XB>
hipError_t launch_rows16(const Instances& in, const uint8_t* x, const uint8_t* xs, const uint8_t* w, const uint8_t* ws,
                         int n, int k, uint16_t* y, int32_t* status, hipStream_t st) {
  // without rows one workgroup, which only looks at the plan
  const int64_t tiles = in.rows == 0 ? 0 : row_tile_ids(in, kRowsS) * ((n + kChanS - 1) / kChanS);
  const int64_t grid = tiles < 1 ? 1 : tiles < (1 << 20) ? tiles : (1 << 20);
  hipLaunchKernelGGL((matmul4_rows16_kernel<XB>), dim3((unsigned)grid), dim3(256), 0, st, in, x, xs, w, ws, n, k,
                     tiles, y, status);
  return hipGetLastError();
}

}  // namespace

int64_t matmul4_tiles(const Instances&, int32_t) { return 0; }

hipError_t launch_matmul4(const Instances& in, int32_t x_bits, const uint8_t* x, const uint8_t* xs, const uint8_t* w,
                          const uint8_t* ws, int32_t n, int32_t k, uint16_t* y, int32_t* status, hipStream_t st) {
  return x_bits == 4 ? launch_rows16<4>(in, x, xs, w, ws, n, k, y, status, st)
                     : launch_rows16<8>(in, x, xs, w, ws, n, k, y, status, st);
}

}  // namespace moe
