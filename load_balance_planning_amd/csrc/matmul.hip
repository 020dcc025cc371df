// The experts' products on gfx950: y[r][c] = sum_j x[r][j] w[e(r)][c][j] over
// e4m3 values with a power-of-two scale per block of 128.
//
// The 16x16x128 matrix instruction takes a block of 128 of both operands and
// multiplies by both scales itself, so a scale costs no arithmetic here.  The
// matrices are its first operand and the rows its second: a lane's four
// results are then four channels of one row.  Which channel a matrix row of
// the instruction stands for is free; row 4g + j of tile i is channel
// 16g + 4i + j, so four tiles give a lane 16 consecutive channels (32 bytes).
#include "experts.h"
#include "fp8_block.h"
#include "instances.h"

namespace moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// 32 of a row's 128 bytes: the 16 of lane group g in each half.  (Both
// operands use the same order, so any order of the block does.)
__device__ __forceinline__ v8i load_block(const uint8_t* __restrict__ row, int g) {
  union {
    v8i v;
    v4i h[2];
  } u;
  u.h[0] = *reinterpret_cast<const v4i*>(row + 16 * g);
  u.h[1] = *reinterpret_cast<const v4i*>(row + 64 + 16 * g);
  return u.v;
}

// 16 rows x 64 channels per workgroup; its four waves take every fourth block
// of the long axis each, straight from memory to registers, and add their sums
// in LDS.
constexpr int kRowsS = 16, kChanS = 64;
__global__ __launch_bounds__(256) void matmul_rows16_kernel(Instances in, const uint8_t* __restrict__ x,
                                                            const uint8_t* __restrict__ xs,
                                                            const uint8_t* __restrict__ w,
                                                            const uint8_t* __restrict__ ws, int n, int k,
                                                            int64_t tiles, uint16_t* __restrict__ y,
                                                            int32_t* __restrict__ status) {
  __shared__ float part[4][kRowsS][kChanS + 4];
  if (blockIdx.x == 0) check_instances(in, status);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int nb = (k + kBlk - 1) / kBlk, ns = (nb + 3) / 4 * 4;
  const int64_t kp = (int64_t)nb * kBlk;
  const int nbn = (n + kBlk - 1) / kBlk, nct = (n + kChanS - 1) / kChanS;
  const int n_inst = instance_count(in);
  for (int64_t id = blockIdx.x; id < tiles; id += gridDim.x) {
    const int64_t rt = id / nct;
    const int c0 = (int)(id - rt * nct) * kChanS;
    Span sp;
    int64_t r0;
    if (!find_row_tile<kRowsS>(in, n_inst, rt, &sp, &r0)) continue;  // the same for all waves
    const int64_t row = min(r0 + r, sp.end - 1);
    const uint8_t* xp = x + row * kp;
    const uint8_t* xsp = xs + row * ns;
    const uint8_t* wsp = ws + ((int64_t)sp.expert * nbn + c0 / kBlk) * ns;
    const uint8_t* wp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = min(c0 + 16 * (r >> 2) + 4 * i + (r & 3), n - 1);
      wp[i] = w + ((int64_t)sp.expert * n + c) * kp;
    }
    v4f acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = v4f{0, 0, 0, 0};
    for (int b = wave; b < nb; b += 4) {
      const v8i xv = load_block(xp + b * kBlk, g);
      const int sx = xsp[b], sw = wsp[b];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(load_block(wp[i] + b * kBlk, g), xv, acc[i], 0, 0, 0,
                                                                  sw, 0, sx);
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
      if (c0 + oc + 3 < n && n % 4 == 0 && ((uintptr_t)y & 7) == 0) {
        *reinterpret_cast<u32x2*>(dst) = u32x2{lo, hi};
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

}  // namespace

hipError_t launch_matmul(const Instances& in, const uint8_t* x, const uint8_t* xs, const uint8_t* w, const uint8_t* ws,
                         int32_t n, int32_t k, uint16_t* y, int32_t* status, hipStream_t st) {
  if (in.rows == 0) return hipSuccess;
  const int64_t tiles = row_tile_ids(in, kRowsS) * ((n + kChanS - 1) / kChanS);
  const int64_t grid = tiles < (1 << 20) ? tiles : (1 << 20);
  hipLaunchKernelGGL(matmul_rows16_kernel, dim3((unsigned)grid), dim3(256), 0, st, in, x, xs, w, ws, n, k, tiles, y,
                     status);
  return hipGetLastError();
}

}  // namespace moe
