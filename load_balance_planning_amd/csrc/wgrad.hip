// Gradient of the experts' matrices on gfx950:
//   dw[e][c][j] = sum over the rows r of e's instances of dy[r][c] x[r][j]
//
// The sum runs over rows, along which both operands change scale, so the
// scaled 8-bit instruction does not apply; the values are widened to bf16 --
// e4m3 times a power of two is a bf16 value exactly -- and multiplied by the
// bf16 instruction.  The instruction wants eight consecutive rows of one
// column in a lane, memory has columns next to each other: a thread loads an
// 8 x 8 piece, widens it, transposes it in registers and writes eight 16-byte
// pieces (eight rows of a column) to LDS.
//
// LDS holds [column][64 rows], 128 bytes a column.  Its 16-byte pieces are
// placed so that both the writes (columns 8 apart) and the reads (consecutive
// columns) of 16 lanes fall into 16 different places of 256 bytes: piece p of
// column c lies at 256 * (c / 2) + 16 * ((8 * (c % 2) + p) ^ s(c)).
#include "experts.h"
#include "fp8_block.h"
#include "instances.h"

namespace moe {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int kStepRows = 64;

__device__ __forceinline__ int lds_piece(int c, int p) {
  const int s = ((c >> 1) & 7) ^ ((c >> 4) & 3) ^ (((c >> 6) & 1) << 3);
  return (c >> 1) * 256 + ((((c & 1) << 3) | p) ^ s) * 16;
}

// Eight rows of eight columns, widened: rows begin + 0..7 (zeros from `end`
// on), columns c .. c+7 of a row of cp bytes.
struct Piece {
  u32x2 q[8];
  uint32_t s[8];
};
__device__ __forceinline__ void load_piece(Piece* p, const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                                           int64_t begin, int64_t end, int64_t cp, int ns, int c) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool in = begin + j < end && c < cp;
    p->q[j] = in ? *reinterpret_cast<const u32x2*>(q + (begin + j) * cp + c) : u32x2{0u, 0u};
    p->s[j] = in ? scale[(begin + j) * ns + c / kBlk] : 127u;
  }
}

// Transposed to LDS: for each column its eight rows as one 16-byte piece.
__device__ __forceinline__ void store_piece(const Piece& p, unsigned char* lds, int c, int piece) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(p.s[j] << 23);  // 255 gives NaN for the whole block
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[8][2];  // [row][columns 4h, 4h+1 | 4h+2, 4h+3]
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[j][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p.q[j][h], f[j], false));
      w[j][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p.q[j][h], f[j], true));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u32x4 o;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o[j] = __builtin_amdgcn_perm(w[2 * j + 1][i / 2], w[2 * j][i / 2], i & 1 ? 0x07060302u : 0x05040100u);
      *reinterpret_cast<u32x4*>(lds + lds_piece(c + 4 * h + i, piece)) = o;
    }
  }
}

// A 128 x 128 piece of dw[e] per workgroup of four waves, 64 x 64 each.
constexpr int kTile128 = 128;
__global__ __launch_bounds__(256) void wgrad_kernel(Instances in, const uint8_t* __restrict__ dy,
                                                    const uint8_t* __restrict__ dys, const uint8_t* __restrict__ x,
                                                    const uint8_t* __restrict__ xs, int n, int k,
                                                    uint16_t* __restrict__ dw, int32_t* __restrict__ status) {
  __shared__ __align__(16) unsigned char a_s[kTile128 * kStepRows * 2];  // columns of x
  __shared__ __align__(16) unsigned char b_s[kTile128 * kStepRows * 2];  // columns of dy
  __shared__ int list[kMaxE + kMaxB];
  __shared__ int list_n;
  if (blockIdx.x == 0) check_instances(in, status);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int ntk = (k + kTile128 - 1) / kTile128, ntn = (n + kTile128 - 1) / kTile128;
  const int tk = blockIdx.x % ntk, rest = blockIdx.x / ntk;
  const int tn = rest % ntn, e = rest / ntn;
  const int n_inst = instance_count(in);
  if (wave == 0) {
    int m = 0;
    for (int i0 = 0; i0 < n_inst; i0 += 64) {
      const bool hit = i0 + lane < n_inst && in.expert[i0 + lane] == e;
      const uint64_t bits = __ballot(hit);
      if (hit) list[m + __popcll(bits & ((1ull << lane) - 1ull))] = i0 + lane;
      m += __popcll(bits);
    }
    if (lane == 0) list_n = m;
  }
  __syncthreads();
  const int nbn = (n + kBlk - 1) / kBlk, nbk = (k + kBlk - 1) / kBlk;
  const int nsn = (nbn + 3) / 4 * 4, nsk = (nbk + 3) / 4 * 4;
  const int64_t np = (int64_t)nbn * kBlk, kp = (int64_t)nbk * kBlk;
  // thread: columns 8 c8 .. of the tile, rows 8 rg .. of the step, for rg and rg + ...
  const int c8 = threadIdx.x % 16, rg0 = threadIdx.x / 16;
  const int wk = (wave & 1) * 64, wn = (wave >> 1) * 64;
  v4f acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0, 0, 0, 0};
  const int m = list_n;
  for (int q = 0; q < m; ++q) {
    Span sp;
    if (!instance_span(in, list[q], &sp)) continue;
    for (int64_t r0 = sp.begin; r0 < sp.end; r0 += kStepRows) {
      {
        // 16 column groups x 8 row groups for each operand: the first half of the threads takes x
        const int rg = rg0 & 7;
        const bool is_x = rg0 < 8;
        Piece p;
        if (is_x) load_piece(&p, x, xs, r0 + 8 * rg, sp.end, kp, nsk, tk * kTile128 + 8 * c8);
        else load_piece(&p, dy, dys, r0 + 8 * rg, sp.end, np, nsn, tn * kTile128 + 8 * c8);
        __syncthreads();
        store_piece(p, is_x ? a_s : b_s, 8 * c8, rg);
        __syncthreads();
      }
#pragma unroll
      for (int s = 0; s < kStepRows / 32; ++s) {
        v8bf a[4], b[4];
        const int l16 = lane & 15, g = lane >> 4;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ca = wk + 16 * (l16 >> 2) + 4 * i + (l16 & 3);
          a[i] = *reinterpret_cast<const v8bf*>(a_s + lds_piece(ca, 4 * s + g));
          b[i] = *reinterpret_cast<const v8bf*>(b_s + lds_piece(wn + 16 * i + l16, 4 * s + g));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
      }
    }
  }
  const int l16 = lane & 15, g = lane >> 4;
  const bool vec = k % 8 == 0 && ((uintptr_t)dw & 15) == 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = tn * kTile128 + wn + 16 * j + l16;
    const int col = tk * kTile128 + wk + 16 * g;
    if (row >= n) continue;
    uint16_t* dst = dw + ((int64_t)e * n + row) * k + col;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        o[2 * i] = pack_bf16(acc[2 * h + i][j][0], acc[2 * h + i][j][1]);
        o[2 * i + 1] = pack_bf16(acc[2 * h + i][j][2], acc[2 * h + i][j][3]);
      }
      if (vec && col + 8 * h + 8 <= k) {
        *reinterpret_cast<u32x4*>(dst + 8 * h) = o;
      } else {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (col + 8 * h + c < k) dst[8 * h + c] = (uint16_t)(o[c / 2] >> (16 * (c & 1)));
      }
    }
  }
}

}  // namespace

hipError_t launch_wgrad(const Instances& in, const uint8_t* dy, const uint8_t* dys, const uint8_t* x,
                        const uint8_t* xs, int32_t n, int32_t k, uint16_t* dw, int32_t* status, hipStream_t st) {
  const int64_t tiles = (int64_t)in.E * ((n + kTile128 - 1) / kTile128) * ((k + kTile128 - 1) / kTile128);
  if (tiles >= (int64_t)1 << 24) return hipErrorInvalidValue;
  hipLaunchKernelGGL(wgrad_kernel, dim3((unsigned)tiles), dim3(256), 0, st, in, dy, dys, x, xs, n, k, dw, status);
  return hipGetLastError();
}

}  // namespace moe
