// Gradient of the experts' matrices on gfx950:
//   dw[e][c][j] = sum over the rows r of e's instances of dy[r][c] x[r][j]
//
// The sum runs over rows, along which both operands change scale, so the
// scaled 8-bit instruction does not apply; the values are widened to bf16 --
// e4m3 times a power of two is a bf16 value exactly, down to bf16's subnormals
// -- and multiplied by the bf16 instruction.  It wants eight rows of one column
// in a lane, memory has columns next to each other: LDS holds the values as
// they come, rows of 256 columns, and the transposing LDS read hands every 16
// lanes four rows of 16 columns, a column to a lane.  (Transposing in registers
// on the way into LDS took twice the vector instructions, and a fifth longer on
// one dense 8192 cubed.)
//
// 256 x 256 of dw[e] per workgroup of four waves, 128 x 128 each, in steps of
// 64 rows: 2048 cycles of products, and some 4 other instructions to a product
// that a wave issues in its shadow.  A step is four slices of 16 rows.  While a
// slice's products run, the next slice's operands are read, and part of the
// next step's values (loaded a step earlier) is widened and written to the
// other half of LDS.  The last slice runs behind the step's only barrier.
//
// LDS rows are 512 bytes, 16 units of 32 (16 columns).  Unit u of row R lies at
// place u ^ 2 (R % 4): the four rows by 32 columns that 32 lanes read together
// are then eight different units of 256 bytes.  Units with bit 2 set have their
// 16-byte halves exchanged, so that eight lanes' writes, one half each of
// consecutive units, go to eight different places of 128 bytes.
//
// x's columns are the instruction's rows, dy's its columns: a lane's 16
// results are then 16 consecutive columns of x (matrix row 8a + 4h + j stands
// for column 16h + 4a + j, h the lane's half of the wave) in one row of dw.
#include "buffers.h"
#include "experts.h"
#include "fp8_block.h"
#include "instances.h"
#include "store_tile.h"

namespace moe {
namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kStepRows = 64;
constexpr int kThreads = 256;

// COLS columns of either operand per workgroup, half of them per wave.
template <int COLS>
struct GradShape {
  static constexpr int kRowBytes = COLS * 2;
  static constexpr int kSliceBytes = 16 * kRowBytes;
  static constexpr int kOperandBytes = kStepRows * kRowBytes;  // one operand's step in LDS
  static constexpr int kLanesPerRow = COLS / 16;               // threads of a row of the step
  static constexpr int kRows = kStepRows * kLanesPerRow / kThreads;  // rows of a thread's piece
  static constexpr int kWave = COLS / 2, kN = kWave / 32;      // a wave's columns, in instruction tiles
};

// The steps of an expert: 64 rows of one instance at a time, instances in
// order.  Every lane of a wave steps alike, and holds one of the 64 instances
// from i0 on, whose bit is set in `mask` if it is a good one of the expert's.
// Instances that lie one behind the other have T*k rows at most; offsets that
// fall in between may repeat them, thousands of times in a large plan, and the
// steps end at T*k.
struct Steps {
  int n_inst, expert;
  int i0;
  uint64_t mask;
  int begin, end_of;  // this lane's instance
  int row, end;       // the instance under way (rows < 2^31)
  int left;           // rows of instances not begun, at most
};
__device__ __forceinline__ void steps_load(Steps* s, const Instances& in) {
  const int mine = s->i0 + (threadIdx.x & 63), i = min(mine, in.cap - 1);
  s->begin = in.offset[i];
  s->end_of = in.offset[i + 1];
  const int e = in.expert[i];
  s->mask = __ballot(mine < s->n_inst && e == s->expert && s->begin >= 0 && s->begin <= s->end_of &&
                     s->end_of <= in.rows);
}
[[maybe_unused]] __device__ __forceinline__ void steps_begin(Steps* s, const Instances& in, int expert) {
  s->expert = expert;
  s->i0 = 0;
  s->row = s->end = 0;
  s->left = (int)in.rows;
  s->n_inst = instance_count(in);
  steps_load(s, in);
}
// The next step's first row and its rows (0: no more).
[[maybe_unused]] __device__ __forceinline__ void next_step(Steps* s, const Instances& in, int* row, int* rows) {
  while (s->row >= s->end) {
    if (s->mask == 0ull) {
      if (s->i0 + 64 >= s->n_inst) break;
      s->i0 += 64;
      steps_load(s, in);
      continue;
    }
    const int who = __ffsll((unsigned long long)s->mask) - 1;
    s->mask &= s->mask - 1;
    s->row = __builtin_amdgcn_readlane(s->begin, who);
    s->end = s->row + min(s->left, __builtin_amdgcn_readlane(s->end_of, who) - s->row);
    s->left -= s->end - s->row;
  }
  *row = s->row;
  *rows = min(kStepRows, s->end - s->row);
  s->row += kStepRows;
  if (*rows <= 0) {
    *rows = 0;
    s->row = s->end;
  }
}

// A thread's rows of 16 columns as loaded.
template <int ROWS>
struct Piece {
  u32x4 q[ROWS];
  uint32_t s[ROWS];
};

template <int COLS>
__global__ __launch_bounds__(kThreads, COLS == 256 ? 1 : 2) void wgrad_kernel(Instances in, const uint8_t* __restrict__ dy,
                                                       const uint8_t* __restrict__ dys, const uint8_t* __restrict__ x,
                                                       const uint8_t* __restrict__ xs, int n, int k,
                                                       uint16_t* __restrict__ dw, int32_t* __restrict__ status) {
#ifdef __HIP_DEVICE_COMPILE__
  using S = GradShape<COLS>;
  constexpr int kRowBytes = S::kRowBytes, kN = S::kN;
  using Piece = Piece<S::kRows>;
  __shared__ __align__(256) unsigned char x0_s[S::kOperandBytes];
  __shared__ __align__(256) unsigned char y0_s[S::kOperandBytes];
  __shared__ __align__(256) unsigned char x1_s[S::kOperandBytes];
  __shared__ __align__(256) unsigned char y1_s[S::kOperandBytes];
  if (blockIdx.x == 0) check_instances(in, status);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ntk = (k + COLS - 1) / COLS, ntn = (n + COLS - 1) / COLS;
  // Workgroups go to the eight XCDs in turn.  Of 128 consecutive ones, each XCD
  // takes sixteen consecutive tiles, two by eight of an expert, which then share
  // their operands in its L2 (128 experts of 1536 x 2048, 131072 rows: 842 us in
  // plain order, 803 so; the experts' loads by Zipf's law, 922 and 860).
  int tile = blockIdx.x;
  if ((tile | 127) < (int)gridDim.x) tile = (tile & ~127) | ((tile & 7) << 4) | ((tile >> 3) & 15);
  const int e = tile / (ntn * ntk), in_expert = tile - e * ntn * ntk;
  const int band = in_expert / (2 * ntk), in_band = in_expert - band * 2 * ntk;
  const int high = min(2, ntn - 2 * band);
  const int tn = 2 * band + in_band % high, tk = in_band / high;
  const int nbn = (n + kBlk - 1) / kBlk, nbk = (k + kBlk - 1) / kBlk;
  const int nsn = (nbn + 3) / 4 * 4, nsk = (nbk + 3) / 4 * 4;
  const int np = nbn * kBlk, kp = nbk * kBlk;
  // this thread's piece of either operand: columns 16 c16 .. of the tile, rows from row0 of the step
  const int c16 = threadIdx.x % S::kLanesPerRow, row0 = threadIdx.x / S::kLanesPerRow * S::kRows;
  const uint32_t off_x = (uint32_t)(row0 * kp + tk * COLS + 16 * c16), off_y = (uint32_t)(row0 * np + tn * COLS + 16 * c16);
  const uint32_t soff_x = (uint32_t)(row0 * nsk + (tk * COLS + 16 * c16) / kBlk);
  const uint32_t soff_y = (uint32_t)(row0 * nsn + (tn * COLS + 16 * c16) / kBlk);
  // Past the step's rows the descriptor ends: values and scales there are 0.
  // Columns past the row's end are some other row's; nothing stores them.
  auto load = [&](Piece* p, const uint8_t* q, const uint8_t* scale, int row, int rows, int cp, int ns, uint32_t off,
                  uint32_t soff) {
    row = __builtin_amdgcn_readfirstlane(row);  // the same in every lane, which the compiler cannot see
    rows = __builtin_amdgcn_readfirstlane(rows);
    const auto buf = buffer_of(q + (int64_t)row * cp, (uint32_t)rows * (uint32_t)cp);
    const auto sbuf = buffer_of(scale + (int64_t)row * ns, (uint32_t)(rows * ns));
#pragma unroll
    for (int j = 0; j < S::kRows; ++j) {
      p->q[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(buf, off + (uint32_t)(j * cp), 0, 0));
      p->s[j] = __builtin_amdgcn_raw_buffer_load_b8(sbuf, soff + (uint32_t)(j * ns), 0, 0);
    }
  };
  // the first (h = 0) or second half of a piece's rows, widened, to LDS
  const int swap = (c16 >> 2) & 1;
  auto widen = [&](const Piece& p, unsigned char* lds, int h) {
#pragma unroll
    for (int j = h * S::kRows / 2; j < (h + 1) * S::kRows / 2; ++j) {
      // the conversion takes the exponent alone: byte 0 is 2^-127, and 255 gives NaN for the whole block
      const float f = __uint_as_float(p.s[j] << 23);
      u32x4 w[2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i / 2][2 * (i & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p.q[j][i], f, false));
        w[i / 2][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p.q[j][i], f, true));
      }
      unsigned char* row = lds + (row0 + j) * kRowBytes + (c16 ^ (2 * ((row0 + j) & 3))) * 32;
      *reinterpret_cast<u32x4*>(row + 16 * swap) = w[0];
      *reinterpret_cast<u32x4*>(row + 16 - 16 * swap) = w[1];
    }
  };
  const int wk = (wave & 1) * S::kWave, wn = (wave >> 1) * S::kWave;
  const int g = lane >> 5;
  // Reads: lane 4t + q of 16 lends the address of row t, four columns, which
  // go to lanes 4q .. 4q + 3.  dy's columns stay in order; x's are taken so that
  // matrix row 8a + 4h + j is column 16h + 4a + j.
  const int t = (lane >> 2) & 3, q = lane & 3, half = (lane >> 4) & 1;
  int at_x[kN], at_y[kN];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int row = (8 * g + t) * kRowBytes;
    const int ux = (wk + 32 * i) / 16 + (q & 1), uy = (wn + 32 * i) / 16 + half;
    at_x[i] = row + (ux ^ (2 * t)) * 32 + (((8 * half + 4 * (q >> 1)) * 2) ^ (16 * ((ux >> 2) & 1)));
    at_y[i] = row + (uy ^ (2 * t)) * 32 + ((4 * q * 2) ^ (16 * ((uy >> 2) & 1)));
  }
  struct Slice {
    v8bf x[kN], y[kN];
  };
  auto read8 = [&](const unsigned char* s) {  // rows 8g .. 8g + 7 of the slice, this lane's column
    typedef short v4s __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4s* lds4;
    union {
      v8bf v;
      v4s h[2];
    } u;
    u.h[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)s);
    u.h[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(s + 4 * kRowBytes));
    return u.v;
  };
  auto read = [&](Slice* f, const unsigned char* x_s, const unsigned char* y_s, int slice) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      f->x[i] = read8(x_s + at_x[i] + slice * S::kSliceBytes);
      f->y[i] = read8(y_s + at_y[i] + slice * S::kSliceBytes);
    }
  };
  acc16 acc[kN][kN];
#pragma unroll
  for (int i = 0; i < kN; ++i)
#pragma unroll
    for (int j = 0; j < kN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
  auto multiply = [&](const Slice& f) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int j = 0; j < kN; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.x[i], f.y[j], acc[i][j], 0, 0, 0);
  };
  // a slice's products with the other work between them: a read each, the
  // writes and loads spread out, vector instructions
  auto spread = [&](bool loads) {
#pragma unroll
    for (int i = 0; i < (kN == 4 ? 16 : 0); ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 2, 0);
      if (i % 3 == 2) __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
      if (loads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
  };
  Steps steps;
  steps_begin(&steps, in, e);
  int row, rows;
  next_step(&steps, in, &row, &rows);
  if (rows > 0) {
    struct Pieces {
      Piece x, y;
    };
    auto load_step = [&](Pieces* p) {
      load(&p->x, x, xs, row, rows, kp, nsk, off_x, soff_x);
      load(&p->y, dy, dys, row, rows, np, nsn, off_y, soff_y);
    };
    Pieces pa, pb;
    load_step(&pa);
    next_step(&steps, in, &row, &rows);
    load_step(&pb);
    int have = rows;  // rows of the step whose values are in registers
    widen(pa.x, x0_s, 0);
    widen(pa.x, x0_s, 1);
    widen(pa.y, y0_s, 0);
    widen(pa.y, y0_s, 1);
    __syncthreads();
    Slice f0, f1;
    read(&f0, x0_s, y0_s, 0);
    // One step from (x_s, y_s); the next one's values, in p, go to (xn_s,
    // yn_s), and those of the step after are loaded to pn.  Past the last step
    // the values are zeros.  Returns the rows that then lie in (xn_s, yn_s).
    auto step = [&](unsigned char* x_s, unsigned char* y_s, unsigned char* xn_s, unsigned char* yn_s, const Pieces& p,
                    Pieces* pn) {
      const int ready = have;
      if (have > 0) next_step(&steps, in, &row, &rows);
      load_step(pn);
      read(&f1, x_s, y_s, 1);
      widen(p.x, xn_s, 0);
      multiply(f0);
      spread(true);
      read(&f0, x_s, y_s, 2);
      widen(p.x, xn_s, 1);
      multiply(f1);
      spread(false);
      read(&f1, x_s, y_s, 3);
      widen(p.y, yn_s, 0);
      widen(p.y, yn_s, 1);
      multiply(f0);
      spread(false);
      __syncthreads();
      read(&f0, xn_s, yn_s, 0);
      multiply(f1);
      spread(false);
      have = rows;
      return ready;
    };
    // two steps a round, without a way out between them (it would have the
    // sums copied); behind an odd number of steps the second adds zeros
    int left;
    do {
      step(x0_s, y0_s, x1_s, y1_s, pb, &pa);
      left = step(x1_s, y1_s, x0_s, y0_s, pa, &pb);
    } while (left > 0);
  }
  __syncthreads();  // every wave has its last operands: LDS is free
  unsigned char* own = wave == 0 ? x0_s : wave == 1 ? y0_s : wave == 2 ? x1_s : y1_s;
  const int c = tn * COLS + wn, col = tk * COLS + wk;
  store_wave_tile<1, 1>(acc, own, dw + ((int64_t)e * n + c) * k + col, k, n - c, k - col);
#endif
}

}  // namespace

namespace {

int64_t grad_tiles(const Instances& in, int32_t n, int32_t k, int cols) {
  return (int64_t)in.E * ((n + cols - 1) / cols) * ((k + cols - 1) / cols);
}
bool large_grad_tiles(const Instances& in, int32_t n, int32_t k) { return grad_tiles(in, n, k, 256) >= 512; }

}  // namespace

int64_t wgrad_tiles(const Instances& in, int32_t n, int32_t k) {
  return grad_tiles(in, n, k, large_grad_tiles(in, n, k) ? 256 : 128);
}

template <int COLS>
hipError_t launch_grad_tiles(const Instances& in, const uint8_t* dy, const uint8_t* dys, const uint8_t* x,
                             const uint8_t* xs, int32_t n, int32_t k, uint16_t* dw, int32_t* status, hipStream_t st) {
  hipLaunchKernelGGL((wgrad_kernel<COLS>), dim3((unsigned)grad_tiles(in, n, k, COLS)), dim3(kThreads), 0, st, in, dy, dys, x, xs, n, k, dw,
                     status);
  return hipGetLastError();
}

hipError_t launch_wgrad(const Instances& in, const uint8_t* dy, const uint8_t* dys, const uint8_t* x,
                        const uint8_t* xs, int32_t n, int32_t k, uint16_t* dw, int32_t* status, hipStream_t st) {
  // 256 x 256 where there are two for every CU (128 experts of 1536 x 2048,
  // 32768 rows: 374 us against 416 in 128 x 128); else 128 x 128, two
  // workgroups to a CU (8 experts of 768 x 1024, 8192 rows: 25 us against 32)
  return large_grad_tiles(in, n, k) ? launch_grad_tiles<256>(in, dy, dys, x, xs, n, k, dw, status, st)
                                    : launch_grad_tiles<128>(in, dy, dys, x, xs, n, k, dw, status, st);
}

}  // namespace moe
