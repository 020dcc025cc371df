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
#include <type_traits>

#include "buffers.h"
#include "experts4.h"
#include "fp4_block.h"
#include "instances.h"
#include "product_tiles.h"
#include "store_tile.h"

namespace moe {
namespace {

// The instruction's operand of 16 bytes of 4-bit values; it reads no more.
__device__ __forceinline__ v8i operand4(v4i v) { return v8i{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }
__device__ __forceinline__ v8i operand8(v4i lo, v4i hi) {
  return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}
__device__ __forceinline__ v4i load16b(const uint8_t* p) { return *reinterpret_cast<const v4i*>(p); }

// 16 rows x 64 channels per workgroup; its four waves take every fourth line of
// the long axis each (256 values: two instructions), straight from memory to
// registers, and add their sums in LDS.  Bound by the matrices' bytes: 512 rows of
// 128 experts of 1536 x 2048 41 us, 5.2 TB/s (the scales loaded by every lane for
// itself: 47 us).
constexpr int kRowsS = 16, kChanS = 64;
template <int XB>
__global__ __launch_bounds__(256) void matmul4_rows16_kernel(Instances in, const uint8_t* __restrict__ x,
                                                             const uint8_t* __restrict__ xs,
                                                             const uint8_t* __restrict__ w,
                                                             const uint8_t* __restrict__ ws, int n, int k,
                                                             int64_t tiles, uint16_t* __restrict__ y,
                                                             int32_t* __restrict__ status) {
  __shared__ float part[4][kRowsS][kChanS + 4];
  __shared__ __align__(8) uint32_t scale_s[4][2 * kChanS];
  if (blockIdx.x == 0) check_instances(in, status);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int nb = (k + kCols4 - 1) / kCols4;                             // lines of a 4-bit row
  const int nb8 = (k + kBlk - 1) / kBlk, ns8 = (nb8 + 3) / 4 * 4;      // blocks of an 8-bit row
  const int64_t line = kCols4 / 2;
  const int nct = (n + kChanS - 1) / kChanS;
  uint32_t* const sc_s = scale_s[wave];
  for (int64_t id = blockIdx.x; id < tiles; id += gridDim.x) {
    const int64_t rt = id / nct;
    const int c0 = (int)(id - rt * nct) * kChanS;
    Span sp;
    int64_t r0;
    if (!find_row_tile<kRowsS>(in, rt, &sp, &r0)) continue;  // the same for all waves
    const int64_t row = min(r0 + r, sp.end - 1);
    const uint8_t* wp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = min(c0 + 16 * (r >> 2) + 4 * i + (r & 3), n - 1);
      wp[i] = w + ((int64_t)sp.expert * n + c) * nb * line + 16 * g;
    }
    // the 64 channels' scales, one to a lane: they pass to the lanes that need them through LDS
    const uint8_t* wsp = ws + ((int64_t)sp.expert * nb * n + min(c0 + lane, n - 1)) * 8;
    v4f acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = v4f{0, 0, 0, 0};
    for (int b = wave; b < nb; b += 4) {
      v8i xv[2];
      uint32_t sx[2];
      v4i wv[4][2];
      const u32x2 ws8 = *reinterpret_cast<const u32x2*>(wsp + (int64_t)b * n * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) wv[i][h] = load16b(wp[i] + b * line + 64 * h);
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
      *reinterpret_cast<u32x2*>(sc_s + 2 * lane) = ws8;
      wave_lds_sync();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x2 s = *reinterpret_cast<const u32x2*>(sc_s + 2 * (16 * (r >> 2) + 4 * i + (r & 3)));
#pragma unroll
        for (int h = 0; h < 2; ++h)
          acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand4(wv[i][h]), xv[h], acc[i], kFp4,
                                                                    XB == 4 ? kFp4 : kFp8, 0, (int)(s[h] >> (8 * g)), 0,
                                                                    (int)sx[h]);
      }
      wave_lds_sync();
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

// ---- tiles ---------------------------------------------------------------------
//
// BC channels x BT rows per workgroup of 2 x 2 waves, as the 8-bit products have
// them: both operands' blocks go to LDS by direct loads, a step ahead of the
// products; a step is two halves, and while a half's products run the other
// half's operands are read into a second set of registers; one barrier a step,
// between its halves.
//
// Steps of a line (4 bits, square tiles): 128 bytes of both operands, 256 values; a
// half is two 32x32x64 instructions deep.  Lane group g takes the four blocks of 32
// from 4 g on, so that its scales are one word, which the instruction indexes by
// byte.  A line's scales come to LDS with it: 8 bytes a row, one load of 16 bytes a
// thread.
//
// Steps of half a line (256 x 128 tiles, and all of rows in 8 bits): 128 values, 64
// bytes of 4-bit rows and 128 of 8-bit ones; a half is one instruction deep.  The
// scales of two steps come to LDS together; those of 8-bit rows, one byte a step,
// go to registers four steps at a time.
//
// One dense 8192 cubed reaches 4.2 PFLOP/s in 4 bits and 2.66 with rows in 8 bits.
// Short axes leave the matrix unit idle half of the time: 131072 rows of 128
// experts of 1536 x 2048 in 8 bits take 458 us (1.8 PFLOP/s), and 362 in a timing
// copy that does not store.  A tile's results (9 us beside 26 of products for 16
// steps of 256 x 128) lie under the other workgroup's products only: the wait at
// the next tile's head is for every memory operation, the stores too, and its
// second block goes where the results still pass.  Not the reason: wave priorities
// that set the two workgroups of a CU apart, or favour either phase (454 to 457),
// workgroups that begin up to 16 us later than others (454 to 464), bands of eight
// row tiles (455; 499 where four take 470, 32768 rows of 32 experts of 7168 x 2688).
//
// LDS rows of 128 bytes are placed as piece_at says.  Of rows of
// 64 bytes, four share 256 bytes: piece p of row R lies at place 4 (R % 4) + (p ^
// s(R)), s two bits in which the rows of 16 lanes differ beside R % 4 and that are
// the same in every instruction tile: bits 2 and 3 of R for the rows operand, 2
// and 4 for the channels.
template <bool CHANNELS>
__device__ __forceinline__ int quad_swizzle(int quad) {  // quad = R / 4
  return CHANNELS ? (quad & 1) | ((quad >> 1) & 2) : quad & 3;
}
template <bool CHANNELS>
__device__ __forceinline__ int quad_piece_at(int row, int p) {
  return (row >> 2) * 256 + (((row & 3) << 2) | (p ^ quad_swizzle<CHANNELS>(row >> 2))) * 16;
}

template <int XB, int BC, int BT>
struct TileShape {
  static constexpr int kThreads = 256;
  static constexpr bool kAlone = BC == 256 && BT == 256;               // one workgroup to a CU
  static constexpr bool kLines = XB == 4 && BC == BT;                  // steps of a line
  static constexpr int kWaveC = BC / 2, kWaveT = BT / 2;               // a wave's channels and rows
  static constexpr int kC = kWaveC / 32, kT = kWaveT / 32;             // in instruction tiles
  static constexpr int kBytesC = kLines ? 128 : 64, kBytesT = XB == 4 ? kBytesC : 128;  // of a row, a step
  static constexpr int kDeep = kLines ? 2 : 1;                         // instructions of a half
  static constexpr int kPieces = XB == 4 ? kDeep : 2;                  // of a row's 16-byte pieces, a half
  static constexpr int kPassC = BC * kBytesC / (16 * kThreads), kPassT = BT * kBytesT / (16 * kThreads);
  static constexpr int kScaled = XB == 4 ? BC + BT : BC;               // rows whose scales go to LDS
  static_assert(BC % 128 == 0 && BT % 128 == 0, "whole parts");
};

// A pointer that is the same for all lanes, in scalar registers.
[[maybe_unused]] __device__ __forceinline__ const uint8_t* scalar(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const uint8_t*>((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                                          (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

// acc += c * t with scale byte OC of sc and OT of st.
template <int XB, int OC, int OT>
__device__ __forceinline__ acc16 multiply32(const v8i& c, const v8i& t, const acc16& acc, int sc, int st) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(c, t, acc, kFp4, XB == 4 ? kFp4 : kFp8, OC, sc, OT, st);
}

// Persistent: workgroup b takes every (gridDim.x / 8)-th tile of its XCD's run.
template <int XB, int BC, int BT>
__global__ __launch_bounds__(256, (TileShape<XB, BC, BT>::kAlone ? 1 : 2)) void matmul4_tile_kernel(
    Instances in, const uint8_t* __restrict__ x, const uint8_t* __restrict__ xs, const uint8_t* __restrict__ w,
    const uint8_t* __restrict__ ws, int n, int k, uint16_t* __restrict__ y, int32_t* __restrict__ status) {
#ifdef __HIP_DEVICE_COMPILE__
  using S = TileShape<XB, BC, BT>;
  __shared__ __align__(256) unsigned char c0_s[BC * S::kBytesC];
  __shared__ __align__(256) unsigned char t0_s[BT * S::kBytesT];
  __shared__ __align__(256) unsigned char c1_s[BC * S::kBytesC];
  __shared__ __align__(256) unsigned char t1_s[BT * S::kBytesT];
  __shared__ __align__(16) unsigned char z0_s[8 * S::kScaled];
  __shared__ __align__(16) unsigned char z1_s[S::kLines ? 8 * S::kScaled : 16];
  __shared__ int32_t sums[4];
  extern __shared__ int32_t pre[];  // [cap + 1]
  // where results pass: a place of their own, or (where two workgroups share
  // the CU's LDS) the second stage, whose next block then comes in later
  constexpr bool kOwnPlace = S::kAlone;
  __shared__ __align__(16) unsigned char out_s[kOwnPlace ? 4 * 4096 : 16];
  constexpr bool kFetch = S::kAlone;
  __shared__ uint32_t fetch_s[kFetch ? 4 * 64 : 1];
  if (blockIdx.x == 0) check_instances(in, status);
  const int nct = (n + BC - 1) / BC;
  const int n_inst = instance_count(in);
  const int row_tiles = __builtin_amdgcn_readfirstlane(count_row_tiles(in, BT, pre, sums));
  int tile, last;
  const int slots = gridDim.x >> 3;
  xcd_run(row_tiles * nct, &tile, &last);
  if (tile >= last) return;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 31, g = lane >> 5;
  const int lines = (k + kCols4 - 1) / kCols4;
  const int nb8 = (k + kBlk - 1) / kBlk, ns8 = (nb8 + 3) / 4 * 4;
  const int nb = S::kLines ? lines : nb8;  // steps
  const uint32_t kpc = (uint32_t)lines * (kCols4 / 2), kpt = XB == 4 ? kpc : (uint32_t)nb8 * kBlk;
  // where this thread's pieces come from: the same place of every pass
  const int pair = threadIdx.x >> 4;
  const int place_t = (threadIdx.x & 15) ^ piece_swizzle<false>(pair);
  const int place_c = (threadIdx.x & 15) ^ piece_swizzle<true>(pair);
  const int wc = wave % 2 * S::kWaveC, wt = wave / 2 * S::kWaveT;
  auto locate = [&](int t) { return locate_tile<BC, BT>(in, pre, n_inst, row_tiles, nct, n, t); };
  constexpr std::integral_constant<int, 0> zero{};
  constexpr std::integral_constant<int, 1> one{};
  Tile at;
  uint32_t off_c[S::kPassC], off_t[S::kPassT], xs_off[S::kT], off_f;
  // this wave's part of a line's scales: 128 channels' or (4 bits) rows' (where
  // there are fewer parts than waves, two load the same)
  constexpr int kPartsC = BC / 128, kParts = S::kScaled / 128;
  const int z_part = wave % kParts;
  const bool z_rows = z_part >= kPartsC;
  const int z_at = (z_rows ? z_part - kPartsC : z_part) * 1024;
  const int64_t z_step = 8 * (z_rows ? in.rows : n);
  // the tile's operands and scales, in scalars
  const uint8_t *w_from, *x_from, *z_from;
  uint32_t w_bytes, x_bytes, z_bytes;
  auto set_offsets = [&]() {
    w_from = scalar(w + ((int64_t)at.expert * n + at.c0) * kpc);
    x_from = scalar(x + (int64_t)at.r0 * kpt);
    z_from = scalar(z_rows ? xs + (int64_t)at.r0 * 8 : ws + ((int64_t)at.expert * lines * n + at.c0) * 8);
    w_bytes = __builtin_amdgcn_readfirstlane(at.chans * kpc);
    x_bytes = __builtin_amdgcn_readfirstlane(at.rows * kpt);
    z_bytes = __builtin_amdgcn_readfirstlane(8 * (z_rows ? at.rows : at.chans));
    const int quad_row = (threadIdx.x >> 2) & 3, quad_place = threadIdx.x & 3;
#pragma unroll
    for (int q = 0; q < S::kPassC; ++q)
      off_c[q] = S::kBytesC == 128
                     ? (uint32_t)min(q * 32 + 2 * pair + (place_c >> 3), at.chans - 1) * kpc + 16 * (place_c & 7)
                     : (uint32_t)min(q * 64 + 4 * pair + quad_row, at.chans - 1) * kpc +
                           16 * (quad_place ^ quad_swizzle<true>(pair));
#pragma unroll
    for (int q = 0; q < S::kPassT; ++q)
      off_t[q] = S::kBytesT == 128
                     ? (uint32_t)min(q * 32 + 2 * pair + (place_t >> 3), at.rows - 1) * kpt + 16 * (place_t & 7)
                     : (uint32_t)min(q * 64 + 4 * pair + quad_row, at.rows - 1) * kpt +
                           16 * (quad_place ^ quad_swizzle<false>(pair));
    if (XB == 8) {
#pragma unroll
      for (int j = 0; j < S::kT; ++j) xs_off[j] = (uint32_t)(min(wt + 32 * j + r, at.rows - 1) * ns8);
    }
    // this wave's share of the lines to fetch ahead
    const int part = wave < 2 ? at.rt & 3 : (at.c0 / BC) & 3;
    off_f = (uint32_t)min(4 * (32 * (wave & 1) + (lane & 31)) + part, (wave < 2 ? at.chans : at.rows) - 1) *
            (wave < 2 ? kpc : kpt);
  };
  // Block b's lines into the XCD's L2, a quarter of them per workgroup: those that
  // share an operand take the others.  The bytes read go nowhere.
  auto fetch = [&](int b) {
    if (!kFetch) return;
    asm volatile("" ::: "memory");  // behind the block loads before it
    const auto buf = buffer_of(wave < 2 ? w_from : x_from, wave < 2 ? w_bytes : x_bytes);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_ptr)(fetch_s + wave * 64), 4, off_f,
                                             b * (wave < 2 ? S::kBytesC : S::kBytesT), 0, 0);
  };
  // A step's blocks, and with them the scales of its line (steps of half a line: of
  // the line that begins with an even step).
  auto load = [&](unsigned char* c_s, unsigned char* t_s, unsigned char* z_s, int b, auto odd) {
    const auto w_buf = buffer_of(w_from, w_bytes), x_buf = buffer_of(x_from, x_bytes);
#pragma unroll
    for (int q = 0; q < S::kPassC; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(w_buf, (lds_ptr)(c_s + (q * 256 + wave * 64) * 16), 16, off_c[q],
                                               b * S::kBytesC, 0, 0);
#pragma unroll
    for (int q = 0; q < S::kPassT; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(x_buf, (lds_ptr)(t_s + (q * 256 + wave * 64) * 16), 16, off_t[q],
                                               b * S::kBytesT, 0, 0);
    if constexpr (S::kLines || decltype(odd)::value == 0) {
      const auto z_buf = buffer_of(z_from + (int64_t)(S::kLines ? b : b >> 1) * z_step, z_bytes);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(z_buf, (lds_ptr)(z_s + z_part * 1024), 16, z_at + lane * 16, 0, 0, 0);
    }
  };
  const int perm = 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3);  // channel of the lane's matrix row
  // This lane's scales, of a step or (steps of half a line) of a round's two, shifted
  // so that those it needs are the lowest bytes (8 bits: bytes 0 and 2).
  constexpr int kOf = S::kLines ? 1 : 2;
  struct Scales {
    int c[kOf][S::kC], t[kOf][S::kT];
  };
  auto read_one = [&](const unsigned char* at_z, int* first, int* second) {
    if constexpr (S::kLines) {
      *first = *reinterpret_cast<const int*>(at_z + 4 * g);
    } else {
      typedef uint32_t u32x2_s __attribute__((ext_vector_type(2)));
      const u32x2_s v = *reinterpret_cast<const u32x2_s*>(at_z);
      constexpr int kBits = XB == 4 ? 16 : 8;
      *first = (int)(v[0] >> (kBits * g));
      *second = (int)(v[1] >> (kBits * g));
    }
  };
  auto read_scales = [&](Scales* s, const unsigned char* z_s) {
#pragma unroll
    for (int i = 0; i < S::kC; ++i) read_one(z_s + (wc + 32 * i + perm) * 8, &s->c[0][i], &s->c[kOf - 1][i]);
    if (XB == 4) {
#pragma unroll
      for (int j = 0; j < S::kT; ++j) read_one(z_s + (BC + wt + 32 * j + r) * 8, &s->t[0][j], &s->t[kOf - 1][j]);
    }
  };
  // rows in 8 bits: scales of x, four steps to a word
  int sx_next[S::kT];
  auto load_sx = [&](int b) {
    if (XB == 4) return;
    const auto xs_buf = buffer_of(xs + (int64_t)at.r0 * ns8, (uint32_t)(at.rows * ns8));
#pragma unroll
    for (int j = 0; j < S::kT; ++j) sx_next[j] = (int)__builtin_amdgcn_raw_buffer_load_b32(xs_buf, xs_off[j], b & ~3, 0);
  };
  auto take_sx = [&](Scales* s, int b) {  // those of block b, b even, to the lowest byte
    if (XB == 4) return;
#pragma unroll
    for (int j = 0; j < S::kT; ++j) s->t[0][j] = sx_next[j] >> (8 * (b & 2));
  };
  // LDS places of this lane's pieces in the first tiles; the others lie at
  // constant distances.
  const int first_c = S::kLines ? piece_at<true>(wc + perm, 4 * g) : quad_piece_at<true>(wc + perm, XB == 4 ? 2 * g : g);
  const int first_t = S::kLines ? piece_at<false>(wt + r, 4 * g)
                      : XB == 4 ? quad_piece_at<false>(wt + r, 2 * g)
                                : piece_at<false>(wt + r, g);
  acc16 acc[S::kC][S::kT];
  // 4-bit operands are kept as what they are, 16 bytes: widened ones would hold
  // registers of zeros from one half to the next
  struct Half {
    v4i c[S::kDeep][S::kC], t[S::kPieces][S::kT];
  };
  auto piece = [&](const unsigned char* s, int place) { return *reinterpret_cast<const v4i*>(s + place); };
  auto read = [&](Half* f, const unsigned char* c_s, const unsigned char* t_s, int half) {
    // The places of the other pieces are made from these two each time: kept, they
    // were 16 registers, and others were spilled.
    int at_c = first_c, at_t = first_t;
    asm volatile("" : "+v"(at_c), "+v"(at_t));
#pragma unroll
    for (int m = 0; m < S::kPieces; ++m)
#pragma unroll
      for (int j = 0; j < S::kT; ++j)
        f->t[m][j] = piece(t_s, (at_t ^ (XB == 4 ? 16 * (S::kDeep * half + m) : 64 * half + 32 * m)) + 32 * j * S::kBytesT);
#pragma unroll
    for (int m = 0; m < S::kDeep; ++m)
#pragma unroll
      for (int i = 0; i < S::kC; ++i)
        f->c[m][i] = piece(c_s, (at_c ^ (XB == 4 ? 16 * (S::kDeep * half + m) : 32 * half)) + 32 * i * S::kBytesC);
  };
  // STEP: even or odd of its round; HALF of the step.
  auto multiply = [&](const Half& f, const Scales& s, auto step, auto half) {
    constexpr int kStep = decltype(step)::value, kHalf = decltype(half)::value;
#pragma unroll
    for (int i = 0; i < S::kC; ++i)
#pragma unroll
      for (int j = 0; j < S::kT; ++j) {
        if constexpr (S::kLines) {
          acc[i][j] = multiply32<XB, 2 * kHalf, 2 * kHalf>(operand4(f.c[0][i]), operand4(f.t[0][j]), acc[i][j],
                                                           s.c[0][i], s.t[0][j]);
          acc[i][j] = multiply32<XB, 2 * kHalf + 1, 2 * kHalf + 1>(operand4(f.c[1][i]), operand4(f.t[1][j]),
                                                                   acc[i][j], s.c[0][i], s.t[0][j]);
        } else if constexpr (XB == 4) {
          acc[i][j] = multiply32<XB, kHalf, kHalf>(operand4(f.c[0][i]), operand4(f.t[0][j]), acc[i][j], s.c[kStep][i],
                                                   s.t[kStep][j]);
        } else {
          acc[i][j] = multiply32<XB, 2 * kHalf, kStep>(operand4(f.c[0][i]), operand8(f.t[0][j], f.t[1][j]), acc[i][j],
                                                       s.c[kStep][i], s.t[0][j]);
        }
      }
  };
  // a half's products, with the other half's reads (and LOADS direct loads)
  // spread between them
  constexpr int kProducts = S::kC * S::kT * S::kDeep;
  constexpr int kReads = S::kDeep * S::kC + S::kPieces * S::kT + S::kC + (XB == 4 ? S::kT : 0);
  auto spread = [&](bool loads) {
    if (kFetch && !loads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // fetch
#pragma unroll
    for (int q = 0; q < kProducts; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product
      __builtin_amdgcn_sched_group_barrier(0x100, (kReads + kProducts - 1) / kProducts, 0);
      if (loads) __builtin_amdgcn_sched_group_barrier(0x020, (S::kPassC + S::kPassT + kProducts) / kProducts, 0);
    }
  };
  // turns of 64 channels by 32 rows in a place of their own; or in the second stage,
  // both parts (4 bits: all at once; 8 bits: half the wave's rows at a time) or one
  constexpr int kParts1 = S::kLines ? 2 : BC == 256 && XB == 8 ? 2 : 1;  // parts of the stage
  constexpr int kTI = kOwnPlace ? S::kC / 2 : S::kLines || kParts1 == 2 || XB == 8 ? 1 : 2;
  constexpr int kTJ = kOwnPlace ? S::kT : S::kLines ? 1 : 2;
  constexpr int kOwn = 2 * S::kWaveC * S::kWaveT / (kTI * kTJ);
  unsigned char* const one_part = XB == 4 ? c1_s : t1_s;
  static_assert(kOwnPlace ? kOwn <= 4096
                : kParts1 == 2 ? 2 * kOwn <= BC * S::kBytesC && 2 * kOwn <= BT * S::kBytesT
                               : 4 * kOwn <= (XB == 4 ? BC * S::kBytesC : BT * S::kBytesT), "a turn fits the wave's part");
  unsigned char* own = kOwnPlace      ? out_s + wave * 4096
                       : kParts1 == 2 ? (wave < 2 ? c1_s : t1_s) + (wave & 1) * kOwn
                                      : one_part + wave * kOwn;
  at = locate(tile);
  set_offsets();
  load_sx(0);
  load(c0_s, t0_s, z0_s, 0, zero);
  if (kOwnPlace) load(c1_s, t1_s, z1_s, min(1, nb - 1), one);
  fetch(min(2, nb - 1));
  for (;;) {
    const Tile next = locate(min(tile + slots, last - 1));  // arrives while this tile's products run
#pragma unroll
    for (int i = 0; i < S::kC; ++i)
#pragma unroll
      for (int j = 0; j < S::kT; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
    Half f0, f1;
    Scales s0, s1;  // of even and odd steps, or s0 of a round
    sync_with_loads();
    if (!kOwnPlace) load(c1_s, t1_s, z1_s, min(1, nb - 1), one);
    read(&f0, c0_s, t0_s, 0);
    read_scales(&s0, z0_s);
    // No branch inside a round: past the last block the loads and reads take
    // some block again, which nothing uses.
    for (int b = 0; b + 2 <= nb; b += 2) {
      take_sx(&s0, b);
      fetch(min(b + 3, nb - 1));
      read(&f1, c0_s, t0_s, 1);
      multiply(f0, s0, zero, zero);
      spread(false);
      sync_with_loads<kFetch ? 1 : 0>();
      load(c0_s, t0_s, z0_s, min(b + 2, nb - 1), zero);
      read(&f0, c1_s, t1_s, 0);
      if (S::kLines) read_scales(&s1, z1_s);
      multiply(f1, s0, zero, one);
      spread(true);
      fetch(min(b + 4, nb - 1));
      read(&f1, c1_s, t1_s, 1);
      multiply(f0, S::kLines ? s1 : s0, one, zero);
      spread(false);
      sync_with_loads<kFetch ? 1 : 0>();
      load_sx(min(b + 2, nb - 1));
      load(c1_s, t1_s, z1_s, min(b + 3, nb - 1), one);
      read(&f0, c0_s, t0_s, 0);
      if (S::kLines) {
        read_scales(&s0, z0_s);
        multiply(f1, s1, one, one);
      } else {
        read_scales(&s1, z0_s);
        multiply(f1, s0, one, one);
        s0 = s1;
      }
      spread(true);
    }
    if (nb & 1) {
      take_sx(&s0, nb - 1);
      read(&f1, c0_s, t0_s, 1);
      multiply(f0, s0, zero, zero);
      multiply(f1, s0, zero, one);
    }
    sync_with_loads();  // every wave has its last operands, and no load into LDS is under way
    // The next tile's first blocks come in while this one's results go out.
    const Tile done = at;
    tile += slots;
    const bool more = tile < last;
    if (more) {
      at = next;
      set_offsets();
      load_sx(0);
      load(c0_s, t0_s, z0_s, 0, zero);
      if (kOwnPlace) load(c1_s, t1_s, z1_s, min(1, nb - 1), one);
      fetch(min(2, nb - 1));
    }
    store_wave_tile<kTI, kTJ>(acc, own, y + (int64_t)(done.r0 + wt) * n + done.c0 + wc, n, done.rows - wt,
                              done.chans - wc);
    if (!more) break;
  }
#endif
}

template <int XB, int BC, int BT>
hipError_t launch_tiles(const Instances& in, const uint8_t* x, const uint8_t* xs, const uint8_t* w, const uint8_t* ws,
                        int n, int k, uint16_t* y, int32_t* status, hipStream_t st) {
  const int64_t most = row_tile_ids(in, BT) * ((n + BC - 1) / BC);
  const int64_t resident = TileShape<XB, BC, BT>::kAlone ? 256 : 512;
  hipLaunchKernelGGL((matmul4_tile_kernel<XB, BC, BT>), dim3((unsigned)((most < resident ? most : resident) + 7) / 8 * 8),
                     dim3(256), sizeof(int32_t) * (in.cap + 1), st, in, x, xs, w, ws, n, k, y, status);
  return hipGetLastError();
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

namespace {

constexpr int kCapWide = 1536;  // instances whose tile counts fit the LDS beside 256 x 256 tiles

// The tile of a product, by the mean of rows per expert (the loads themselves are
// on the device).  us in a graph of such launches, in turn with other matrices
// where there are few rows (they are not in the caches then).  "*": what the rule
// takes.
//
// Few rows: bound by the matrices, which the streaming kernel reads straight into
// registers, 16 rows at a time; in it and in 128 x 128 and 256 x 128 tiles:
//   experts     n     k  rows an expert   4 bits                   8 bits
//       128  1536  2048               4    44.6*  48.1   48.2      41.1*  59.8   53.2
//       128  1536  2048              12    55.3   50.5*  49.6      52.8*  60.9   54.1
//        32  5376  7168               8   147.3  126.0* 140.7     125.5* 166.0  153.9
//        32  5376  7168              16   182.5  128.1* 142.5     169.3  168.1  157.3*
//         8  1536  2048              24     8.8*  11.9   16.3       9.4*  14.3   18.8
//         8  3000  4096               6    16.2*  21.0   29.5      15.1*  27.5   34.1
//         8  3000  4096              12    21.6   21.2*  29.8      21.4*  27.9   34.4
//         1  2048  4096              64     7.8   15.5*  22.8       9.4   21.2*  27.9
//         1  8192  8192              32    14.9   35.7*  54.8      17.0   51.0*  63.9
//         1  8192  8192             128    42.8   39.8*  58.1      53.5   58.5*  71.1
// Few matrices leave the tiles to their latency, one workgroup walking a long axis
// alone.  The rule sees that below 2^26 values only: larger single matrices with 7
// (8 bits: 13) to some 100 rows lose up to 2.4 and 3 times.  So do a few hot experts
// among very many idle ones the other way: their mean says streaming, which reads a
// matrix once per 16 rows.
//
// us in 128 x 128, 256 x 128 and 256 x 256 (channels x rows):
//   rows experts     n     k   4 bits                     8 bits
//   2048       1  4096  4096    27.2*   30.4    33.6        39.4*    36.9
//   1024       8  4096  4096    29.7*   34.9    40.0        40.2*    40.5
//   4096       8  1536  2048    18.1*   19.3    24.4        22.2*    21.7
//  16384       8  2048  4096    91.9*  101.1   106.5       153.4    124.6*
//  16384       8  4096  4096   181.7   180.9*  177.7       291.9    235.8*
//  16384       8  4096  4608   198.5   202.4   202.6*      311.7    265.1*
//  32768       8  4096  4608   391.5   391.7   354.9*      612.8    517.1*
//  32768     128  1536  2048   117.9   109.0*  127.5       158.0    133.7*
//  32768      32  7168  2688   535.5   479.1*  506.3       730.3    618.2*
//  32768      32  5376  7168   910.2   877.4   796.1*     1377.8   1180.2*
//   8192       1  8192  8192   305.7   301.0   266.8*      522.3    420.3*
// So rows in 8 bits take 256 x 128 (two workgroups to a CU, one's products under
// the other's results; the LDS keeps up with them) but where that would leave
// channels or CUs idle.  Rows in 4 bits need more of the LDS than the products
// last in any tile but the largest: that one for many tiles and long axes, 256 x
// 128 for very many tiles, which amortize its results.
struct Tile4 {
  int channels, rows;
};
Tile4 matmul4_tile(const Instances& in, int x_bits, int n, int k) {
  const bool small = (double)in.E * n * k < (double)(1 << 26);
  if (in.rows <= (int64_t)(small ? 32 : x_bits == 4 ? 6 : 12) * in.E) return {0, 0};
  const int64_t across = (n + 255) / 256, used = in.rows < in.E ? in.rows : in.E;
  const int blocks = (n + 127) / 128;
  if (blocks == 1 || blocks == 3) return {128, 128};
  if (x_bits == 8) return (in.rows / 128 + used) * across >= 300 ? Tile4{256, 128} : Tile4{128, 128};
  if (k > 4096 && in.rows / 256 * across >= 1024 && in.rows >= (int64_t)192 * in.E && in.cap <= kCapWide)
    return {256, 256};
  return in.rows / 128 * across >= 1536 ? Tile4{256, 128} : Tile4{128, 128};
}

template <int XB>
hipError_t launch(const Instances& in, const uint8_t* x, const uint8_t* xs, const uint8_t* w, const uint8_t* ws, int n,
                  int k, uint16_t* y, int32_t* status, hipStream_t st) {
  const Tile4 tile = matmul4_tile(in, XB, n, k);
  if (tile.channels == 0) return launch_rows16<XB>(in, x, xs, w, ws, n, k, y, status, st);
  if (tile.channels == 128) return launch_tiles<XB, 128, 128>(in, x, xs, w, ws, n, k, y, status, st);
  if constexpr (XB == 4)
    if (tile.rows == 256) return launch_tiles<XB, 256, 256>(in, x, xs, w, ws, n, k, y, status, st);
  return launch_tiles<XB, 256, 128>(in, x, xs, w, ws, n, k, y, status, st);
}

}  // namespace

int64_t matmul4_tiles(const Instances& in, int32_t x_bits, int32_t n, int32_t k) {
  const Tile4 tile = matmul4_tile(in, x_bits, n, k);
  return tile.channels == 0 ? 0 : row_tile_ids(in, tile.rows) * ((n + tile.channels - 1) / tile.channels);
}

hipError_t launch_matmul4(const Instances& in, int32_t x_bits, const uint8_t* x, const uint8_t* xs, const uint8_t* w,
                          const uint8_t* ws, int32_t n, int32_t k, uint16_t* y, int32_t* status, hipStream_t st) {
  return x_bits == 4 ? launch<4>(in, x, xs, w, ws, n, k, y, status, st)
                     : launch<8>(in, x, xs, w, ws, n, k, y, status, st);
}

}  // namespace moe
