// The experts' products on gfx950: y[r][c] = sum_j x[r][j] w[e(r)][c][j] over
// e4m3 values with a power-of-two scale per block of 128.
//
// The 16x16x128 matrix instruction takes a block of 128 of both operands and
// multiplies by both scales itself, so a scale costs no arithmetic here.  The
// matrices are its first operand and the rows its second: a lane's four
// results are then four channels of one row.  Which channel a matrix row of
// the instruction stands for is free; row 4g + j of tile i is channel
// 16g + 4i + j, so four tiles give a lane 16 consecutive channels (32 bytes).
//
// Both 8-bit instructions used here (16x16x128 and 32x32x64) sum in groups of
// eight consecutive values of the long axis: of each product, what lies below
// 2^-13 of the group's largest 2^(exponent of x + exponent of w) is cut off,
// towards zero (a subnormal's exponent is -6).  The groups' sums and the
// accumulator are added in fp32.  A group is off by less than 7 * 2^-13 of that
// power: normally distributed operands give results off by 2^-16 of their root
// mean square, so that bf16's rounding takes 1.2 % of them to the other
// neighbour; quantizing the operands moved them by 2^-5.  Only a sum of small
// products in groups whose large ones cancel loses more.  The bf16 instruction
// would keep all of it at half the rate.
#include "buffers.h"
#include "experts.h"
#include "fp8_block.h"
#include "instances.h"
#include "product_tiles.h"
#include "store_tile.h"

namespace moe {
namespace {

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
  for (int64_t id = blockIdx.x; id < tiles; id += gridDim.x) {
    const int64_t rt = id / nct;
    const int c0 = (int)(id - rt * nct) * kChanS;
    Span sp;
    int64_t r0;
    if (!find_row_tile<kRowsS>(in, rt, &sp, &r0)) continue;  // the same for all waves
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
// BC channels x BT rows per workgroup of WC x WT waves.  Both operands' blocks
// of 128 go to LDS by direct loads, a step (one block of the long axis) ahead
// of the products.  A step is two halves of 64 bytes, one 32x32x64 instruction
// deep; while a half's products run, the other half's operands are read from
// LDS into a second set of registers.  There is one barrier a step, between
// its halves: there the block's reads are all done, so the block after next
// may be loaded over it, and the next block has arrived.
//
// The wave tile decides what LDS has to deliver: 128 x 64 tiles of eight waves
// read 192 KB a step and 64 KB are written, at 128 bytes a cycle as long as
// the products themselves take (2048 cycles), 128 x 128 tiles of four waves read
// 128 KB.
//
// A lane's 16 results are matrix rows 8a + 4h + j, h its half of the wave, of
// one column.  Matrix row 8a + 4h + j stands for channel 16h + 4a + j, so they
// are 16 consecutive channels of one row of y.
template <int BC, int BT, int WC, int WT>
struct TileShape {
  static constexpr int kWaves = WC * WT, kThreads = 64 * kWaves;
  static constexpr int kWaveC = BC / WC, kWaveT = BT / WT;       // a wave's channels and rows
  static constexpr int kC = kWaveC / 32, kT = kWaveT / 32;       // in instruction tiles
  static constexpr int kPassC = BC * kBlk / (16 * kThreads), kPassT = BT * kBlk / (16 * kThreads);
  static_assert(kWaveC % 32 == 0 && kBlk % kWaveC == 0, "a wave's channels share one scale and make whole tiles");
  static_assert(BC * kBlk % (16 * kThreads) == 0 && BT * kBlk % (16 * kThreads) == 0, "whole passes");
};

// Persistent: workgroup b takes every (gridDim.x / 8)-th tile of its XCD's run.
// (A workgroup per tile left the CUs without one for 22 % of the time on short
// axes: 131072 rows, 2048 x 1536: 544 us, and 505 so.)
template <int BC, int BT, int WC, int WT>
__global__ __launch_bounds__((TileShape<BC, BT, WC, WT>::kThreads), BC == 256 ? 1 : 2) void matmul_tile_kernel(
    Instances in, const uint8_t* __restrict__ x, const uint8_t* __restrict__ xs, const uint8_t* __restrict__ w,
    const uint8_t* __restrict__ ws, int n, int k, uint16_t* __restrict__ y, int32_t* __restrict__ status) {
#ifdef __HIP_DEVICE_COMPILE__
  using S = TileShape<BC, BT, WC, WT>;
  __shared__ __align__(256) unsigned char c0_s[BC * kBlk];
  __shared__ __align__(256) unsigned char t0_s[BT * kBlk];
  __shared__ __align__(256) unsigned char c1_s[BC * kBlk];
  __shared__ __align__(256) unsigned char t1_s[BT * kBlk];
  __shared__ int32_t pre[kMaxE + kMaxB + 1];
  __shared__ int32_t sums[4];
  // where results pass: a place of their own, or (where two workgroups share
  // the CU's LDS) the second stage, whose next block then comes in later
  constexpr bool kOwnPlace = BC == 256;
  __shared__ __align__(16) unsigned char out_s[kOwnPlace ? 4 * 4096 : 16];
  constexpr bool kFetch = BC == 256;
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
  const int nb = (k + kBlk - 1) / kBlk, ns = (nb + 3) / 4 * 4;
  const uint32_t kp = (uint32_t)nb * kBlk;
  const int nbn = (n + kBlk - 1) / kBlk;
  // where this thread's pieces come from: the same place of every pass
  constexpr int kRowsPerPass = S::kThreads / 8;
  static_assert(kRowsPerPass % 32 == 0, "the swizzle does not change from pass to pass");
  const int pair = threadIdx.x >> 4;
  const int place_c = (threadIdx.x & 15) ^ piece_swizzle<true>(pair);
  const int place_t = (threadIdx.x & 15) ^ piece_swizzle<false>(pair);
  const int wc = wave % WC * S::kWaveC, wt = wave / WC * S::kWaveT;
  auto locate = [&](int t) { return locate_tile<BC, BT>(in, pre, n_inst, row_tiles, nct, n, t); };
  Tile at;
  uint32_t off_c[S::kPassC], off_t[S::kPassT], xs_off[S::kT], off_f;
  auto set_offsets = [&]() {
#pragma unroll
    for (int q = 0; q < S::kPassC; ++q)
      off_c[q] = (uint32_t)min(q * kRowsPerPass + 2 * pair + (place_c >> 3), at.chans - 1) * kp + 16 * (place_c & 7);
#pragma unroll
    for (int q = 0; q < S::kPassT; ++q)
      off_t[q] = (uint32_t)min(q * kRowsPerPass + 2 * pair + (place_t >> 3), at.rows - 1) * kp + 16 * (place_t & 7);
#pragma unroll
    for (int j = 0; j < S::kT; ++j) xs_off[j] = (uint32_t)(min(wt + 32 * j + r, at.rows - 1) * ns);
    // this wave's share of the lines to fetch ahead
    const int part = wave < 2 ? at.rt & 3 : (at.c0 / BC) & 3;
    off_f = (uint32_t)min(4 * (32 * (wave & 1) + (lane & 31)) + part, (wave < 2 ? at.chans : at.rows) - 1) * kp;
  };
  // Block b's lines into the XCD's L2, a quarter of them per workgroup: those that
  // share an operand take the others.  The workgroups of an XCD ask for a block's
  // lines at about the same time, so without this all of them wait for memory
  // (32768 rows, 32 experts of 5376 x 7168: 1263 -> 1236 us; of 2048 x 1536, 131072
  // rows: 553 -> 524).  The bytes read go nowhere.
  auto fetch = [&](int b) {
    if (!kFetch) return;
    asm volatile("" ::: "memory");  // behind the block loads before it
    const auto buf = wave < 2 ? buffer_of(w + ((int64_t)at.expert * n + at.c0) * kp, (uint32_t)at.chans * kp)
                              : buffer_of(x + (int64_t)at.r0 * kp, (uint32_t)at.rows * kp);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (lds_ptr)(fetch_s + wave * 64), 4, off_f, b * kBlk, 0, 0);
  };
  auto load = [&](unsigned char* c_s, unsigned char* t_s, int b) {
    const auto w_buf = buffer_of(w + ((int64_t)at.expert * n + at.c0) * kp, (uint32_t)at.chans * kp);
    const auto x_buf = buffer_of(x + (int64_t)at.r0 * kp, (uint32_t)at.rows * kp);
#pragma unroll
    for (int q = 0; q < S::kPassC; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(w_buf, (lds_ptr)(c_s + (q * S::kThreads + wave * 64) * 16), 16, off_c[q],
                                               b * kBlk, 0, 0);
#pragma unroll
    for (int q = 0; q < S::kPassT; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(x_buf, (lds_ptr)(t_s + (q * S::kThreads + wave * 64) * 16), 16, off_t[q],
                                               b * kBlk, 0, 0);
  };
  // scales, four blocks to a word: of this lane's row in each instruction
  // tile, and of the wave's channels
  int sx[S::kT], sw, sx_next[S::kT], sw_next;
  auto load_scales = [&](int b) {
    const auto xs_buf = buffer_of(xs + (int64_t)at.r0 * ns, (uint32_t)(at.rows * ns));
    const uint8_t* ws_base = ws + ((int64_t)at.expert * nbn + min((at.c0 + wc) / kBlk, nbn - 1)) * ns;
#pragma unroll
    for (int j = 0; j < S::kT; ++j) sx_next[j] = (int)__builtin_amdgcn_raw_buffer_load_b32(xs_buf, xs_off[j], b & ~3, 0);
    sw_next = *reinterpret_cast<const int*>(ws_base + (b & ~3));
  };
  auto take_scales = [&](int b) {  // those of block b, b even, to the lowest byte
#pragma unroll
    for (int j = 0; j < S::kT; ++j) sx[j] = sx_next[j] >> (8 * (b & 2));
    sw = sw_next >> (8 * (b & 2));
  };
  auto next_scales = [&]() {
#pragma unroll
    for (int j = 0; j < S::kT; ++j) sx[j] >>= 8;
    sw >>= 8;
  };
  // LDS places of this lane's pieces in the first tiles; the others lie at
  // constant distances.  Half h of a block is pieces 4h .. 4h+3, lanes 0..31
  // take the first and third of them, lanes 32..63 the others.
  const int at_c = piece_at<true>(wc + 16 * ((r >> 2) & 1) + 4 * (r >> 3) + (r & 3), g);
  const int at_t = piece_at<false>(wt + r, g);
  acc16 acc[S::kC][S::kT];
  struct Half {
    v8i c[S::kC], t[S::kT];
  };
  auto frag = [&](const unsigned char* s, int at, int half, int add) {
    union {
      v8i v;
      v4i h[2];
    } u;
    u.h[0] = *reinterpret_cast<const v4i*>(s + (at ^ (half * 64)) + add);         // piece 4 half + g
    u.h[1] = *reinterpret_cast<const v4i*>(s + (at ^ (half * 64 + 32)) + add);    // piece 4 half + g + 2
    return u.v;
  };
  auto read = [&](Half* f, const unsigned char* c_s, const unsigned char* t_s, int half) {
#pragma unroll
    for (int j = 0; j < S::kT; ++j) f->t[j] = frag(t_s, at_t, half, 32 * j * kBlk);
#pragma unroll
    for (int i = 0; i < S::kC; ++i) f->c[i] = frag(c_s, at_c, half, 32 * i * kBlk);
  };
  auto multiply = [&](const Half& f) {
#pragma unroll
    for (int i = 0; i < S::kC; ++i)
#pragma unroll
      for (int j = 0; j < S::kT; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f.c[i], f.t[j], acc[i][j], 0, 0, 0, sw, 0, sx[j]);
  };
  // a half's products, with the other half's reads (and LOADS direct loads)
  // spread between them
  constexpr int kProducts = S::kC * S::kT, kReads = 2 * (S::kC + S::kT);
  auto spread = [&](bool loads) {
    if (kFetch && !loads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // fetch
#pragma unroll
    for (int q = 0; q < kProducts; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // a product
      __builtin_amdgcn_sched_group_barrier(0x100, (kReads + kProducts - 1) / kProducts, 0);
      if (loads) __builtin_amdgcn_sched_group_barrier(0x020, (S::kPassC + S::kPassT + kProducts - 1) / kProducts, 0);
    }
  };
  static_assert(S::kWaves == 4 && BC == BT, "four equal parts");
  constexpr int kTI = kOwnPlace ? S::kC / 2 : 1, kTJ = kOwnPlace ? S::kT : 1;  // turns of 64 channels by 32 rows, or one
  constexpr int kOwn = 2 * S::kWaveC * S::kWaveT / (kTI * kTJ);
  static_assert(kOwn <= (kOwnPlace ? 4096 : BC * kBlk / 2), "a turn fits the wave's part");
  unsigned char* own = kOwnPlace ? out_s + wave * 4096 : (wave < 2 ? c1_s : t1_s) + (wave & 1) * kOwn;
  at = locate(tile);
  set_offsets();
  load_scales(0);
  load(c0_s, t0_s, 0);
  if (kOwnPlace) load(c1_s, t1_s, min(1, nb - 1));
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
    sync_with_loads();
    if (!kOwnPlace) load(c1_s, t1_s, min(1, nb - 1));
    read(&f0, c0_s, t0_s, 0);
    // No branch inside a round: past the last block the loads and reads take
    // some block again, which nothing uses.
    for (int b = 0; b + 2 <= nb; b += 2) {
      take_scales(b);
      fetch(min(b + 3, nb - 1));
      read(&f1, c0_s, t0_s, 1);
      multiply(f0);
      spread(false);
      sync_with_loads<kFetch ? 1 : 0>();
      load(c0_s, t0_s, min(b + 2, nb - 1));
      read(&f0, c1_s, t1_s, 0);
      multiply(f1);
      spread(true);
      next_scales();
      fetch(min(b + 4, nb - 1));
      read(&f1, c1_s, t1_s, 1);
      multiply(f0);
      spread(false);
      sync_with_loads<kFetch ? 1 : 0>();
      load_scales(min(b + 2, nb - 1));
      load(c1_s, t1_s, min(b + 3, nb - 1));
      read(&f0, c0_s, t0_s, 0);
      multiply(f1);
      spread(true);
    }
    if (nb & 1) {
      take_scales(nb - 1);
      read(&f1, c0_s, t0_s, 1);
      multiply(f0);
      multiply(f1);
    }
    sync_with_loads();  // every wave has its last operands, and no load into LDS is under way
    // The next tile's first blocks come in while this one's results go out.
    const Tile done = at;
    tile += slots;
    const bool more = tile < last;
    if (more) {
      at = next;
      set_offsets();
      load_scales(0);
      load(c0_s, t0_s, 0);
      if (kOwnPlace) load(c1_s, t1_s, min(1, nb - 1));
      fetch(min(2, nb - 1));
    }
    store_wave_tile<kTI, kTJ>(acc, own, y + (int64_t)(done.r0 + wt) * n + done.c0 + wc, n, done.rows - wt,
                              done.chans - wc);
    if (!more) break;
  }
#endif
}

template <int BC, int BT, int WC, int WT>
hipError_t launch_tiles(const Instances& in, const uint8_t* x, const uint8_t* xs, const uint8_t* w, const uint8_t* ws,
                        int n, int k, uint16_t* y, int32_t* status, hipStream_t st) {
  const int64_t most = row_tile_ids(in, BT) * ((n + BC - 1) / BC), resident = BC == 256 ? 256 : 512;
  hipLaunchKernelGGL((matmul_tile_kernel<BC, BT, WC, WT>), dim3((unsigned)((most < resident ? most : resident) + 7) / 8 * 8),
                     dim3(TileShape<BC, BT, WC, WT>::kThreads), 0, st, in, x, xs, w, ws, n, k, y, status);
  return hipGetLastError();
}

}  // namespace

namespace {

// The tile of a product, 0 for the streaming kernel, by the mean of rows per expert (the loads themselves are on the device):
//   up to 8   bound by the matrices, which the streaming kernel reads straight
//             into registers (128 experts of 1536 x 2048, 512 rows: 75 us
//             against 89 in 128 x 128 tiles; 2048 rows: 99 against 91)
//   large     256 x 256 tiles, where rows fill them and there are two for
//             every CU (32768 rows: 201 us against 209 in 128 x 128 tiles; 4096
//             rows: 131 against 98; 8 experts of 768 x 1024, 8192 rows, 96
//             tiles: 20 against 14)
//   between   128 x 128 tiles, two workgroups to a CU
int matmul_tile(const Instances& in, int n) {
  if (in.rows <= (int64_t)8 * in.E) return 0;
  const bool fills = in.rows / 256 * ((n + 255) / 256) >= 512;
  return in.rows >= (int64_t)192 * in.E && fills ? 256 : 128;
}

}  // namespace

int64_t matmul_tiles(const Instances& in, int32_t n) {
  const int tile = matmul_tile(in, n);
  return tile == 0 ? 0 : row_tile_ids(in, tile) * ((n + tile - 1) / tile);
}

hipError_t launch_matmul(const Instances& in, const uint8_t* x, const uint8_t* xs, const uint8_t* w, const uint8_t* ws,
                         int32_t n, int32_t k, uint16_t* y, int32_t* status, hipStream_t st) {
  const int tile = matmul_tile(in, n);
  if (tile == 256) return launch_tiles<256, 256, 2, 2>(in, x, xs, w, ws, n, k, y, status, st);
  if (tile == 128) return launch_tiles<128, 128, 2, 2>(in, x, xs, w, ws, n, k, y, status, st);
  // without rows one workgroup, which only looks at the plan
  const int64_t tiles = in.rows == 0 ? 0 : row_tile_ids(in, kRowsS) * ((n + kChanS - 1) / kChanS);
  const int64_t grid = tiles < 1 ? 1 : tiles < (1 << 20) ? tiles : (1 << 20);
  hipLaunchKernelGGL(matmul_rows16_kernel, dim3((unsigned)grid), dim3(256), 0, st, in, x, xs, w, ws, n, k, tiles, y,
                     status);
  return hipGetLastError();
}

}  // namespace moe
