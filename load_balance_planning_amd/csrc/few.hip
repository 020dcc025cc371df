// A layer's experts for at most 64 tokens in two launches on gfx950.
//
//   up    (g, u) = W1[e] Q(hidden[t]),  a = Q(g sigmoid(g) u)   per slot (t, j)
//   down  out[t] = sum_j weight[t][j] W2[e_tj] a_tj
//
// Q rounds to e4m3 with a power-of-two scale per 32.  What bounds both launches
// is the matrices' bytes, once each, so the tokens of an expert are one operand
// of the matrix instruction (its columns, mostly empty) and an expert's rows go
// straight from memory to registers.  With a scale per 32 of the summed axis a
// workgroup of 32 channels quantizes its activations by itself, and a lane holds
// whole blocks.
//
// Which tokens an expert has is found by every workgroup from the top-k (at most
// 2048 numbers).
#include "buffers.h"
#include "experts4.h"
#include "fp4_block.h"
#include "lane_group.h"
#include "row_load.h"

namespace moe {
namespace {

typedef float float2_ __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// What there is to multiply: entries of an expert and up to 16 of its slots t * k +
// j (tokens ascending; one operand of the instruction).  In dynamic LDS: masks u64
// [E] of tokens, then per entry its first place in the list of slots, int32 [cap +
// 1], and its expert, uint16 [cap], then the list, uint16 [T * k], and where each
// expert's slots begin there, uint16 [E].  Experts ascend.
constexpr int kCols = 16;
struct Chosen {
  uint64_t* mask;
  int32_t* first;
  uint16_t* expert;
  uint16_t* slot;
  int n;
  struct One {
    int expert, first, count;
  };
  __device__ __forceinline__ One one(int a) const {
    One o;
    o.expert = __builtin_amdgcn_readfirstlane(expert[a]);
    o.first = __builtin_amdgcn_readfirstlane(first[a]);
    o.count = __builtin_amdgcn_readfirstlane(first[a + 1]) - o.first;
    return o;
  }
  // slot `which` of an entry, -1 if there are no more
  __device__ __forceinline__ int slot_of(const One& o, int which) const {
    return which < o.count ? slot[o.first + which] : -1;
  }
};
// Entries at most: an expert's first, and one more for every 16 slots.
__host__ __device__ inline int chosen_cap(const Dims& d) {
  const int slots = d.T * d.k;
  return (d.E < slots ? d.E : slots) + (d.T > kCols ? slots / kCols : 0);
}
__host__ __device__ inline size_t chosen_lds(const Dims& d) {
  return ((size_t)10 * d.E + 4 * (chosen_cap(d) + 1) + 2 * chosen_cap(d) + 2 * d.T * d.k + 15) / 16 * 16;
}

template <int THREADS>
__device__ __forceinline__ Chosen collect_lds(const Dims& d, const int32_t* __restrict__ topk, unsigned char* lds,
                                              int32_t* status) {
  const int slots = d.T * d.k, cap = chosen_cap(d), lane = threadIdx.x & 63;
  Chosen c;
  c.mask = reinterpret_cast<uint64_t*>(lds);
  c.first = reinterpret_cast<int32_t*>(lds + 8 * d.E);
  c.expert = reinterpret_cast<uint16_t*>(c.first + cap + 1);
  c.slot = c.expert + cap;
  uint16_t* const where = c.slot + slots;
  __shared__ int repeated;
  constexpr int kPer = 2048 / THREADS;  // slots of a thread at most
  int e[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = threadIdx.x + i * THREADS;
    e[i] = s < slots ? topk[s] : -1;
  }
  for (int i = threadIdx.x; i < d.E; i += THREADS) c.mask[i] = 0ull;
  if (threadIdx.x == 0) repeated = 0;
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
    if ((atomicOr(reinterpret_cast<unsigned long long*>(c.mask + e[i]), (unsigned long long)bit) & bit) != 0ull) {
      bad = true;
      repeated = 1;
    }
  }
  if (bad && status && blockIdx.x == 0) atomicOr(status, MOE_STATUS_BAD_TOPK);
  __syncthreads();
  if (repeated) {  // the first of a token's slots with an expert is the one that counts
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = threadIdx.x + i * THREADS;
      if (s >= slots) continue;
      for (int before = s / d.k * d.k; before < s; ++before)
        if (topk[before] == e[i]) e[i] = -1;
    }
  }
  // Entries and their slots, counted together, 16 bits each.  Every wave goes over all
  // experts and writes the same, so that none waits for another.
  const int per = (d.E + 63) / 64, from = lane * per;
  int mine = 0;
  for (int i = from; i < min(from + per, d.E); ++i) {
    const int m = __popcll(c.mask[i]);
    mine += (m + kCols - 1) / kCols * 0x10000 + m;
  }
  const int incl = group_incl_scan<64>(mine, lane), all = __builtin_amdgcn_readlane(incl, 63);
  int before = incl - mine;
  c.n = all >> 16;
  for (int i = from; i < min(from + per, d.E); ++i) {
    where[i] = (uint16_t)before;
    for (int m = __popcll(c.mask[i]); m > 0; m -= kCols) {
      c.expert[before >> 16] = (uint16_t)i;
      c.first[before >> 16] = before & 0xffff;
      before += 0x10000 + min(m, kCols);
    }
  }
  if (lane == 0) c.first[c.n] = all & 0xffff;
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = threadIdx.x + i * THREADS;
    if (s >= slots || (unsigned)e[i] >= (unsigned)d.E) continue;
    c.slot[where[e[i]] + __popcll(c.mask[e[i]] & ((1ull << (s / d.k)) - 1ull))] = (uint16_t)s;
  }
  __syncthreads();
  return c;
}

// The same where there are at most 64 slots, one to a lane, in every wave's
// registers: slots of an expert are a mask in LDS (u64 [E]), and that is all.
// Entries in the order of their first slots.  (A token: 0.8 us less in the first
// launch and 0.5 in the second than by lists; 64 slots: 0 and 0.9.)
struct ChosenSmall {
  int e;      // of the lane's slot; -1: none
  int order;  // of the slot among its expert's
  int rank;   // of the slot's entry where it is the entry's first; -1 elsewhere
  int n;
  struct One {
    int expert, count, list;  // list: lane i has the entry's slot i
  };
  __device__ __forceinline__ One one(int a) const {
    const int lane = threadIdx.x & 63, lead = (int)__builtin_ctzll(__ballot(rank == a));
    One o;
    o.expert = __builtin_amdgcn_readlane(e, lead);
    const bool mine = e == o.expert && order / kCols == __builtin_amdgcn_readlane(order, lead) / kCols;
    const uint64_t set = __ballot(mine), below = (1ull << lane) - 1ull;
    o.count = __popcll(set);
    // other slots go behind, so that every lane has one place
    const int place = mine ? __popcll(set & below) : o.count + __popcll(~set & below);
    o.list = __builtin_amdgcn_ds_permute(4 * place, lane);
    return o;
  }
  __device__ __forceinline__ int slot_of(const One& o, int which) const {
    const int s = __builtin_amdgcn_ds_bpermute(4 * (which & 63), o.list);
    return which < o.count ? s : -1;
  }
};
template <int THREADS>
__device__ __forceinline__ ChosenSmall collect_small(const Dims& d, const int32_t* __restrict__ topk,
                                                     unsigned char* lds, int32_t* status) {
  const int slots = d.T * d.k, lane = threadIdx.x & 63;
  unsigned long long* mask = reinterpret_cast<unsigned long long*>(lds);
  ChosenSmall c;
  c.e = lane < slots ? topk[lane] : -1;
  for (int i = threadIdx.x; i < d.E; i += THREADS) mask[i] = 0ull;
  __syncthreads();
  const bool good = (unsigned)c.e < (unsigned)d.E;
  bool bad = lane < slots && !good;
  if (!good) c.e = -1;
  uint64_t same = 0ull;
  if (good) {  // every wave sets the same bits, and sees its own at least
    atomicOr(mask + c.e, 1ull << lane);
    same = *reinterpret_cast<volatile unsigned long long*>(mask + c.e);
  }
  // an earlier slot of the same token with the same expert is the one that counts
  const uint64_t earlier = ((1ull << lane) - 1ull) & ~((1ull << (lane / d.k * d.k)) - 1ull);
  const uint64_t repeated = __ballot((same & earlier) != 0ull);
  if (repeated >> lane & 1ull) {
    bad = true;
    c.e = -1;
  }
  same &= ~repeated;
  c.order = __popcll(same & ((1ull << lane) - 1ull));
  const uint64_t leader = __ballot(c.e >= 0 && c.order % kCols == 0);
  c.n = __popcll(leader);
  c.rank = leader >> lane & 1ull ? __popcll(leader & ((1ull << lane) - 1ull)) : -1;
  if (status && blockIdx.x == 0 && threadIdx.x < 64 && __ballot(bad) != 0ull && lane == 0)
    atomicOr(status, MOE_STATUS_BAD_TOPK);
  return c;
}
template <bool SMALL, int THREADS>
__device__ __forceinline__ auto collect(const Dims& d, const int32_t* __restrict__ topk, unsigned char* lds,
                                        int32_t* status) {
  if constexpr (SMALL)
    return collect_small<THREADS>(d, topk, lds, status);
  else
    return collect_lds<THREADS>(d, topk, lds, status);
}

// Eight values of a row from column c on; zeros from column `cols` on.
[[maybe_unused]] __device__ __forceinline__ u32x4 load8_row(const uint16_t* __restrict__ x, int64_t row_at, int c,
                                                            int cols, int64_t total) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (c >= cols) return v;
  v = row_at + c + 8 <= total ? (u32x4) * reinterpret_cast<const u32x4_any*>(x + row_at + c)
                              : load8_edge(x, row_at + c, total);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] &= (c + 2 * i < cols ? 0xffffu : 0u) | (c + 2 * i + 1 < cols ? 0xffff0000u : 0u);
  return v;
}

// What eight values of a row become by rounding to e4m3 with a scale per 32, as
// bf16 again: the four lanes of an aligned quad hold a block.  All NaN where that
// holds a NaN or an infinity.
[[maybe_unused]] __device__ __forceinline__ u32x4 round8(u32x4 x) {
  typedef short s16x2 __attribute__((ext_vector_type(2)));
  uint32_t top = x[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 4; ++i) top = pk_max(top, x[i] & 0x7fff7fffu);
  top = max(top << 16, top & 0xffff0000u);
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xf, 0xf, false));
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xf, 0xf, false));
  const float by = __uint_as_float(scale_byte(top) << 23);  // the conversions take its exponent, 255 for NaN
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    s16x2 q = {0, 0};
    q = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(q, two_bf16(x[i]), by, false);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(q, two_bf16(x[i + 1]), by, true);
    const uint32_t p = __builtin_bit_cast(uint32_t, q);
    o[i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p, by, false));
    o[i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(p, by, true));
  }
  return o;
}

// Only the device pass knows buffers.
#ifdef __HIP_DEVICE_COMPILE__
// Rows [row0, row0 + rows) of an expert's matrix of `all` rows and `cols` columns
// in WB bits, and their scales to the end of the expert's table.  A lane's row is
// a 32-bit offset; rows past the end read as zeros.
template <int WB>
struct Matrix {
  __amdgpu_buffer_rsrc_t q, s;
  uint32_t row_bytes, s_step;  // s_step: scale bytes from line to line (4 bits), from 128 rows to the next (8 bits)
};
template <int WB>
__device__ __forceinline__ Matrix<WB> matrix_rows(const uint8_t* __restrict__ w, const uint8_t* __restrict__ ws,
                                                  int expert, int all, int row0, int rows, int cols) {
  Matrix<WB> m;
  if (WB == 4) {
    const int nb = (cols + kCols4 - 1) / kCols4;
    m.row_bytes = (uint32_t)nb * (kCols4 / 2);
    m.s_step = (uint32_t)all * 8;
    m.s = buffer_of(ws + ((int64_t)expert * nb * all + row0) * 8, (uint32_t)nb * m.s_step - 8 * row0);
  } else {
    const int nb = (cols + kBlk - 1) / kBlk;
    m.row_bytes = (uint32_t)nb * kBlk;
    m.s_step = (uint32_t)(nb + 3) / 4 * 4;
    const uint32_t table = (uint32_t)((all + kBlk - 1) / kBlk) * m.s_step;
    m.s = buffer_of(ws + (int64_t)expert * table, table);
  }
  m.q = buffer_of(w + ((int64_t)expert * all + row0) * m.row_bytes, (uint32_t)rows * m.row_bytes);
  return m;
}
__device__ __forceinline__ v4i load16b(__amdgpu_buffer_rsrc_t b, uint32_t at, uint32_t line) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(b, (int)at, (int)line, 0));
}

// How many blocks of 128 columns a step has: 4 bits: a line of 256 columns, 8
// bits: 128 columns.
constexpr int halves(int bits) { return bits == 4 ? 2 : 1; }

// acc += values * x over a step's half: lane (r, g) has row r's columns, 4 bits: 32
// g .. + 31 of the half; 8 bits: 16 g .. + 15 and 64 + 16 g .. + 15.  s: their scale.
template <int WB>
__device__ __forceinline__ v4f multiply(u32x4 q0, u32x4 q1, uint32_t s, const u32x4* x, v4f acc) {
  const float by = __uint_as_float(s << 23);  // the conversions take its exponent, 255 for NaN
#pragma unroll
  for (int p = 0; p < 4; ++p) {  // eight columns
    union {
      bf16x2 two[4];
      bf16x8 all;
    } a, c;
#pragma unroll
    for (int i = 0; i < 4; ++i) c.two[i] = two_bf16(x[p][i]);
    if constexpr (WB == 4) {
      const uint32_t q = q0[p];
      a.two[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, by, 0);
      a.two[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, by, 1);
      a.two[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, by, 2);
      a.two[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, by, 3);
    } else {
      const uint32_t lo = p < 2 ? q0[2 * p] : q1[2 * p - 4], hi = p < 2 ? q0[2 * p + 1] : q1[2 * p - 3];
      a.two[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, by, false);
      a.two[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, by, true);
      a.two[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, by, false);
      a.two[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, by, true);
    }
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.all, c.all, acc, 0, 0, 0);
  }
  return acc;
}
#endif

// 32 gate and 32 up channels of one entry per unit; the waves take steps of the
// long axis in turn and add their sums in LDS.
//
// The products are the bf16 instruction's, of values that are exact in bf16: the
// 8-bit one cuts products off at 2^-13 of a neighbour's, and sums so far off
// (2^-16 of their root mean square) round some activations to the other e4m3
// neighbour, 6 % of their value away.
//
// A step's loads are few, so that the cache's ports keep up with memory: the
// matrices' lines; one load for the scales of all 64 rows; and of the tokens' rows
// what there is of them, the lanes side by side (two tokens a load).  Scales and
// rows (rounded) pass through LDS, the wave's own part of it, to the lanes that
// multiply.  Loaded by those lanes each for itself, scales took 8 % and rows 14 %
// of the time (8 tokens, 29 experts of 2 x 2688 x 7168: 132 us then, 107 now, 5.6
// TB/s of matrices).  Workgroups that are all resident, two to a CU, choose experts
// once: 1024 of them take 48.6 us where 512 take 44.9 (64 tokens, 128 experts of 2 x
// 768 x 2048, 4.4 TB/s; with long axes 106 and 107).  Such short axes lose to what a
// unit costs beside its steps, two a wave; the next unit's loads under a unit's last
// products too, or as many units to every workgroup, were slower (48.5, 48.2).
constexpr int kChan = 32;
template <int WB, int WAVES, bool SMALL>
__global__ __launch_bounds__(64 * WAVES, 2) void experts_up_kernel(
    Dims d, const uint16_t* __restrict__ hidden, const int32_t* __restrict__ topk, const uint8_t* __restrict__ w,
    const uint8_t* __restrict__ ws, int f, uint8_t* __restrict__ act, uint8_t* __restrict__ act_scale,
    uint32_t* __restrict__ counter, int counters, int32_t* __restrict__ status) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int kHalves = halves(WB), kChunks = 16 * kHalves;   // chunks of 8 columns of a token's step
  constexpr int kAtOnce = 64 / kChunks, kSets = kCols / kAtOnce;  // tokens of a load, loads of 16 tokens
  constexpr int kPartRow = 2 * kChan + 4, kRows = kCols * kChunks * 16;
  extern __shared__ __align__(16) unsigned char lds[];
  constexpr int kTurns = WAVES == 4 ? 2 : 1;  // places of sums: with two a unit needs one barrier
  __shared__ __align__(16) unsigned char own_s[WAVES][kRows];  // a wave's rows of a step
  __shared__ __align__(16) float part_s[kTurns][WAVES][kCols * kPartRow];
  __shared__ __align__(16) uint32_t scale_s[WAVES][64 * kHalves];
  if (blockIdx.x == 0)  // for the launch behind this one
    for (int i = threadIdx.x; i < counters; i += 64 * WAVES) counter[i] = 0u;
  const auto ch = collect<SMALL, 64 * WAVES>(d, topk, lds, status);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int chunks = (f + kChan - 1) / kChan, units = ch.n * chunks;
  const int fp = (int)padded_cols4(f), steps = (d.H + kHalves * kBlk - 1) / (kHalves * kBlk);
  const int whole = d.H / (kHalves * kBlk);  // steps before a row's end
  const int64_t total = (int64_t)d.T * d.H;
  unsigned char* const rows_s = own_s[wave];
  uint32_t* const sc_s = scale_s[wave];
  // A unit: entry a's 32 channels from c0 on; this lane's rows of the matrices, the
  // one of the 64 whose scales it loads, and the elements of the tokens' rows.
  struct Unit {
    decltype(ch.one(0)) one;
    Matrix<WB> gate, up;
    int chunk;
    uint32_t at, at_16, s_at, from[kSets];
  };
  auto begin = [&](int a, int chunk) {
    Unit u;
    u.one = ch.one(a);
    u.chunk = chunk;
    const int c0 = chunk * kChan, valid = min(kChan, f - c0);
    u.gate = matrix_rows<WB>(w, ws, u.one.expert, 2 * f, c0, valid, d.H);
    u.up = matrix_rows<WB>(w, ws, u.one.expert, 2 * f, f + c0, valid, d.H);
    u.at = (uint32_t)r * u.gate.row_bytes + 16 * g;
    u.at_16 = u.at + 16 * u.gate.row_bytes;
    const int s_row = min(lane & 31, valid - 1) + (lane >= 32 ? f : 0);
    u.s_at = WB == 4 ? (uint32_t)s_row * 8 : (uint32_t)((c0 + s_row) / kBlk) * u.gate.s_step;
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
      if (i * kAtOnce >= u.one.count) break;
      const int s = max(ch.slot_of(u.one, i * kAtOnce + lane / kChunks), 0);
      u.from[i] = (uint32_t)(s / d.k) * d.H + 8 * (lane % kChunks);
    }
    return u;
  };
  struct Step {
    u32x4 q[4][2];
    u32x2 s;
    u32x4 x[kSets];
  };
  auto load = [&](Step* o, const Unit& u, int b) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        o->q[i][p] = __builtin_bit_cast(
            u32x4, load16b(i < 2 ? u.gate.q : u.up.q, (i & 1 ? u.at_16 : u.at) + 64 * p, b * kBlk));
    if constexpr (WB == 4)
      o->s = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_raw_buffer_load_b64(u.gate.s, (int)u.s_at, b * (int)u.gate.s_step, 0));
    else
      o->s[0] = __builtin_amdgcn_raw_buffer_load_b8(u.gate.s, (int)u.s_at, b, 0);
    if (b >= whole) return;
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
      if (i * kAtOnce >= u.one.count) break;
      o->x[i] = *reinterpret_cast<const u32x4_any*>(hidden + u.from[i] + b * kHalves * kBlk);
    }
  };
  // unit = a * chunks + chunk, stepped without divisions
  const int step_a = (int)gridDim.x / chunks, step_c = (int)gridDim.x - step_a * chunks;
  int a = (int)blockIdx.x / chunks, unit = blockIdx.x;
  if (unit >= units) return;
  Unit u = begin(a, unit - a * chunks);
  Step next;
  if (wave < steps) load(&next, u, wave);
  for (int turn = 0;; ++turn) {
    v4f acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = v4f{0, 0, 0, 0};
    for (int b = wave; b < steps; b += WAVES) {
      // rows and scales to LDS: token t's chunk c lies at c ^ t, so that 16 tokens' lie apart
      auto put = [&](int i, const u32x4& v) {
        const int t = i * kAtOnce + lane / kChunks;
        *reinterpret_cast<u32x4*>(rows_s + (t * kChunks + ((lane % kChunks) ^ t)) * 16) = round8(v);
      };
      if (b < whole) {
#pragma unroll
        for (int i = 0; i < kSets; ++i) {
          if (i * kAtOnce >= u.one.count) break;
          put(i, next.x[i]);
        }
      } else {  // the rows' end, loaded here: its edges would take the registers of every step
#pragma unroll 1
        for (int i = 0; i * kAtOnce < u.one.count; ++i) {
          const int64_t row_at = (int64_t)(max(ch.slot_of(u.one, i * kAtOnce + lane / kChunks), 0) / d.k) * d.H;
          put(i, load8_row(hidden, row_at, b * kHalves * kBlk + 8 * (lane % kChunks), d.H, total));
        }
      }
      if (WB == 4)
        *reinterpret_cast<u32x2*>(sc_s + 2 * lane) = next.s;
      else
        sc_s[lane] = next.s[0];
      u32x4 q[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int p = 0; p < 2; ++p) q[i][p] = next.q[i][p];
      wave_lds_sync();
      if (b + WAVES < steps) load(&next, u, b + WAVES);
      u32x2 s[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (WB == 4)
          s[i] = *reinterpret_cast<const u32x2*>(sc_s + 2 * (16 * i + r));
        else
          s[i][0] = sc_s[16 * i + r];
      }
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        u32x4 x[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int c = WB == 4 ? 16 * h + 4 * g + p : (p & 1) + 8 * (p >> 1) + 2 * g;
          x[p] = *reinterpret_cast<const u32x4*>(rows_s + (r * kChunks + (c ^ r)) * 16);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[i] = WB == 4 ? multiply<WB>(q[i][h], q[i][h], s[i][h] >> (8 * g) & 0xffu, x, acc[i])
                           : multiply<WB>(q[i][0], q[i][1], s[i][0], x, acc[i]);
      }
      wave_lds_sync();
    }
    const auto& parts = part_s[turn % kTurns];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<v4f*>(&part_s[turn % kTurns][wave][r * kPartRow + 16 * i + 4 * g]) = acc[i];
    // the next unit's first step comes in under this one's sums
    const auto one = u.one;
    const int chunk = u.chunk, c0 = chunk * kChan;
    unit += gridDim.x;
    const bool more = unit < units;
    if (more) {
      int c = chunk + step_c;
      a += step_a;
      if (c >= chunks) {
        c -= chunks;
        ++a;
      }
      u = begin(a, c);
      if (wave < steps) load(&next, u, wave);
    }
    __syncthreads();
    // the entry's first slots fall to another wave each turn
    const int row = (int)((threadIdx.x >> 4) + 4 * turn) % (4 * WAVES), c = 2 * (threadIdx.x & 15);
    if (row < kCols && row / 4 * 4 < one.count) {  // whole waves
      float2_ gv = {0.0f, 0.0f}, uv = {0.0f, 0.0f};
#pragma unroll
      for (int q = 0; q < WAVES; ++q) {
        const float* p = parts[q] + row * kPartRow + c;
        gv += *reinterpret_cast<const float2_*>(p);
        uv += *reinterpret_cast<const float2_*>(p + kChan);
      }
      float v[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) v[j] = c0 + c + j < f ? swiglu(gv[j], uv[j]) : 0.0f;
      uint32_t top = max(magnitude(v[0]), magnitude(v[1]));
      top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xf, 0xf, false));
      top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xf, 0xf, false));
      top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x141, 0xf, 0xf, false));
      top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x140, 0xf, 0xf, false));
      const int64_t to = ch.slot_of(one, row);
      if (to >= 0) {
        const uint32_t s = scale_byte(top);
        const float inv = inverse_scale(s);
        uint8_t* dst = act + to * fp + c0 + c;
        *reinterpret_cast<uint16_t*>(dst) = (uint16_t)pack_e4m3(v[0] * inv, v[1] * inv, 0.0f, 0.0f);
        uint8_t* sc = act_scale + to * (fp / kBlk4) + chunk;
        if (c == 0) *sc = (uint8_t)s;
        if (chunk == chunks - 1)  // zeros up to the line's end
          for (int z = 1; c0 + z * kChan < fp; ++z) {
            *reinterpret_cast<uint16_t*>(dst + z * kChan) = 0;
            if (c == 0) sc[z] = 127;
          }
      }
    }
    if (!more) break;
    if (kTurns == 1) __syncthreads();
  }
#endif
}

// Up to 32 channels of the result and a share of the entries' long axes per workgroup:
// its waves take runs of steps and add them, times the slots' weights, to sums of
// their own in LDS.  The shares of the same channels meet in memory: the workgroup
// that is the last to write its sums adds them all, in order, and writes the result.
//
// Activations and scales pass through LDS as in the launch before.  8 tokens, 29
// experts of 7168 x 2688: 56 us, 5.6 TB/s; 64 tokens, 128 experts of 2048 x 768: 26.5
// us, of which some 10 are the choice of experts and the shares' meeting.  A second
// step's loads ahead brought nothing (26.7).
constexpr int kOut = 32, kMaxShares = 8;
template <int WB, bool SMALL, int kDownWaves>
__global__ __launch_bounds__(64 * kDownWaves, kDownWaves == 16 ? 4 : 2) void experts_down_kernel(
    Dims d, const int32_t* __restrict__ topk, const float* __restrict__ weight, const uint8_t* __restrict__ w,
    const uint8_t* __restrict__ ws, int f, const uint8_t* __restrict__ act, const uint8_t* __restrict__ act_scale,
    int width, int chunks, int shares, float* partial, uint32_t* counter, uint16_t* __restrict__ out) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int kDownThreads = 64 * kDownWaves;
  constexpr int kHalves = halves(WB), kPieces = 8 * kHalves;      // 16-byte pieces of a slot's step
  constexpr int kAtOnce = 64 / kPieces, kSets = kCols / kAtOnce;  // slots of a load, loads of 16 slots
  extern __shared__ __align__(16) unsigned char lds[];
  __shared__ __align__(16) unsigned char act_s[kDownWaves][kCols * kPieces * 16];
  __shared__ __align__(16) uint32_t act_scale_s[kDownWaves][kCols * kHalves];
  __shared__ __align__(16) uint32_t scale_s[kDownWaves][kOut * kHalves];
  __shared__ uint32_t arrived;
  float* sums = reinterpret_cast<float*>(lds);  // [waves][T + 1][kOut], the choice behind it
  const int per_wave = d.T * kOut, stride = per_wave + kOut;
  const auto ch = collect<SMALL, kDownThreads>(d, topk, lds + sizeof(float) * kDownWaves * stride, nullptr);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
  float* mine = sums + wave * stride;
  auto clear = [&]() {  // this wave's sums
    for (int i = lane; i < per_wave / 4; i += 64) *reinterpret_cast<v4f*>(mine + 4 * i) = v4f{0, 0, 0, 0};
  };
  const int share = blockIdx.x / chunks, chunk = blockIdx.x - share * chunks;
  const int c0 = chunk * width, valid = min(width, d.H - c0);
  const int fp = (int)padded_cols4(f), steps = (f + kHalves * kBlk - 1) / (kHalves * kBlk);
  const auto act_buf = buffer_of(act, (uint32_t)(d.T * d.k) * fp);
  const auto act_s_buf = buffer_of(act_scale, (uint32_t)(d.T * d.k) * (fp / kBlk4));
  // this wave's run of the ch.n * steps steps
  const int all = ch.n * steps, parts = shares * kDownWaves, part = share * kDownWaves + wave;
  const int from = (int)((int64_t)all * part / parts), to = (int)((int64_t)all * (part + 1) / parts);
  if (from < to) {
    int a = from / steps, b = from - a * steps;
    auto one = ch.one(a);
    Matrix<WB> m;
    uint32_t x_at[kSets], sx_at;
    // entry a: its matrix; the activations that this lane loads (past the buffers
    // where there is no slot: zeros)
    auto begin = [&]() {
      one = ch.one(a);
      m = matrix_rows<WB>(w, ws, one.expert, d.H, c0, valid, f);
#pragma unroll
      for (int i = 0; i < kSets; ++i) {
        const int s = ch.slot_of(one, i * kAtOnce + lane / kPieces);
        x_at[i] = s >= 0 ? (uint32_t)s * fp + 16 * (lane % kPieces) : 0x80000000u;
      }
      const int s = ch.slot_of(one, lane / kHalves);
      sx_at = s >= 0 ? (uint32_t)s * (fp / kBlk4) + 4 * (lane % kHalves) : 0x80000000u;
    };
    begin();
    const uint32_t at = (uint32_t)r * m.row_bytes + 16 * g, at_16 = at + 16 * m.row_bytes;
    const int s_row = min(lane & 31, valid - 1);
    const uint32_t s_at = WB == 4 ? s_row * 8 : (uint32_t)((c0 + s_row) / kBlk) * m.s_step;
    struct Step {
      v4i q[2][2];
      u32x2 s;
      v4i x[kSets];
      uint32_t sx;
    };
    auto load = [&](Step* o) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int p = 0; p < 2; ++p) o->q[i][p] = load16b(m.q, (i ? at_16 : at) + 64 * p, b * kBlk);
      if constexpr (WB == 4)
        o->s = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(m.s, (int)s_at, b * (int)m.s_step, 0));
      else
        o->s[0] = __builtin_amdgcn_raw_buffer_load_b8(m.s, (int)s_at, b, 0);
#pragma unroll
      for (int i = 0; i < kSets; ++i) {
        if (i * kAtOnce >= one.count) break;
        o->x[i] = load16b(act_buf, x_at[i], b * kHalves * kBlk);
      }
      o->sx = __builtin_amdgcn_raw_buffer_load_b32(act_s_buf, (int)sx_at, 4 * kHalves * b, 0);
    };
    // 16-byte place of a slot's piece: 16 slots' lie apart
    auto place = [&](int slot, int p) {
      return WB == 4 ? slot * 16 + (p ^ slot) : (slot >> 1) * 16 + (((slot & 1) << 3 | p) ^ (slot >> 1));
    };
    // Lanes without a slot add to the row behind the tokens'.  (A branch of lanes draws
    // the products in under it, where masked operands are wrong.)
    auto add = [&](int s, const v4f* acc) {
      const float by = weight[max(s, 0)];
      float* const row = mine + (s >= 0 ? s / d.k : d.T) * kOut + 4 * g;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v4f* sum = reinterpret_cast<v4f*>(row + 16 * i);
        v4f v = *sum;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += by * acc[i][j];
        *sum = v;
      }
    };
    Step next;
    load(&next);
    clear();  // while the first step comes in
    v4f acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    for (int item = from; item < to; ++item) {
      const auto entry = one;
      const bool last = ++b == steps;  // of this entry
#pragma unroll
      for (int i = 0; i < kSets; ++i) {
        if (i * kAtOnce >= entry.count) break;
        *reinterpret_cast<v4i*>(act_s[wave] + place(i * kAtOnce + lane / kPieces, lane % kPieces) * 16) = next.x[i];
      }
      if (lane < kCols * kHalves) act_scale_s[wave][lane] = next.sx;
      if (lane < kOut) {
        if (WB == 4)
          *reinterpret_cast<u32x2*>(scale_s[wave] + 2 * lane) = next.s;
        else
          scale_s[wave][lane] = next.s[0];
      }
      v4i q[2][2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int p = 0; p < 2; ++p) q[i][p] = next.q[i][p];
      wave_lds_sync();
      if (item + 1 < to) {
        if (last) {
          b = 0;
          ++a;
          begin();
        }
        load(&next);
      }
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const v4i lo = *reinterpret_cast<const v4i*>(act_s[wave] + place(r, 8 * h + g) * 16);
        const v4i hi = *reinterpret_cast<const v4i*>(act_s[wave] + place(r, 8 * h + 4 + g) * 16);
        const v8i xv = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        const uint32_t sx = act_scale_s[wave][r * kHalves + h] >> (8 * g);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const v4i q0 = q[i][h], q1 = q[i][1];
          const v8i qv = WB == 4 ? v8i{q0[0], q0[1], q0[2], q0[3], 0, 0, 0, 0}
                                 : v8i{q0[0], q0[1], q0[2], q0[3], q1[0], q1[1], q1[2], q1[3]};
          const uint32_t s = scale_s[wave][kHalves * (16 * i + r) + h] >> (WB == 4 ? 8 * g : 0);
          acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(qv, xv, acc[i], WB == 4 ? kFp4 : kFp8, kFp8, 0,
                                                                    (int)s, 0, (int)sx);
        }
      }
      if (last || item + 1 == to) {
        add(ch.slot_of(entry, r), acc);
#pragma unroll
        for (int i = 0; i < 2; ++i) acc[i] = v4f{0, 0, 0, 0};
      }
      wave_lds_sync();
    }
  } else {
    clear();
  }
  __syncthreads();
  auto write = [&](int i, float v) {  // sum i of [T][kOut]
    const int c = i % kOut;
    if (c < valid) out[(int64_t)(i / kOut) * d.H + c0 + c] = (uint16_t)pack_bf16(v, 0.0f);
  };
  typedef unsigned long long pair_;
  pair_* own = reinterpret_cast<pair_*>(partial + ((int64_t)chunk * shares + share) * per_wave);
  for (int i = threadIdx.x; i < per_wave / 2; i += kDownThreads) {
    float2_ v = {0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < kDownWaves; ++q) v += *reinterpret_cast<const float2_*>(sums + q * stride + 2 * i);
    if (shares > 1) {
      __hip_atomic_store(own + i, __builtin_bit_cast(pair_, v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    } else {
      write(2 * i, v[0]);
      write(2 * i + 1, v[1]);
    }
  }
  if (shares == 1) return;
  // The sums were written through to where all XCDs see them, and are there before
  // the arrival: the store of a device-wide atomic ends, for its wave's counter,
  // where it is visible.  (Fences instead write back and drop whole L2s: 384
  // workgroups took 27 us longer.)
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    arrived = __hip_atomic_fetch_add(counter + chunk, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  if (arrived != (uint32_t)shares - 1u) return;
  const pair_* every = reinterpret_cast<const pair_*>(partial) + (int64_t)chunk * shares * (per_wave / 2);
  for (int i = threadIdx.x; i < per_wave / 2; i += kDownThreads) {
    pair_ got[kMaxShares];  // all loads before the first sum
#pragma unroll
    for (int q = 0; q < kMaxShares; ++q)
      got[q] = __hip_atomic_load(every + (int64_t)min(q, shares - 1) * (per_wave / 2) + i, __ATOMIC_RELAXED,
                                 __HIP_MEMORY_SCOPE_AGENT);
    float2_ v = {0.0f, 0.0f};
#pragma unroll
    for (int q = 0; q < kMaxShares; ++q)
      if (q < shares) v += __builtin_bit_cast(float2_, got[q]);
    write(2 * i, v[0]);
    write(2 * i + 1, v[1]);
  }
#endif
}

// Where a call's memory goes: activations [T * k][fp], their scales [T * k][fp /
// 32], a counter per piece of channels, the shares' sums.
struct Work {
  int fp, waves, width, chunks, shares;
  int64_t scale, counter, partial, bytes;
};
Work work_of(const Dims& d, int f) {
  Work k;
  k.fp = (int)padded_cols4(f);
  // Sixteen waves to a workgroup, one for every CU, where their sums (128 bytes a
  // token and wave) fit the LDS beside their steps; else two of four waves.  (A token
  // with 8 experts of 2048 x 768: 5.9 us in sixteen, 7.8 in four; 16 tokens of 128 such
  // experts in 8 bits 23.1 and 23.4; 8 tokens, 29 experts of 7168 x 2688 55.8, 54.8.)
  k.waves = d.T <= 16 ? 16 : 4;
  const int want = k.waves == 16 ? 256 : 512;
  // shares cost a pass through memory: four lines a wave at least
  const int64_t lines = (int64_t)chosen_cap(d) * (k.fp / kCols4), most = lines / (4 * k.waves);
  // As wide as 32 channels; but of many channels so that their number divides among
  // the CUs (7168 channels: 256 workgroups of 28 and not 224 of 32), and where there
  // is nothing to share so narrow that all CUs have some (a token with 8 experts of 768
  // x 2048: 7.5 us in 64 workgroups, 6.0 in 256).  Shares of wide pieces are better
  // than narrow ones (16 tokens, 8 each of 128 experts, in 8 bits: 23 us and 33).
  k.width = kOut;
  if (d.H > 128 * kOut || most < 2) {
    const int rounds = (d.H + 256 * kOut - 1) / (256 * kOut);
    const int even = ((d.H + 256 * rounds - 1) / (256 * rounds) + 3) / 4 * 4;
    k.width = even < 8 ? 8 : even < kOut ? even : kOut;
  }
  k.chunks = (d.H + k.width - 1) / k.width;
  const int64_t fill = want / k.chunks;
  k.shares = (int)(fill < most ? fill : most);
  if (k.shares > kMaxShares) k.shares = kMaxShares;
  if (k.shares < 1) k.shares = 1;
  const int64_t slots = (int64_t)d.T * d.k;
  k.scale = slots * k.fp;
  k.counter = (k.scale + slots * (k.fp / kBlk4) + 15) / 16 * 16;
  k.partial = k.counter + ((int64_t)k.chunks * 4 + 15) / 16 * 16;
  k.bytes = k.partial + (k.shares > 1 ? (int64_t)k.chunks * k.shares * d.T * kOut * 4 : 0);
  return k;
}

template <int WB, bool SMALL, int WAVES>
hipError_t launch_down(const Dims& d, const Work& k, size_t lds, const int32_t* topk_idx, const float* weight,
                       int32_t f, const uint8_t* w2, const uint8_t* w2s, uint8_t* work, uint16_t* out,
                       hipStream_t st) {
  lds += (size_t)WAVES * (d.T + 1) * kOut * sizeof(float);
  // what 64 tokens with 32 of 2048 experts take is the most: every call sets the same,
  // those of other threads too
  constexpr int kMost = 72 * 1024;
  if (lds > kMost) return hipErrorInvalidValue;
  if (lds > 32768) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(experts_down_kernel<WB, SMALL, WAVES>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((experts_down_kernel<WB, SMALL, WAVES>), dim3((unsigned)(k.chunks * k.shares)), dim3(64 * WAVES),
                     lds, st, d, topk_idx, weight, w2, w2s, f, work, work + k.scale, k.width, k.chunks, k.shares,
                     reinterpret_cast<float*>(work + k.partial), reinterpret_cast<uint32_t*>(work + k.counter), out);
  return hipGetLastError();
}

template <int WB, bool SMALL, int WAVES>
hipError_t launch(const Dims& d, const uint16_t* hidden, const int32_t* topk_idx, const float* weight, int32_t f,
                  const uint8_t* w1, const uint8_t* w1s, const uint8_t* w2, const uint8_t* w2s, uint8_t* work,
                  uint16_t* out, int32_t* status, hipStream_t st) {
  const Work k = work_of(d, f);
  const int64_t units = (int64_t)chosen_cap(d) * ((f + kChan - 1) / kChan);
  const size_t lds = SMALL ? (size_t)8 * d.E : chosen_lds(d);
  // 512 workgroups are two to a CU (one where there are very many experts)
  hipLaunchKernelGGL((experts_up_kernel<WB, WAVES, SMALL>), dim3((unsigned)(units < 512 ? units : 512)),
                     dim3(64 * WAVES), lds, st, d, hidden, topk_idx, w1, w1s, f, work, work + k.scale,
                     reinterpret_cast<uint32_t*>(work + k.counter), k.chunks, status);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return k.waves == 16 ? launch_down<WB, SMALL, 16>(d, k, lds, topk_idx, weight, f, w2, w2s, work, out, st)
                       : launch_down<WB, SMALL, 4>(d, k, lds, topk_idx, weight, f, w2, w2s, work, out, st);
}

}  // namespace

int64_t experts_work_bytes(const Dims& d, int32_t f) { return work_of(d, f).bytes; }

hipError_t launch_experts(const Dims& d, const uint16_t* hidden, const int32_t* topk_idx, const float* weight,
                          int32_t w_bits, int32_t f, const uint8_t* w1, const uint8_t* w1s, const uint8_t* w2,
                          const uint8_t* w2s, uint8_t* work, uint16_t* out, int32_t* status, hipStream_t st) {
  if (d.T == 0) return hipSuccess;
  // Eight waves to a unit where there are fewer units than CUs: half the lines one after
  // the other (a token, 8 experts of 2 x 768 x 2048: 7.4 us, in four waves 7.8; 7 tokens
  // of 2 x 380 x 1000 in 8 bits 6.5, 7.0).
  const bool small = d.T * d.k <= 64, wide = (int64_t)chosen_cap(d) * ((f + kChan - 1) / kChan) <= 256;
  auto go = w_bits == 4 ? small ? wide ? launch<4, true, 8> : launch<4, true, 4> : launch<4, false, 4>
                        : small ? wide ? launch<8, true, 8> : launch<8, true, 4> : launch<8, false, 4>;
  return go(d, hidden, topk_idx, weight, f, w1, w1s, w2, w2s, work, out, status, st);
}

}  // namespace moe
