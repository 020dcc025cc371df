// Internal declarations of the expert-layer operators (moe_experts.h).
#pragma once

#include "internal.h"
#include "moe_experts.h"

namespace moe {

constexpr int kBlk = 128;         // columns (and, for matrices, rows) under one scale
constexpr int kMaxGateGroups = 64;

// Bytes of a quantized row of c columns, and scale bytes of it.
inline __host__ __device__ int64_t padded_cols(int64_t c) { return (c + kBlk - 1) / kBlk * kBlk; }
inline __host__ __device__ int64_t scale_cols(int64_t c) { return (padded_cols(c) / kBlk + 3) / 4 * 4; }

// The router; *counted: its few tokens were one workgroup's, which wrote omega and
// count itself (only with masks_wanted false: the masks are then not written).
hipError_t launch_gate(const Dims& d, const moex_gate_config& g, const float* logits, const float* bias,
                       const int32_t* prev_topk, int32_t* topk_idx, float* topk_val, float* weight,
                       uint64_t* tile_mask, uint64_t* prev_mask, bool masks_wanted, int32_t* omega, int32_t* count,
                       bool* counted, int32_t* status, hipStream_t st);
hipError_t launch_gate_grad(const Dims& d, const moex_gate_config& g, const float* logits, const int32_t* topk_idx,
                            const float* grad_weight, float* grad_logits, int32_t* status, hipStream_t st);

hipError_t launch_quantize(const uint16_t* x, int64_t rows, int32_t cols, uint8_t* q, uint8_t* scale, hipStream_t st);
hipError_t launch_quantize_weights(const uint16_t* w, int32_t experts, int32_t n, int32_t k, uint8_t* q,
                                   uint8_t* scale, uint8_t* qt, uint8_t* scale_t, hipStream_t st);
hipError_t launch_swiglu(const uint16_t* y, int64_t rows, int32_t f, uint8_t* q, uint8_t* scale, hipStream_t st);
hipError_t launch_swiglu_grad(const uint16_t* y, const uint16_t* grad, int64_t rows, int32_t f, uint8_t* q,
                              uint8_t* scale, hipStream_t st);

// The rows of a plan's instances, as the products read them.
struct Instances {
  const int32_t* n_inst;
  const int32_t* expert;
  const int32_t* offset;
  int32_t cap;   // instance capacity E + B
  int32_t E;
  int64_t rows;  // T * k
};
int64_t matmul_tiles(const Instances& in, int32_t n);  // workgroups of launch_matmul's tile kernels (0: it loops)
hipError_t launch_matmul(const Instances& in, const uint8_t* x, const uint8_t* xs, const uint8_t* w, const uint8_t* ws,
                         int32_t n, int32_t k, uint16_t* y, int32_t* status, hipStream_t st);
int64_t wgrad_tiles(const Instances& in, int32_t n, int32_t k);  // workgroups of launch_wgrad
hipError_t launch_wgrad(const Instances& in, const uint8_t* dy, const uint8_t* dys, const uint8_t* x,
                        const uint8_t* xs, int32_t n, int32_t k, uint16_t* dw, int32_t* status, hipStream_t st);

hipError_t launch_combine_weighted(const Dims& d, const float* weight, const int32_t* slot_pos,
                                   const uint16_t* expert_out, uint16_t* out, int32_t* status, hipStream_t st);
hipError_t launch_combine_grad(const Dims& d, const float* weight, const int32_t* slot_pos,
                               const uint16_t* expert_out, const uint16_t* grad_out, uint16_t* grad_expert_out,
                               float* grad_weight, int32_t* status, hipStream_t st);

}  // namespace moe
