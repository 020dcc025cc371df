// C ABI of the expert-layer operators: argument checks and launches.  See
// include/moe_experts.h for the contract.
#include <math.h>

#include "experts.h"
#include "handle.h"

using moe::begin_call;
using moe::DeviceScope;
using moe::hip_rc;

namespace {

int check_gate(const moe::Dims& d, const moex_gate_config* g) {
  if (!g || (g->score != MOEX_SOFTMAX && g->score != MOEX_SIGMOID)) return MOE_ERR_INVALID_ARG;
  if (g->n_group < 1 || d.E % g->n_group != 0 || g->topk_group < 1 || g->topk_group > g->n_group)
    return MOE_ERR_INVALID_ARG;
  const int per = d.E / g->n_group;
  if (g->n_group > 1 && (g->group_top < 1 || g->group_top > 2 || g->group_top > per)) return MOE_ERR_INVALID_ARG;
  if ((int64_t)g->topk_group * per < d.k) return MOE_ERR_INVALID_ARG;
  // scale / (sum + 1e-20), and its product with a weight's gradient, stay finite; a NaN is refused too
  if (!(fabsf(g->scale) <= 4294967296.0f)) return MOE_ERR_INVALID_ARG;
  if (g->n_group > moe::kMaxGateGroups) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A quantized operand: present, and its rows where the kernels load them.
bool blocks_ok(const void* q, const void* scale) { return q && scale && aligned(q, 16) && aligned(scale, 4); }

int check_product(moe_plan_t h, const moe_plan_out* plan, const int32_t* inst_offset, int32_t n, int32_t k) {
  if (!h || !plan || !plan->n_inst || !plan->inst_expert || !inst_offset || n < 1 || k < 1) return MOE_ERR_INVALID_ARG;
  // a tile of 256 rows is addressed with 32-bit offsets
  if (n > (1 << 20) || k > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe::Instances instances(const moe::Dims& d, const moe_plan_out* plan, const int32_t* inst_offset) {
  return moe::Instances{plan->n_inst, plan->inst_expert, inst_offset, d.cap, d.E, (int64_t)d.T * d.k};
}

int check_rows(moe_plan_t h, int64_t rows, int32_t cols) {
  if (!h || rows < 0 || cols < 1) return MOE_ERR_INVALID_ARG;
  if (rows >= (int64_t)1 << 31 || cols > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" int moex_gate(moe_plan_t h, const moex_gate_config* gate, const float* logits, const float* bias,
                         const int32_t* prev_topk, const moe_route_out* out, float* weight, void* stream) {
  if (!h || !out || !out->expert_count || !out->omega) return MOE_ERR_INVALID_ARG;
  const moe::Dims& d = h->d;
  if (d.T > 0 && (!logits || !out->topk_idx || !weight)) return MOE_ERR_INVALID_ARG;
  const int rc = check_gate(d, gate);
  if (rc != MOE_OK) return rc;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  hipStream_t st = begin_call(h, stream);
  const int32_t* prev = (prev_topk && out->trans) ? prev_topk : nullptr;
  bool counted = false;
  hipError_t e = moe::launch_gate(d, *gate, logits, bias, prev, out->topk_idx, out->topk_val, weight,
                                  h->ws.tile_mask, h->ws.prev_mask, out->cooc || prev, out->omega, out->expert_count,
                                  &counted, h->ws.status, st);
  if (e == hipSuccess && !counted)
    e = moe::launch_scan_pairs(d, h->ws.tile_mask, nullptr, out->omega, out->expert_count, h->ws.prev_mask,
                               out->cooc, prev ? out->trans : nullptr, h->ws.pair_part, st);
  return hip_rc(e);
}

extern "C" int moex_gate_grad(moe_plan_t h, const moex_gate_config* gate, const float* logits,
                              const int32_t* topk_idx, const float* grad_weight, float* grad_logits, void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  const moe::Dims& d = h->d;
  const int rc = check_gate(d, gate);
  if (rc != MOE_OK) return rc;
  if (d.T > 0 && (!logits || !topk_idx || !grad_weight || !grad_logits)) return MOE_ERR_INVALID_ARG;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_gate_grad(d, *gate, logits, topk_idx, grad_weight, grad_logits, h->ws.status,
                                      begin_call(h, stream)));
}

extern "C" int moex_quantize(moe_plan_t h, const uint16_t* x, int64_t rows, int32_t cols, uint8_t* q, uint8_t* scale,
                             void* stream) {
  const int rc = check_rows(h, rows, cols);
  if (rc != MOE_OK) return rc;
  if (rows > 0 && (!x || !blocks_ok(q, scale))) return MOE_ERR_INVALID_ARG;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_quantize(x, rows, cols, q, scale, begin_call(h, stream)));
}

extern "C" int moex_quantize_weights(moe_plan_t h, const uint16_t* w, int32_t experts, int32_t n, int32_t k,
                                     uint8_t* q, uint8_t* scale, uint8_t* qt, uint8_t* scale_t, void* stream) {
  if (!h || experts < 0 || n < 1 || k < 1) return MOE_ERR_INVALID_ARG;
  if (n > (1 << 24) || k > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (experts > 0 && (!w || !blocks_ok(q, scale))) return MOE_ERR_INVALID_ARG;
  if ((qt == nullptr) != (scale_t == nullptr) || (qt && !blocks_ok(qt, scale_t))) return MOE_ERR_INVALID_ARG;
  // one 256-thread workgroup per block, fewer than 2^32 threads; by division, as the product can pass 64 bits
  const int64_t per_matrix = (moe::padded_cols(n) / moe::kBlk) * (moe::padded_cols(k) / moe::kBlk);
  if (experts > (((int64_t)1 << 24) - 1) / per_matrix) return MOE_ERR_UNSUPPORTED;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_quantize_weights(w, experts, n, k, q, scale, qt, scale_t, begin_call(h, stream)));
}

extern "C" int moex_swiglu(moe_plan_t h, const uint16_t* y, int64_t rows, int32_t f, uint8_t* q, uint8_t* scale,
                           void* stream) {
  const int rc = check_rows(h, rows, f);
  if (rc != MOE_OK) return rc;
  if (rows > 0 && (!y || !blocks_ok(q, scale))) return MOE_ERR_INVALID_ARG;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_swiglu(y, rows, f, q, scale, begin_call(h, stream)));
}

extern "C" int moex_swiglu_grad(moe_plan_t h, const uint16_t* y, const uint16_t* grad, int64_t rows, int32_t f,
                                uint8_t* q, uint8_t* scale, void* stream) {
  const int rc = check_rows(h, rows, f);
  if (rc != MOE_OK) return rc;
  if (rows > 0 && (!y || !grad || !blocks_ok(q, scale))) return MOE_ERR_INVALID_ARG;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_swiglu_grad(y, grad, rows, f, q, scale, begin_call(h, stream)));
}

extern "C" int moex_matmul(moe_plan_t h, const moe_plan_out* plan, const int32_t* inst_offset, const uint8_t* x,
                           const uint8_t* x_scale, const uint8_t* w, const uint8_t* w_scale, int32_t n, int32_t k,
                           uint16_t* y, void* stream) {
  const int rc = check_product(h, plan, inst_offset, n, k);
  if (rc != MOE_OK) return rc;
  if (h->d.T > 0 && (!blocks_ok(x, x_scale) || !blocks_ok(w, w_scale) || !y)) return MOE_ERR_INVALID_ARG;
  // one 256-thread workgroup per tile, fewer than 2^32 work-items a launch
  if (moe::matmul_tiles(instances(h->d, plan, inst_offset), n) >= (int64_t)1 << 24) return MOE_ERR_UNSUPPORTED;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_matmul(instances(h->d, plan, inst_offset), x, x_scale, w, w_scale, n, k, y, h->ws.status,
                                   begin_call(h, stream)));
}

extern "C" int moex_wgrad(moe_plan_t h, const moe_plan_out* plan, const int32_t* inst_offset, const uint8_t* dy,
                          const uint8_t* dy_scale, const uint8_t* x, const uint8_t* x_scale, int32_t n, int32_t k,
                          uint16_t* dw, void* stream) {
  const int rc = check_product(h, plan, inst_offset, n, k);
  if (rc != MOE_OK) return rc;
  if (!dw || (h->d.T > 0 && (!blocks_ok(dy, dy_scale) || !blocks_ok(x, x_scale)))) return MOE_ERR_INVALID_ARG;
  if (moe::wgrad_tiles(instances(h->d, plan, inst_offset), n, k) >= (int64_t)1 << 24) return MOE_ERR_UNSUPPORTED;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_wgrad(instances(h->d, plan, inst_offset), dy, dy_scale, x, x_scale, n, k, dw,
                                  h->ws.status, begin_call(h, stream)));
}

extern "C" int moex_combine(moe_plan_t h, const float* weight, const int32_t* slot_pos, const uint16_t* expert_out,
                            uint16_t* out, void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  if (h->d.T > 0 && (!slot_pos || !expert_out || !out)) return MOE_ERR_INVALID_ARG;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_combine_weighted(h->d, weight, slot_pos, expert_out, out, h->ws.status,
                                             begin_call(h, stream)));
}

extern "C" int moex_combine_grad(moe_plan_t h, const float* weight, const int32_t* slot_pos,
                                 const uint16_t* expert_out, const uint16_t* grad_out, uint16_t* grad_expert_out,
                                 float* grad_weight, void* stream) {
  if (!h) return MOE_ERR_INVALID_ARG;
  if (h->d.T > 0 && (!weight || !slot_pos || !expert_out || !grad_out || !grad_expert_out || !grad_weight))
    return MOE_ERR_INVALID_ARG;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_combine_grad(h->d, weight, slot_pos, expert_out, grad_out, grad_expert_out, grad_weight,
                                         h->ws.status, begin_call(h, stream)));
}
