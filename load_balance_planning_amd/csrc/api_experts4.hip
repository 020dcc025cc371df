// C ABI of the 4-bit operators and of the layer of few tokens: argument checks
// and launches.  See include/moe_experts4.h for the contract.
#include "experts4.h"
#include "handle.h"

using moe::begin_call;
using moe::DeviceScope;
using moe::hip_rc;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// A quantized operand: present, and its rows where the kernels load them.
bool blocks_ok(const void* q, const void* scale) { return q && scale && aligned(q, 16) && aligned(scale, 4); }
bool blocks4_ok(const void* q, const void* scale) { return q && scale && aligned(q, 16) && aligned(scale, 8); }

int check_rows(moe_plan_t h, int64_t rows, int32_t cols) {
  if (!h || rows < 0 || cols < 1) return MOE_ERR_INVALID_ARG;
  if (rows >= (int64_t)1 << 31 || cols > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" int moex4_quantize(moe_plan_t h, const uint16_t* x, int64_t rows, int32_t cols, uint8_t* q, uint8_t* scale,
                              void* stream) {
  const int rc = check_rows(h, rows, cols);
  if (rc != MOE_OK) return rc;
  if (rows > 0 && (!x || !blocks4_ok(q, scale))) return MOE_ERR_INVALID_ARG;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_quantize4(x, rows, cols, q, scale, begin_call(h, stream)));
}

extern "C" int moex4_quantize_weights(moe_plan_t h, const uint16_t* w, int32_t experts, int32_t n, int32_t k,
                                      uint8_t* q, uint8_t* scale, uint8_t* qt, uint8_t* scale_t, void* stream) {
  if (!h || experts < 0 || n < 1 || k < 1) return MOE_ERR_INVALID_ARG;
  if (n > (1 << 24) || k > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if (experts > 0 && (!w || !blocks4_ok(q, scale))) return MOE_ERR_INVALID_ARG;
  if ((qt == nullptr) != (scale_t == nullptr) || (qt && !blocks4_ok(qt, scale_t))) return MOE_ERR_INVALID_ARG;
  // one 256-thread workgroup per piece and up to seven more, fewer than 2^32 threads; by division, as the product
  // can pass 64 bits
  const int64_t per_matrix = (moe::padded_cols4(n) / moe::kBlk) * (moe::padded_cols4(k) / moe::kBlk);
  if (experts > (((int64_t)1 << 24) - 8) / per_matrix) return MOE_ERR_UNSUPPORTED;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_quantize_weights4(w, experts, n, k, q, scale, qt, scale_t, begin_call(h, stream)));
}

extern "C" int moex4_values(moe_plan_t h, const uint8_t* q, const uint8_t* scale, int32_t matrices, int64_t rows,
                            int32_t cols, uint16_t* x, void* stream) {
  if (matrices < 0) return MOE_ERR_INVALID_ARG;
  int rc = check_rows(h, rows, cols);
  if (rc == MOE_OK) rc = check_rows(h, rows * matrices, cols);  // both below 2^31
  if (rc != MOE_OK) return rc;
  if (rows * matrices > 0 && (!x || !blocks4_ok(q, scale))) return MOE_ERR_INVALID_ARG;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_values4(q, scale, matrices, rows, cols, x, begin_call(h, stream)));
}

extern "C" int moex4_swiglu(moe_plan_t h, const uint16_t* y, int64_t rows, int32_t f, uint8_t* q, uint8_t* scale,
                            void* stream) {
  const int rc = check_rows(h, rows, f);
  if (rc != MOE_OK) return rc;
  if (rows > 0 && (!y || !blocks4_ok(q, scale))) return MOE_ERR_INVALID_ARG;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_swiglu4(y, rows, f, q, scale, begin_call(h, stream)));
}

extern "C" int moex4_matmul(moe_plan_t h, const moe_plan_out* plan, const int32_t* inst_offset, int32_t x_bits,
                            const uint8_t* x, const uint8_t* x_scale, const uint8_t* w, const uint8_t* w_scale,
                            int32_t n, int32_t k, uint16_t* y, void* stream) {
  if (!h || !plan || !plan->n_inst || !plan->inst_expert || !inst_offset || n < 1 || k < 1) return MOE_ERR_INVALID_ARG;
  if (x_bits != 4 && x_bits != 8) return MOE_ERR_INVALID_ARG;
  // a tile of 256 rows is addressed with 32-bit offsets
  if (n > (1 << 20) || k > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (h->d.T > 0 && (!(x_bits == 4 ? blocks4_ok(x, x_scale) : blocks_ok(x, x_scale)) || !blocks4_ok(w, w_scale) || !y))
    return MOE_ERR_INVALID_ARG;
  const moe::Instances in{plan->n_inst, plan->inst_expert, inst_offset, h->d.cap, h->d.E, (int64_t)h->d.T * h->d.k};
  // moex_matmul's limit; no call reaches it whose result fits the card's memory
  if (moe::matmul4_tiles(in, x_bits, n, k) >= (int64_t)1 << 24) return MOE_ERR_UNSUPPORTED;
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_matmul4(in, x_bits, x, x_scale, w, w_scale, n, k, y, h->ws.status, begin_call(h, stream)));
}

namespace {

// Sizes that the layer of few tokens takes: its kernels address an expert's scales with 32 bits.
int check_few(moe_plan_t h, int32_t f) {
  if (!h || f < 1) return MOE_ERR_INVALID_ARG;
  const moe::Dims& d = h->d;
  if (d.T > moe::kMaxFewTokens || f > (1 << 20) || d.H > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (2 * (int64_t)f * (moe::padded_cols4(d.H) / 32) >= (int64_t)1 << 31 ||
      (int64_t)d.H * (moe::padded_cols4(f) / 32) >= (int64_t)1 << 31)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" int moex4_experts_work(moe_plan_t h, int32_t f, int64_t* bytes) {
  if (!bytes) return MOE_ERR_INVALID_ARG;
  const int rc = check_few(h, f);
  if (rc == MOE_OK) *bytes = moe::experts_work_bytes(h->d, f);
  return rc;
}

extern "C" int moex4_experts(moe_plan_t h, const uint16_t* hidden, const int32_t* topk_idx, const float* weight,
                             int32_t w_bits, int32_t f, const uint8_t* w1, const uint8_t* w1_scale, const uint8_t* w2,
                             const uint8_t* w2_scale, uint8_t* work, uint16_t* out, void* stream) {
  if (w_bits != 4 && w_bits != 8) return MOE_ERR_INVALID_ARG;
  const int rc = check_few(h, f);
  if (rc != MOE_OK) return rc;
  if (h->d.T > 0) {
    if (!hidden || !topk_idx || !weight || !out || !work || !aligned(work, 16)) return MOE_ERR_INVALID_ARG;
    if (w_bits == 4 ? !blocks4_ok(w1, w1_scale) || !blocks4_ok(w2, w2_scale)
                    : !blocks_ok(w1, w1_scale) || !blocks_ok(w2, w2_scale))
      return MOE_ERR_INVALID_ARG;
  }
  const DeviceScope on_device(h->device);
  if (!on_device.ok()) return MOE_ERR_HIP;
  return hip_rc(moe::launch_experts(h->d, hidden, topk_idx, weight, w_bits, f, w1, w1_scale, w2, w2_scale, work, out,
                                    h->ws.status, begin_call(h, stream)));
}
