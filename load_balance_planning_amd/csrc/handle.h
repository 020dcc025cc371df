// The handle behind moe_plan_t and the set-up that every C entry point shares.
#pragma once

#include "internal.h"

struct moe_plan {
  moe::Dims d;
  moe_plan_config cfg;
  int device;
  moe::Workspace ws;
  void* ws_base;
  size_t ws_bytes;
  hipStream_t last_stream;  // stream of the last call that enqueued work (moe_plan_status waits for it)
  moe::KernelEvents gather_ev;  // moe_plan_set_events / moe_plan_set_gather_order: hooks around every gather launch
  bool acc_dirty;           // a step failed after its top-k was queued: the accumulator may hold counts
};

namespace moe {

// Makes `device` current for the duration of a call and gives the caller's
// current device back when the call returns.
class DeviceScope {
 public:
  explicit DeviceScope(int device) {
    if (hipGetDevice(&prev_) != hipSuccess) return;
    if (prev_ != device && hipSetDevice(device) != hipSuccess) return;
    switched_ = prev_ != device;
    ok_ = true;
  }
  ~DeviceScope() {
    if (switched_) (void)hipSetDevice(prev_);
  }
  DeviceScope(const DeviceScope&) = delete;
  DeviceScope& operator=(const DeviceScope&) = delete;
  bool ok() const { return ok_; }

 private:
  int prev_ = -1;
  bool switched_ = false;
  bool ok_ = false;
};

inline int hip_rc(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// Set-up shared by the calls that enqueue work: clears an error an earlier
// HIP call of the caller left behind (so that a failure reported by this
// call is its own) and remembers the stream for moe_plan_status.
inline hipStream_t begin_call(moe_plan_t h, void* stream) {
  (void)hipGetLastError();
  h->last_stream = static_cast<hipStream_t>(stream);
  return h->last_stream;
}

}  // namespace moe
