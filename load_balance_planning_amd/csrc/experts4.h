// Internal declarations of the operators of moe_experts4.h.
#pragma once

#include "experts.h"
#include "moe_experts4.h"

namespace moe {

// Columns of a 4-bit row as it is kept.
inline __host__ __device__ int64_t padded_cols4(int64_t c) { return (c + 255) / 256 * 256; }

constexpr int kMaxFewTokens = 64;  // a token set is one 64-bit mask

hipError_t launch_quantize4(const uint16_t* x, int64_t rows, int32_t cols, uint8_t* q, uint8_t* scale, hipStream_t st);
hipError_t launch_swiglu4(const uint16_t* y, int64_t rows, int32_t f, uint8_t* q, uint8_t* scale, hipStream_t st);
hipError_t launch_quantize_weights4(const uint16_t* w, int32_t experts, int32_t n, int32_t k, uint8_t* q,
                                    uint8_t* scale, uint8_t* qt, uint8_t* scale_t, hipStream_t st);
hipError_t launch_values4(const uint8_t* q, const uint8_t* scale, int32_t matrices, int64_t rows, int32_t cols,
                          uint16_t* x, hipStream_t st);

// Most tiles of launch_matmul4 (0: its kernel loops over any number).
int64_t matmul4_tiles(const Instances& in, int32_t x_bits, int32_t n, int32_t k);
hipError_t launch_matmul4(const Instances& in, int32_t x_bits, const uint8_t* x, const uint8_t* xs, const uint8_t* w,
                          const uint8_t* ws, int32_t n, int32_t k, uint16_t* y, int32_t* status, hipStream_t st);

int64_t experts_work_bytes(const Dims& d, int32_t f);
hipError_t launch_experts(const Dims& d, const uint16_t* hidden, const int32_t* topk_idx, const float* weight,
                          int32_t w_bits, int32_t f, const uint8_t* w1, const uint8_t* w1s, const uint8_t* w2,
                          const uint8_t* w2s, uint8_t* work, uint16_t* out, int32_t* status, hipStream_t st);

}  // namespace moe
