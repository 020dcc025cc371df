/*
 * moe_experts4 -- the expert layer with matrices in 4-bit floating point, and
 * a whole layer for few tokens, on MI355X.  Same library, handles, status word
 * and error codes as moe_plan.h; rows in 8 bits, plan and instances as in
 * moe_experts.h.
 *
 *   moex4_quantize     bf16 rows to e2m1 with one scale per 1 x 32 block
 *   moex4_quantize_weights
 *                      bf16 expert matrices, and the transposed matrices
 *   moex4_values       the bf16 values of such blocks
 *   moex4_swiglu       the gated activation between two products, quantized so
 *   moex4_matmul       each instance's rows, in 4 or 8 bits, times its expert's
 *                      matrix in 4 bits
 *   moex4_experts      a layer's experts for at most 64 tokens, from their top-k
 *                      and weights to the combined rows; matrices in 4 or 8 bits
 *
 * Forward pass of many tokens:
 *   moex_gate -> moe_plan_plan -> moe_plan_dispatch -> moex_quantize or
 *   moex4_quantize -> moex4_matmul (gate and up) -> moex_swiglu or moex4_swiglu
 *   -> moex4_matmul (down) -> moex_combine.
 * Backward: moex4_matmul of moex_quantize's or moex_swiglu_grad's rows with the
 * transposed matrices in place of moex_matmul; the gradient of the matrices is
 * moex_wgrad's, of rows in 8 bits.
 * Of few tokens: moex_gate -> moex4_experts.
 *
 * Blocks of 32.  A quantized row of C columns holds Cp e2m1 values (1 sign, 2
 * exponent and 1 mantissa bits: 0, 0.5, 1, 1.5, 2, 3, 4, 6), Cp = C rounded up
 * to 256, zeros from column C on, two to a byte, the first in the low half, and
 * one scale byte per 32 columns (E8M0 as in moe_experts.h; 127 for a block of
 * zeros).  The scales of 256 columns lie together, those of consecutive rows
 * one behind the other:
 *   rows      q uint8 [rows][Cp/2], scale uint8 [Cp/256][rows][8]
 *   matrices  q uint8 [E][N][Kp/2], scale uint8 [E][Kp/256][N][8]
 * where scale[b][r][i] is that of row r, columns 256 b + 32 i on.  (So 32 rows'
 * scales, which the products read at once, are two lines of memory and not 32.)
 * Scale byte 255 marks a block that held a NaN or an infinity (its values are
 * kept as 0), and every sum over such a block is NaN.
 * The quantizer's scale is the smallest power of two with which the block's
 * largest magnitude is at most 6 (not below 2^-126; 1 for a block of zeros), and
 * each value is x / scale rounded to the nearest e2m1, ties to the even code.
 * The products take any scale bytes.  q must be 16-byte aligned, scale 8-byte
 * aligned, else MOE_ERR_INVALID_ARG.
 *
 * No call needs memory of its own or touches the handle's workspace (the status
 * word aside): calls of one handle may run on several streams at once.  Every
 * call can be captured into a HIP graph.
 */
#ifndef MOE_EXPERTS4_H
#define MOE_EXPERTS4_H

#include "moe_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * x bf16 [rows][cols] to blocks of 1 x 32.  rows >= 0, cols >= 1;
 * MOE_ERR_UNSUPPORTED from 2^31 rows on and above 2^24 columns.
 */
int moex4_quantize(moe_plan_t h, const uint16_t* x, int64_t rows, int32_t cols, uint8_t* q, uint8_t* scale,
                   void* stream);

/*
 * w bf16 [experts][n][k] to blocks along k: q [experts][n][kp/2] and scale
 * [experts][kp/256][n][8], and (both or neither) the transposed matrices in
 * blocks along n: qt [experts][k][np/2] and scale_t [experts][np/256][k][8],
 * which moex4_matmul needs for the input gradient.  Their values differ from
 * q's: a value's block, and so its scale, is another.
 * experts >= 0, 1 <= n, k; MOE_ERR_UNSUPPORTED for n or k above 2^24 and for
 * 2^24 blocks of 128 x 128 or more in all matrices together (n and k rounded up
 * to 256).
 */
int moex4_quantize_weights(moe_plan_t h, const uint16_t* w, int32_t experts, int32_t n, int32_t k, uint8_t* q,
                           uint8_t* scale, uint8_t* qt, uint8_t* scale_t, void* stream);

/*
 * x bf16 [matrices][rows][cols]: the values of blocks q [matrices][rows][Cp/2]
 * with scale [matrices][Cp/256][rows][8] (rows: matrices = 1), value * scale
 * rounded to bf16 -- exact but below bf16's smallest subnormal and past its
 * range (infinite); NaN in a marked block.  matrices, rows >= 0, cols >= 1;
 * MOE_ERR_UNSUPPORTED for 2^31 rows or more in all and above 2^24 columns.
 */
int moex4_values(moe_plan_t h, const uint8_t* q, const uint8_t* scale, int32_t matrices, int64_t rows, int32_t cols,
                 uint16_t* x, void* stream);

/*
 * y bf16 [rows][2 f]: gate columns, then up columns.  moex_swiglu's value in
 * fp32 (within 2^-20 of it), quantized as a row of f columns.  rows and f as rows and cols of
 * moex4_quantize.
 */
int moex4_swiglu(moe_plan_t h, const uint16_t* y, int64_t rows, int32_t f, uint8_t* q, uint8_t* scale, void* stream);

/*
 * The experts' products, as moex_matmul:
 *   y[r][c] = bf16( sum over j of x[r][j] * w[e][c][j] )
 * w: 4-bit blocks of matrices [E][n][k]; x: rows [T*k][k], x_bits 4: 4-bit blocks
 * of rows, x_bits 8: moex_quantize's.  Sums in fp32 by the matrix instruction,
 * rounded once.  (With rows in 8 bits it cuts products off as in moex_matmul.
 * With 4 bits nothing is lost within a block; the blocks' sums are added as in
 * fp32, cut off below 2^-23 of the largest product.)  Instances, limits, errors
 * and the status word as in moex_matmul.
 */
int moex4_matmul(moe_plan_t h, const moe_plan_out* plan, const int32_t* inst_offset, int32_t x_bits, const uint8_t* x,
                 const uint8_t* x_scale, const uint8_t* w, const uint8_t* w_scale, int32_t n, int32_t k, uint16_t* y,
                 void* stream);

/*
 * A layer's experts for T <= 64 tokens, without plan or dispatch:
 *   (g, u)   = w1[e] times Q(hidden[t]),  a = Q(g * sigmoid(g) * u)
 *   out[t]   = bf16( sum over j of weight[t][j] * (w2[e] times a) ),  e = topk_idx[t][j]
 * hidden bf16 [T][H]; topk_idx int32 [T][k]; weight float [T][k] (moex_gate's, or
 * any); w1 matrices [E][2 f][H], gate rows then up rows, w2 [E][H][f], w_bits 4:
 * in blocks of 32 as above, w_bits 8: moex_quantize_weights'; out bf16 [T][H],
 * fully overwritten; neither it nor work may overlap anything that the call
 * reads, or the other.  Q rounds to e4m3 with one E8M0 scale per 1 x 32, by
 * moex_quantize's rules; all else is fp32, the sums in a fixed order.  The first
 * product takes values as bf16 (as moex4_values gives them; e4m3 * scale), so that
 * its sums lose nothing but what bf16 has not: steps below 2^-133, and values from
 * 2^128 on, which are infinite; the second cuts products off as moex_matmul does.
 * work: memory for one call at a time, 16-byte aligned, as many bytes as
 * moex4_experts_work says for the handle and f (host only).  After the call it
 * begins with the activations a, uint8 [T*k][fp], and their scales, uint8
 * [T*k][fp/32], fp = f rounded up to 256, of the slots whose index is good.
 * An index outside [0, E) or repeated within a token sets MOE_STATUS_BAD_TOPK; such
 * a slot is left out, of a repeated index all but the first.  f >= 1; MOE_ERR_UNSUPPORTED for more than 64 tokens, for f
 * or H above 2^20, and for matrices of 2^36 values or more.
 */
int moex4_experts_work(moe_plan_t h, int32_t f, int64_t* bytes);
int moex4_experts(moe_plan_t h, const uint16_t* hidden, const int32_t* topk_idx, const float* weight, int32_t w_bits,
                  int32_t f, const uint8_t* w1, const uint8_t* w1_scale, const uint8_t* w2, const uint8_t* w2_scale,
                  uint8_t* work, uint16_t* out, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_EXPERTS4_H */
