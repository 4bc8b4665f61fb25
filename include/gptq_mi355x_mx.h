/*
 * gptq_mi355x_mx.h - microscaled (MX) operators of libgptq_mi355x.so on one MI355X (gfx950): quantization to
 * 4 and 8 bits, the product of a quantized linear layer, and that layer's backward pass from an 8-bit (or
 * 4-bit) checkpoint of its input.
 *
 * Format (OCP Microscaling Formats v1.0 elements and scales). A matrix is quantized row by row in blocks of
 * 32 consecutive columns that share one power of two:
 *   value(r, c) = element(r, c) * 2^(byte(r, c / 32) - 127),   byte 255: the whole block is NaN.
 *   GPTQ_MX_E2M1  4 bits: sign and 0, .5, 1, 1.5, 2, 3, 4, 6. byte - 127 = floor(log2 amax) - 2, amax the
 *                 block's largest magnitude, and at least -125; values past 6 saturate.
 *   GPTQ_MX_E4M3  8 bits: sign, 4 exponent bits (bias 7), 3 mantissa bits, largest 448. byte - 127 is the
 *                 smallest exponent with amax <= 448 * 2^exponent, and at least -117, so nothing saturates.
 * Elements are rounded to nearest, ties to even. A block that holds a NaN or an infinity gets byte 255
 * and codes of 0. The least exponents keep every non-zero value a normal number in bf16, so values are exact
 * in bf16 and fp32, but for E4M3 elements of magnitude 248 * 2^120 and more: they round to 2^128, which both
 * types hold as infinity. Scale bytes below the least ones, which quantization does not write, are read as
 * the formula has them, values being rounded once to the type that holds them (the gradients' operands: bf16).
 *
 * Storage. codes: rows of gptq_mx_code_bytes_per_row(cols, fmt) bytes, columns in order, two E2M1 codes to a
 * byte with the even column in the low half, zeros from the last column to the next multiple of 128. scales:
 * rows of gptq_mx_scale_bytes_per_row(cols) bytes, block b's byte at position b, zeros behind the last block.
 * Both start at 16-byte aligned addresses. Rows are independent: a run of rows is itself such a matrix.
 *
 * Conventions are those of gptq_mi355x.h: row-major matrices, device pointers, caller-owned buffers and
 * workspaces (sized by the *_workspace_bytes queries, 256-byte aligned, contents unspecified, no
 * initialisation), stream-ordered and asynchronous calls, nothing launched on an argument error. No call
 * here synchronises or allocates, so all of them can be captured into a graph. Results lie apart from every
 * operand and from the workspace. n = 0 (no tokens) is valid
 * everywhere. Results are bitwise reproducible: no sum's order changes between calls of the same sizes.
 * Sizes: 1 <= in <= 65536, 1 <= out <= 2^20, 0 <= n < 2^31; others are GPTQ_ERR_INVALID_ARG, like NULL or
 * misaligned pointers, unknown formats or dtypes and leading dimensions below the row length.
 */
#ifndef GPTQ_MI355X_MX_H
#define GPTQ_MI355X_MX_H

#include "gptq_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { GPTQ_MX_E2M1 = 0, GPTQ_MX_E4M3 = 1 } gptq_mx_format;

/* Row lengths in bytes (0 for bad arguments): ceil(cols / 128) * 64 or * 128, and ceil(cols / 512) * 16. */
int64_t gptq_mx_code_bytes_per_row(int64_t cols, int fmt);
int64_t gptq_mx_scale_bytes_per_row(int64_t cols);

/* X (n x in, ld_x >= in, GPTQ_F32 or GPTQ_BF16) -> codes and scales. */
int gptq_mx_quantize(const void* X, int x_dtype, int64_t n, int64_t in, int64_t ld_x, int fmt, uint8_t* codes,
                     uint8_t* scales, void* stream);

/* codes and scales (n x in) -> Y (ld_y >= in, GPTQ_F32 or GPTQ_BF16), exactly. */
int gptq_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int fmt, int64_t n, int64_t in, void* Y,
                       int y_dtype, int64_t ld_y, void* stream);

/* Y = A W^T (+ bias) (then max(., 0) when relu == 1; NaN stays NaN). A n x in in a_fmt, W out x in in E2M1, bias
 * fp32[out] or NULL, Y n x out in GPTQ_F32 or GPTQ_BF16 (one rounding, at the end). Products are exact; sums are
 * held in fp32, whatever Y's type. */
size_t gptq_mx_matmul_workspace_bytes(int64_t n, int64_t in, int64_t out, int a_fmt);
int gptq_mx_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int a_fmt, int64_t n, int64_t in,
                   const uint8_t* w_codes, const uint8_t* w_scales, int64_t out, const float* bias, int relu,
                   void* Y, int y_dtype, int64_t ld_y, void* ws, size_t ws_bytes, void* stream);

/* Y = Q(X) W^T (+ bias) (ReLU): gptq_mx_quantize of X to act_fmt followed by gptq_mx_matmul, bit for bit, in one launch
 * for few tokens (n <= 16, n x in <= 32768). X n x in in x_dtype, ld_x >= in. */
size_t gptq_mx_linear_workspace_bytes(int64_t n, int64_t in, int64_t out, int act_fmt);
int gptq_mx_linear(const void* X, int x_dtype, int64_t n, int64_t in, int64_t ld_x, int act_fmt,
                   const uint8_t* w_codes, const uint8_t* w_scales, int64_t out, const float* bias, int relu,
                   void* Y, int y_dtype, int64_t ld_y, void* ws, size_t ws_bytes, void* stream);

/* dX = dY W, and where mask_codes is not NULL dX = 0 wherever the mask's value is not > 0: the backward pass of
 * the ReLU whose quantized outputs the mask holds (the layer's own input checkpoint). The mask is the checkpoint's,
 * not the activation's: a positive activation that was rounded to 0 shuts its gradient too. In E4M3 that is one of at
 * most 2^-10 of its block's scale (above the least scale at least 2.2e5 times below the block's largest), in E2M1 one of
 * at most 1/4 of the scale (1/32 to 1/16 of the block's largest; some 7 % of a Gaussian's positive half).
 * dY n x out bf16 (ld_dy >= out), W out x in in E2M1, mask n x in in mask_fmt, dX n x in in GPTQ_F32 or
 * GPTQ_BF16 (ld_dx >= in). Sums in fp32. The workspace holds W's values in bf16 and a padded copy of dY, which is written
 * only where dY's rows are not 16-byte aligned, longer than 2^20 elements or out is not a multiple of 64. */
size_t gptq_mx_grad_input_workspace_bytes(int64_t n, int64_t in, int64_t out);
int gptq_mx_grad_input(const void* dY, int64_t ld_dy, int64_t n, int64_t out, const uint8_t* w_codes,
                       const uint8_t* w_scales, int64_t in, const uint8_t* mask_codes, const uint8_t* mask_scales,
                       int mask_fmt, void* dX, int dx_dtype, int64_t ld_dx, void* ws, size_t ws_bytes, void* stream);

/* dW = dY^T A (out x in) and, where db is not NULL, db = column sums of dY (fp32[out]). dY n x out bf16 (ld_dy >=
 * out), A n x in in a_fmt: the checkpoint of the layer's input. accumulate == 1 (GPTQ_F32 only, UNSUPPORTED
 * otherwise): dW and db are added to. Sums in fp32 (db's in fp64, rounded once). n = 0 writes zeros (or adds nothing). The
 * workspace holds the checkpoint's values in bf16, twice an E4M3 checkpoint's bytes, and a padded copy of dY, which is
 * written only where dY's rows are not 16-byte aligned or longer than 2^20 elements. */
size_t gptq_mx_grad_weight_workspace_bytes(int64_t n, int64_t in, int64_t out);
int gptq_mx_grad_weight(const void* dY, int64_t ld_dy, int64_t n, int64_t out, const uint8_t* a_codes,
                        const uint8_t* a_scales, int a_fmt, int64_t in, int accumulate, void* dW, int dw_dtype,
                        int64_t ld_dw, float* db, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_MI355X_MX_H */
