/*
 * gptq_mi355x_int8.h - operators of libgptq_mi355x.so on 8-bit integers with a scale for each row: quantization of tokens,
 * the product of a linear layer whose weights are GPTQ's integer codes, that layer on unquantized tokens, and the
 * root-mean-square norm that writes what the products read, with its gradient.
 *
 * Format. value(r, c) = code(r, c) * scale(r), codes whole numbers in 8 bits, scales fp32: what gptq_quantize_layer
 * returns on the symmetric grid with one grid per row (2 to 8 bits), and what gptq_int8_quantize makes of tokens:
 *   scale = max(max|x|, 1e-12) / 127 (fp32, rounded once), code = x / scale, the exact quotient rounded to nearest,
 *   ties to even. A row that holds a NaN or an infinity gets the scale NaN and codes of 0, so all it enters is NaN.
 *
 * Storage. codes: rows of gptq_int8_code_bytes_per_row(cols) bytes, zeros from the last column to the next multiple of
 * 128, starting at a 16-byte aligned address. Rows are independent: a run of rows is itself such a matrix. GPTQ's codes
 * have this form where `in` is a multiple of 128; gptq_int8_pad_codes copies others into it.
 *
 * Conventions are those of gptq_mi355x.h: row-major matrices, device pointers, caller-owned buffers and workspaces (sized
 * by the *_workspace_bytes queries, 256-byte aligned, contents unspecified, no initialisation), stream-ordered and
 * asynchronous calls, nothing launched on an argument error. No call here synchronises or allocates, so all of them can
 * be captured into a graph; calls that may run at the same time need workspaces of their own. Results lie apart from every
 * operand and from the workspace, but for the norm's sum (below). n = 0 (no tokens) is valid everywhere. Results are
 * bitwise reproducible: no sum's order changes between calls of the same sizes. Sizes: 1 <= in <= 65536,
 * 1 <= out <= 2^20, 0 <= n < 2^31; others are GPTQ_ERR_INVALID_ARG, like NULL or misaligned pointers, unknown formats or
 * dtypes and leading dimensions below the row length.
 */
#ifndef GPTQ_MI355X_INT8_H
#define GPTQ_MI355X_INT8_H

#include "gptq_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Row length in bytes (0 for bad arguments): ceil(cols / 128) * 128. */
int64_t gptq_int8_code_bytes_per_row(int64_t cols);

/* X (n x in, ld_x >= in, GPTQ_F32 or GPTQ_BF16) -> codes and scales (fp32[n]). */
int gptq_int8_quantize(const void* X, int x_dtype, int64_t n, int64_t in, int64_t ld_x, int8_t* codes, float* scales,
                       void* stream);

/* codes and scales (n x in) -> Y = code * scale (ld_y >= in, GPTQ_F32 or GPTQ_BF16; rounded to fp32, then to Y's type). */
int gptq_int8_dequantize(const int8_t* codes, const float* scales, int64_t n, int64_t in, void* Y, int y_dtype,
                         int64_t ld_y, void* stream);

/* Contiguous codes (out x in, as gptq_quantize_layer writes them; any address) -> rows of the storage above. */
int gptq_int8_pad_codes(const int8_t* codes, int64_t out, int64_t in, int8_t* padded, void* stream);

/* Y = A W^T (+ bias) (then max(., 0) when relu == 1; NaN stays NaN). A n x in, W out x in, bias fp32[out] or NULL, Y
 * n x out in GPTQ_F32 or GPTQ_BF16. The sum S of code products is a whole number and exact. p = fp32(S) * a_scale, S and
 * the product each rounded to fp32; y = p * w_scale + bias (0 for NULL) in one step, rounded once; bf16 is rounded to at the
 * end. p has fp32's range: where |S| a_scale reaches 2^128 y is infinite whatever w_scale is, and below 2^-126 p loses
 * bits. */
size_t gptq_int8_matmul_workspace_bytes(int64_t n, int64_t in, int64_t out);
int gptq_int8_matmul(const int8_t* a_codes, const float* a_scales, int64_t n, int64_t in, const int8_t* w_codes,
                     const float* w_scales, int64_t out, const float* bias, int relu, void* Y, int y_dtype, int64_t ld_y,
                     void* ws, size_t ws_bytes, void* stream);

/* Y = Q(X) W^T (+ bias) (ReLU): gptq_int8_quantize of X followed by gptq_int8_matmul, bit for bit. X n x in in x_dtype,
 * ld_x >= in. */
size_t gptq_int8_linear_workspace_bytes(int64_t n, int64_t in, int64_t out);
int gptq_int8_linear(const void* X, int x_dtype, int64_t n, int64_t in, int64_t ld_x, const int8_t* w_codes,
                     const float* w_scales, int64_t out, const float* bias, int relu, void* Y, int y_dtype, int64_t ld_y,
                     void* ws, size_t ws_bytes, void* stream);

/* Root-mean-square norm of h = X + R (h = X where R is NULL), weighted, in 8 bits:
 *   h: the sum is rounded to fp32, then to R's type and, where R is not NULL, written to H (that type, ld_h >= d);
 *   rstd = 1 / sqrt(mean of h^2 + eps), sums in fp64, rounded to fp32 and written where rstd is not NULL (fp32[n]);
 *   u = h * weight, rounded to fp32 (weight: fp32[d]);
 *   GPTQ_NORM_INT8: u is quantized as by gptq_int8_quantize, and the row's scale is then multiplied by rstd;
 *   GPTQ_NORM_E4M3: u * rstd, rounded to fp32, is quantized as by gptq_mx_quantize to GPTQ_MX_E4M3.
 * codes and scales have the format's storage (scales: fp32[n], or MX scale bytes, 16-byte aligned). H may be R itself
 * (same address, ld_h == ld_r: the residual is updated in place); it lies apart from all else. 1 <= d <= 65536, eps finite
 * and at least 1e-30. */
typedef enum { GPTQ_NORM_INT8 = 0, GPTQ_NORM_E4M3 = 1 } gptq_norm_format;
int gptq_rms_norm(const void* X, int x_dtype, int64_t ld_x, const void* R, int r_dtype, int64_t ld_r, int64_t n, int64_t d,
                  const float* weight, double eps, void* H, int64_t ld_h, int fmt, void* codes, void* scales, float* rstd,
                  void* stream);

/* The norm's gradient for dY, the gradient of u * rstd (the rounding to 8 bits passes it on unchanged):
 *   g = dY * weight;  dX = rstd * (g - h * rstd^2 * mean of g h) (+ dH);  dweight = sum over rows of dY * h * rstd.
 * dY n x d in y_dtype; h (n x d) and dX in h_dtype; dH, where not NULL, is the gradient of the sum h itself, in h_dtype;
 * dX is the gradient of X and of R alike. dweight fp32[d]; accumulate == 1: it is added to. n = 0 writes zeros there (or adds
 * nothing). Sums of a row in fp32, those of dweight in fp64. */
size_t gptq_rms_norm_grad_workspace_bytes(int64_t n, int64_t d);
int gptq_rms_norm_grad(const void* dY, int y_dtype, int64_t ld_dy, const void* h, int h_dtype, int64_t ld_h,
                       const float* rstd, const float* weight, const void* dH, int64_t ld_dh, int64_t n, int64_t d,
                       int accumulate, void* dX, int64_t ld_dx, float* dweight, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_MI355X_INT8_H */
