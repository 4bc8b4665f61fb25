// Shared definitions of the 8-bit integer operators and the norm.
#pragma once

#include "../../include/gptq_mi355x_int8.h"
#include "mx.h"

namespace gptq {

static inline int64_t int8_code_row(int64_t cols) { return ceil_div(cols, 128) * 128; }

// One operand: rows of codes at their fixed row length, a scale for each.
struct Int8Matrix {
  const int8_t* codes;
  const float* scales;
  int64_t rows, cols;
};

// int8_quant.hip
hipError_t int8_quantize_launch(const void* X, int x_dtype, int64_t n, int64_t in, int64_t ld_x, int8_t* codes,
                                float* scales, hipStream_t stream);
hipError_t int8_dequantize_launch(const Int8Matrix& q, void* Y, int y_dtype, int64_t ld_y, hipStream_t stream);
hipError_t int8_pad_launch(const int8_t* codes, int64_t out, int64_t in, int8_t* padded, hipStream_t stream);

// int8_gemm.hip: Y = A W^T (+ bias) (ReLU)
size_t int8_matmul_ws_bytes(int64_t n, int64_t in, int64_t out);
hipError_t int8_matmul_launch(const Int8Matrix& a, const Int8Matrix& w, const float* bias, int relu, void* Y, int y_dtype,
                              int64_t ld_y, void* ws, hipStream_t stream);
size_t int8_linear_ws_bytes(int64_t n, int64_t in, int64_t out);
hipError_t int8_linear_launch(const void* X, int x_dtype, int64_t n, int64_t ld_x, const Int8Matrix& w, const float* bias,
                              int relu, void* Y, int y_dtype, int64_t ld_y, void* ws, hipStream_t stream);

// int8_few.hip: the same for few tokens, in codes or, where they are small enough, quantized on their way in. us against the tile
// product: 17 x 4096 x 4096 6.7 / 9.5, 32 x 4096 x 4096 8.0 / 9.7, 32 x 512 x 512 2.9 / 4.6, but 24 x 11008 x 4096 18 / 17 and
// 24 x 4096 x 11008 (two rounds of workgroups, each loading all tokens) 19 / 15.
static inline bool int8_few(int64_t n, int64_t in, int64_t out) {
  return n <= 16 || (n <= 32 && in <= 4096 && out <= 4096);
}
// us of GPU time so / with a launch to quantize them, which also costs a call 3 us on the host: 1 x 4096 x 4096 7.1 / 8.4,
// 4 x 4096 x 4096 8.6 / 8.7, 8 x 4096 x 4096 10.2 / 9.3, 16 x 4096 x 4096 (too many) - / 9.4. Every workgroup of 16 channels
// quantizes all tokens anew, so wide layers lose by it what a launch does not cost: 8 x 4096 x 11008 19.3 / 16.3, 16 x 2048 x
// 11008 16.1 / 12.1, and at 131072 channels 1 x 4096 93 / 93, 8 x 4096 135 / 117, 16 x 2048 123 / 80. The rule does not look at `out`.
static inline bool int8_few_fused(int64_t n, int64_t in) {
  return n <= 16 && in >= 8 && (n <= 2 ? n : n <= 4 ? 4 : n <= 8 ? 8 : 16) * in <= 8 * 4096;
}
hipError_t int8_matmul_few_launch(const Int8Matrix& x, const Int8Matrix& w, const float* bias, int relu, void* Y, int y_dtype,
                                  int64_t ld_y, hipStream_t stream);
hipError_t int8_linear_few_launch(const void* X, int x_dtype, int64_t n, int64_t ld_x, const Int8Matrix& w, const float* bias,
                                  int relu, void* Y, int y_dtype, int64_t ld_y, hipStream_t stream);

// norm.hip
struct NormArgs {
  const void *x, *r;
  int64_t ldx, ldr, n;
  int d;
  const float* weight;
  double eps;
  void* h;
  int64_t ldh;
  uint8_t* codes;
  void* scales;
  float* rstd;
};
hipError_t rms_norm_launch(const NormArgs& a, int x_dtype, int r_dtype, int fmt, hipStream_t stream);

// norm_grad.hip
struct NormGradArgs {
  const void *dy, *h, *dh;
  int64_t ldy, ldh, lddh, n;
  int d;
  const float *rstd, *weight;
  void* dx;
  int64_t lddx;
  int accumulate;
  float* dweight;
  double* part;  // rows of d partial sums of dweight, one for each workgroup
};
size_t rms_norm_grad_ws_bytes(int64_t n, int64_t d);
hipError_t rms_norm_grad_launch(const NormGradArgs& a, int y_dtype, int h_dtype, hipStream_t stream);

// A result from its exact sum: times the token's scale, times the channel's (plus bias, 0 for none, in the same step), no
// less than low. Every kernel finishes by this, so results do not depend on the one that a size takes. The first product
// has fp32's range: it overflows for tokens of 2^105 and more only (a scale of 2^98 times a sum of 2^30).
__device__ __forceinline__ float int8_result(float sum, float token, float channel, float bias, float low) {
  const float y = fmaf(sum * token, channel, bias);
  return y < low ? low : y;  // NaN stays
}

}  // namespace gptq
