// Shared definitions of the MX (microscaled) operators.
#pragma once

#include "../../include/gptq_mi355x_mx.h"
#include "common.h"

namespace gptq {

constexpr int MX_BLOCK = 32;  // columns that share a scale

static inline int64_t mx_code_row(int64_t cols, int fmt) { return ceil_div(cols, 128) * (fmt == GPTQ_MX_E2M1 ? 64 : 128); }
static inline int64_t mx_scale_row(int64_t cols) { return ceil_div(cols, 512) * 16; }

// every row of p starts at a 16-byte aligned address
static inline bool vec_rows(const void* p, int64_t ld, int dtype) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * (dtype == GPTQ_F32 ? 4 : 2)) % 16 == 0;
}

// One MX operand: rows of codes and scales at their fixed row lengths.
struct MxMatrix {
  const uint8_t* codes;
  const uint8_t* scales;
  int fmt;
  int64_t rows, cols;
};

// mx_quant.hip
hipError_t mx_quantize_launch(const void* X, int x_dtype, int64_t n, int64_t in, int64_t ld_x, int fmt, uint8_t* codes,
                              uint8_t* scales, hipStream_t stream);
hipError_t mx_dequantize_launch(const MxMatrix& q, void* Y, int y_dtype, int64_t ld_y, hipStream_t stream);

// mx_gemm.hip: Y = A W^T (+ bias) (ReLU)
size_t mx_matmul_ws_bytes(int64_t n, int64_t in, int64_t out, int a_fmt);
hipError_t mx_matmul_launch(const MxMatrix& a, const MxMatrix& w, const float* bias, int relu, void* Y, int y_dtype,
                            int64_t ld_y, void* ws, hipStream_t stream);
size_t mx_linear_ws_bytes(int64_t n, int64_t in, int64_t out, int act_fmt);
hipError_t mx_linear_launch(const void* X, int x_dtype, int64_t n, int64_t ld_x, int act_fmt, const MxMatrix& w,
                            const float* bias, int relu, void* Y, int y_dtype, int64_t ld_y, void* ws,
                            hipStream_t stream);

// mx_grad.hip: dX = dY W (masked), dW = dY^T A and db
size_t mx_grad_input_ws_bytes(int64_t n, int64_t in, int64_t out);
hipError_t mx_grad_input_launch(const uint16_t* dY, int64_t ld_dy, int64_t n, const MxMatrix& w, const MxMatrix* mask,
                                void* dX, int dx_dtype, int64_t ld_dx, void* ws, hipStream_t stream);
size_t mx_grad_weight_ws_bytes(int64_t n, int64_t in, int64_t out);
hipError_t mx_grad_weight_launch(const uint16_t* dY, int64_t ld_dy, int64_t out, const MxMatrix& a, int accumulate,
                                 void* dW, int dw_dtype, int64_t ld_dw, float* db, void* ws, hipStream_t stream);

typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(2))) short i16x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;

// bf16 bits of a float, to nearest, ties to even (NaN stays NaN)
__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) { return bf16_bits(lo) | (bf16_bits(hi) << 16); }

// max(y, 0) that keeps NaN
__device__ __forceinline__ float relu_nan(float y) { return y < 0.f ? 0.f : y; }

}  // namespace gptq
