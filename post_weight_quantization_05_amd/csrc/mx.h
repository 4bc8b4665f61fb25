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

// mx_few.hip: the same for at most MX_FEW tokens, in MX form or, where they are small enough, quantized on their way in.
// us of GPU time (E4M3) so / with a launch to quantize them, which also costs a call 4 us on the host: 1 x 4096 x 4096 4.8 /
// 5.5, 8 x 4096 x 4096 5.6 / 6.3, 4 x 4096 x 11008 10.4 / 9.7, but 12 x 11008 x 4096 13.4 / 11.2, 16 x 4096 x 11008 15.8 / 13.3.
constexpr int MX_FEW = 16;
static inline bool mx_few_fused(int64_t n, int64_t in) { return n <= MX_FEW && n * in <= 8 * 4096; }
hipError_t mx_matmul_few_launch(const MxMatrix& x, const MxMatrix& w, const float* bias, int relu, void* Y, int y_dtype,
                                int64_t ld_y, hipStream_t stream);
hipError_t mx_linear_few_launch(const void* X, int x_dtype, int64_t n, int64_t ld_x, int act_fmt, const MxMatrix& w,
                                const float* bias, int relu, void* Y, int y_dtype, int64_t ld_y, hipStream_t stream);

// mx_grad.hip: dX = dY W (masked), dW = dY^T A and db
size_t mx_grad_input_ws_bytes(int64_t n, int64_t in, int64_t out);
hipError_t mx_grad_input_launch(const uint16_t* dY, int64_t ld_dy, int64_t n, const MxMatrix& w, const MxMatrix* mask,
                                void* dX, int dx_dtype, int64_t ld_dx, void* ws, hipStream_t stream);
size_t mx_grad_weight_ws_bytes(int64_t n, int64_t in, int64_t out);
hipError_t mx_grad_weight_launch(const uint16_t* dY, int64_t ld_dy, int64_t out, const MxMatrix& a, int accumulate,
                                 void* dW, int dw_dtype, int64_t ld_dw, float* db, void* ws, hipStream_t stream);

typedef __attribute__((ext_vector_type(2))) int i32x2;
typedef __attribute__((ext_vector_type(4))) int i32x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;
typedef __attribute__((ext_vector_type(16))) int i32x16;
// 16 bytes at any address that their elements may have: global memory takes them at full width
typedef i32x4 __attribute__((aligned(2))) i32x4_any;
typedef f32x4 __attribute__((aligned(4))) f32x4_any;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(2))) short i16x2;
typedef __attribute__((ext_vector_type(2))) unsigned short u16x2;
typedef __attribute__((ext_vector_type(2))) float f32x2;

// bf16 bits of a float, to nearest, ties to even (NaN stays NaN)
__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) { return bf16_bits(lo) | (bf16_bits(hi) << 16); }

// Parts of an E4M3 fragment whose exponents differ by at most 7: codes with the top exponent bit set, and the rest.
// The matrix core aligns the products of a block to the largest of them and drops what lies more than about 13 bits below
// (256 x 6 - 256 x 6 + 1/8 x 1/2 comes out as 0); with half of the exponents to each part nothing is dropped against E2M1
// weights (which span 7 bits against each other), so the sum is exact up to fp32 rounding. Blocks are added in fp32, however
// far their scales lie apart. Two instructions a product cost twice the matrix cores' time: 2048 x 4096 x 11008 takes 143 to
// 169 us by the card's power, and 88 with one, whose results lie 2.6e-4 off.
__device__ __forceinline__ void split_e4m3(const i32x8& a, i32x8& hi, i32x8& lo) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t t = (uint32_t)a[q] & 0x40404040u;
    const uint32_t m = (t << 1) - (t >> 6);  // 0x7F in every byte whose top exponent bit is set
    hi[q] = (int)((uint32_t)a[q] & (m | 0x80808080u));
    lo[q] = (int)((uint32_t)a[q] & ~m);
  }
}

// max(y, 0) that keeps NaN
__device__ __forceinline__ float relu_nan(float y) { return y < 0.f ? 0.f : y; }

}  // namespace gptq
