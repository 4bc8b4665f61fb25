// Y = A W^T s_a s_w (+ bias) (ReLU) with A (n x in) and W (out x in) in 8-bit integers, on v_mfma_i32_32x32x32_i8: sums are
// whole numbers of at most 128^2 x 65536 = 2^30 and exact in 32 bits.
//
// W is the first operand, so that a lane of the result holds four consecutive columns of Y. Lane l of an operand holds row
// l % 32, columns 16 (l / 32) .. + 15 of the 32.
#include <algorithm>

#include "int8.h"

namespace gptq {

namespace {

struct MatmulArgs {
  const int8_t *ac, *wc;
  const float *as, *ws, *bias;
  void* Y;
  int64_t n, ld;
  int kp, out, relu;
};

// a workgroup forms 64 x 64, each wave 32 x 32, operands straight from memory
template <bool YBF16>
__global__ __launch_bounds__(256) void k_int8_matmul(const MatmulArgs g) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 31, h = lane >> 5;
  const int64_t row = (int64_t)blockIdx.y * 64 + (wave >> 1) * 32 + r;
  const int o0 = blockIdx.x * 64 + (wave & 1) * 32;
  const int8_t* a = g.ac + min(row, g.n - 1) * g.kp + 16 * h;
  const int8_t* w = g.wc + (int64_t)min(o0 + r, g.out - 1) * g.kp + 16 * h;
  i32x16 acc = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
  for (int k = 0; k < g.kp; k += 32)
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(*reinterpret_cast<const i32x4*>(w + k), *reinterpret_cast<const i32x4*>(a + k),
                                                acc, 0, 0, 0);
  if (row >= g.n) return;
  const float s = g.as[row];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = o0 + 8 * (i / 4) + 4 * h + i % 4;
    if (c >= g.out) continue;
    float y = (float)acc[i] * s * g.ws[c];
    if (g.bias) y += g.bias[c];
    if (g.relu) y = relu_nan(y);
    if (YBF16) static_cast<uint16_t*>(g.Y)[row * g.ld + c] = (uint16_t)bf16_bits(y);
    else static_cast<float*>(g.Y)[row * g.ld + c] = y;
  }
}

}  // namespace

size_t int8_matmul_ws_bytes(int64_t n, int64_t in, int64_t out) { return 0; }

hipError_t int8_matmul_launch(const Int8Matrix& a, const Int8Matrix& w, const float* bias, int relu, void* Y, int y_dtype,
                              int64_t ld_y, void* ws, hipStream_t stream) {
  MatmulArgs g = {};
  g.kp = (int)int8_code_row(a.cols);
  g.wc = w.codes, g.ws = w.scales, g.bias = bias, g.ld = ld_y, g.out = (int)w.rows, g.relu = relu;
  constexpr int64_t ROWS_MAX = 64 * 256;
  for (int64_t r = 0; r < a.rows; r += ROWS_MAX) {
    g.n = std::min(ROWS_MAX, a.rows - r);
    g.ac = a.codes + r * g.kp, g.as = a.scales + r;
    g.Y = static_cast<uint8_t*>(Y) + r * ld_y * (y_dtype == GPTQ_BF16 ? 2 : 4);
    const dim3 grid((unsigned)ceil_div(w.rows, 64), (unsigned)ceil_div(g.n, 64));
    hipLaunchKernelGGL(y_dtype == GPTQ_BF16 ? k_int8_matmul<true> : k_int8_matmul<false>, grid, dim3(256), 0, stream, g);
  }
  return hipGetLastError();
}

size_t int8_linear_ws_bytes(int64_t n, int64_t in, int64_t out) {
  return align_up(n * int8_code_row(in), 256) + align_up(n * 4, 256) + int8_matmul_ws_bytes(n, in, out);
}

hipError_t int8_linear_launch(const void* X, int x_dtype, int64_t n, int64_t ld_x, const Int8Matrix& w, const float* bias,
                              int relu, void* Y, int y_dtype, int64_t ld_y, void* ws, hipStream_t stream) {
  int8_t* codes = static_cast<int8_t*>(ws);
  float* scales = reinterpret_cast<float*>(codes + align_up(n * int8_code_row(w.cols), 256));
  uint8_t* rest = reinterpret_cast<uint8_t*>(scales) + align_up(n * 4, 256);
  const hipError_t e = int8_quantize_launch(X, x_dtype, n, w.cols, ld_x, codes, scales, stream);
  if (e != hipSuccess) return e;
  const Int8Matrix a = {codes, scales, n, w.cols};
  return int8_matmul_launch(a, w, bias, relu, Y, y_dtype, ld_y, rest, stream);
}

}  // namespace gptq
