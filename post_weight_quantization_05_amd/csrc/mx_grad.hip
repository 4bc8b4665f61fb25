// Backward pass of a quantized linear layer on gfx950: dX = dY W (masked by the ReLU that made the layer's input)
// and dW = dY^T A with db = column sums of dY.
//
// The quantized operand's values (4 significant bits at most, times a power of two) are exact in bf16, so it is first
// written out in bf16 and the products run on the bf16 matrix cores, exact and summed in fp32.
//
// Simple form: a wave forms 32 x 32 of the result, its lanes loading their own elements of each step of 16 of the
// summed dimension. The quantized operand is the first one, so that a lane of the result holds four consecutive
// columns.
#include <algorithm>

#include "mx.h"

namespace gptq {

namespace {

// out[s][f] = sum_k F[k][f] S(k, s): S(k, s) = S[s][k] (GRAD_INPUT) or S[k][s] (weight gradient)
template <bool GRAD_INPUT, bool YBF16, int MASK>
__global__ __launch_bounds__(256) void k_mx_grad_simple(const uint16_t* __restrict__ F, int64_t ldf, int nf,
                                                        const uint16_t* __restrict__ S, int64_t lds, int ns, int nk,
                                                        const uint8_t* __restrict__ mc, const uint8_t* __restrict__ ms,
                                                        int accumulate, void* __restrict__ Y, int64_t ld) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 31, h = lane >> 5;
  const int tiles_f = (nf + 63) / 64;
  const int f0 = (blockIdx.x % tiles_f) * 64 + (wave & 1) * 32, s0 = (blockIdx.x / tiles_f) * 64 + (wave >> 1) * 32;
  if (f0 >= nf || s0 >= ns) return;
  const int f = min(f0 + r, nf - 1), s = min(s0 + r, ns - 1);
  f32x16 acc;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int k = 0; k < nk; k += 16) {
    bf16x8 a, b;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int kk = k + 8 * h + j;
      const bool ok = kk < nk;
      const uint16_t av = ok ? F[(int64_t)kk * ldf + f] : (uint16_t)0;
      const uint16_t bv = ok ? (GRAD_INPUT ? S[(int64_t)s * lds + kk] : S[(int64_t)kk * lds + s]) : (uint16_t)0;
      a[j] = __builtin_bit_cast(__bf16, av);
      b[j] = __builtin_bit_cast(__bf16, bv);
    }
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, acc, 0, 0, 0);
  }
  if (s0 + r >= ns) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = f0 + 8 * (i >> 2) + 4 * h + (i & 3);
    if (c >= nf) continue;
    float y = acc[i];
    if (MASK != 0) {
      const int kp = (nf + 127) / 128 * 128, srow = (nf + 511) / 512 * 16;
      uint32_t code;
      bool pos;
      if (MASK == 1) {
        code = mc[(int64_t)s * (kp / 2) + (c >> 1)] >> (4 * (c & 1)) & 15u;
        pos = code >= 1u && code <= 7u;
      } else {
        code = mc[(int64_t)s * kp + c];
        pos = code >= 1u && code <= 0x7Eu;
      }
      if (!pos || ms[(int64_t)s * srow + (c >> 5)] == 255) y = 0.f;
    }
    const int64_t at = (int64_t)s * ld + c;
    if (YBF16) {
      static_cast<uint16_t*>(Y)[at] = (uint16_t)bf16_bits(y);
    } else {
      float* p = static_cast<float*>(Y) + at;
      *p = accumulate ? *p + y : y;
    }
  }
}

__global__ __launch_bounds__(256) void k_colsum_simple(const uint16_t* __restrict__ S, int64_t ld, int64_t n, int cols,
                                                       int accumulate, float* __restrict__ db) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= cols) return;
  double sum = 0.0;
  for (int64_t k = 0; k < n; ++k) sum += (double)__uint_as_float((uint32_t)S[k * ld + c] << 16);
  db[c] = (float)(accumulate ? (double)db[c] + sum : sum);
}

}  // namespace

size_t mx_grad_input_ws_bytes(int64_t, int64_t in, int64_t out) { return align_up(out * ceil_div(in, 128) * 256, 256); }
size_t mx_grad_weight_ws_bytes(int64_t n, int64_t in, int64_t) { return align_up(n * ceil_div(in, 128) * 256, 256); }

hipError_t mx_grad_input_launch(const uint16_t* dY, int64_t ld_dy, int64_t n, const MxMatrix& w, const MxMatrix* mask,
                                void* dX, int dx_dtype, int64_t ld_dx, void* ws, hipStream_t stream) {
  const int64_t in = w.cols, ldf = ceil_div(in, 128) * 128;
  const hipError_t e = mx_dequantize_launch(w, ws, GPTQ_BF16, ldf, stream);
  if (e != hipSuccess) return e;
  const uint16_t* F = static_cast<const uint16_t*>(ws);
  const int64_t tiles_f = ceil_div(in, 64), rows_max = std::max<int64_t>(1, ((int64_t)1 << 23) / tiles_f) * 64;
  for (int64_t r = 0; r < n; r += rows_max) {
    const int64_t m = std::min(rows_max, n - r);
    const dim3 grid((unsigned)(tiles_f * ceil_div(m, 64)));
    const uint8_t* mc = mask ? mask->codes + r * mx_code_row(in, mask->fmt) : nullptr;
    const uint8_t* ms = mask ? mask->scales + r * mx_scale_row(in) : nullptr;
    void* y = static_cast<uint8_t*>(dX) + r * ld_dx * (dx_dtype == GPTQ_BF16 ? 2 : 4);
    const int kind = !mask ? 0 : mask->fmt == GPTQ_MX_E2M1 ? 1 : 2;
#define GPTQ_GO(B, M)                                                                                                \
  hipLaunchKernelGGL((k_mx_grad_simple<true, B, M>), grid, dim3(256), 0, stream, F, ldf, (int)in, dY + r * ld_dy,    \
                     ld_dy, (int)m, (int)w.rows, mc, ms, 0, y, ld_dx)
    if (dx_dtype == GPTQ_BF16) {
      if (kind == 0) GPTQ_GO(true, 0);
      else if (kind == 1) GPTQ_GO(true, 1);
      else GPTQ_GO(true, 2);
    } else {
      if (kind == 0) GPTQ_GO(false, 0);
      else if (kind == 1) GPTQ_GO(false, 1);
      else GPTQ_GO(false, 2);
    }
#undef GPTQ_GO
  }
  return hipGetLastError();
}

hipError_t mx_grad_weight_launch(const uint16_t* dY, int64_t ld_dy, int64_t out, const MxMatrix& a, int accumulate,
                                 void* dW, int dw_dtype, int64_t ld_dw, float* db, void* ws, hipStream_t stream) {
  const int64_t in = a.cols, ldf = ceil_div(in, 128) * 128;
  if (a.rows > 0) {
    const hipError_t e = mx_dequantize_launch(a, ws, GPTQ_BF16, ldf, stream);
    if (e != hipSuccess) return e;
  }
  const uint16_t* F = static_cast<const uint16_t*>(ws);
  const dim3 grid((unsigned)(ceil_div(in, 64) * ceil_div(out, 64)));
  if (dw_dtype == GPTQ_BF16)
    hipLaunchKernelGGL((k_mx_grad_simple<false, true, 0>), grid, dim3(256), 0, stream, F, ldf, (int)in, dY, ld_dy,
                       (int)out, (int)a.rows, nullptr, nullptr, 0, dW, ld_dw);
  else
    hipLaunchKernelGGL((k_mx_grad_simple<false, false, 0>), grid, dim3(256), 0, stream, F, ldf, (int)in, dY, ld_dy,
                       (int)out, (int)a.rows, nullptr, nullptr, accumulate, dW, ld_dw);
  if (db)
    hipLaunchKernelGGL(k_colsum_simple, dim3((unsigned)ceil_div(out, 256)), dim3(256), 0, stream, dY, ld_dy, a.rows,
                       (int)out, accumulate, db);
  return hipGetLastError();
}

}  // namespace gptq
