// Y = A W^T (+ bias) (ReLU) with A (n x in, E2M1 or E4M3) and W (out x in, E2M1) in MX form, on the scaled matrix
// instructions of gfx950: v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 4- and 8-bit elements and applies each
// block's two scale bytes to its 32 products before they are added in fp32.
//
// Simple form: a wave forms 32 x 32 of Y, its lanes loading their own elements of each 64-column step. W is the
// first operand, so that a lane of the result holds four consecutive columns of Y.
//
// Lane l = 32 h + r of an operand holds row r: 4-bit elements of columns 32 h .. 32 h + 31 of the 64; 8-bit
// elements of columns 16 h .. 16 h + 15 and 32 + 16 h .. 32 + 16 h + 15; in both cases the scale byte of block h.
// (Found with an in-bounds check of the instruction's layout.)
#include <algorithm>

#include "mx.h"

namespace gptq {

namespace {

// Parts of an E4M3 operand whose exponents differ by at most 6: codes with the top exponent bit set, and the rest.
// The matrix core aligns the products of one instruction to their largest and drops what lies more than about 13
// bits below; with 7 exponents to each part nothing is dropped against E2M1 weights, so the sum is exact up to
// fp32 rounding.
__device__ __forceinline__ void split_e4m3(const i32x8& a, i32x8& hi, i32x8& lo) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t t = (uint32_t)a[q] & 0x40404040u;
    const uint32_t m = (t << 1) - (t >> 6);  // 0x7F in every byte whose top exponent bit is set
    hi[q] = (int)((uint32_t)a[q] & m);
    lo[q] = (int)((uint32_t)a[q] & ~m);
    hi[q] |= (int)((uint32_t)a[q] & 0x80808080u);
  }
}

template <int FMT, bool SPLIT, bool YBF16>
__global__ __launch_bounds__(256) void k_mx_matmul_simple(const uint8_t* __restrict__ ac, const uint8_t* __restrict__ as,
                                                          int n, const uint8_t* __restrict__ wc,
                                                          const uint8_t* __restrict__ wsc, int out, int kp, int64_t srow,
                                                          const float* __restrict__ bias, int relu,
                                                          void* __restrict__ Y, int64_t ld) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 31, h = lane >> 5;
  const int tiles_o = (out + 63) / 64;
  const int o0 = (blockIdx.x % tiles_o) * 64 + (wave & 1) * 32, t0 = (blockIdx.x / tiles_o) * 64 + (wave >> 1) * 32;
  if (o0 >= out || t0 >= n) return;
  const int o = min(o0 + r, out - 1), t = min(t0 + r, n - 1);  // rows past the end repeat the last; never stored
  const uint8_t* wp = wc + (int64_t)o * (kp / 2);
  const uint8_t* ap = ac + (int64_t)t * (FMT == GPTQ_MX_E2M1 ? kp / 2 : kp);
  const uint8_t *wsp = wsc + o * srow, *asp = as + t * srow;
  f32x16 acc;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  for (int k = 0; k < kp; k += 64) {
    i32x8 w = {0, 0, 0, 0, 0, 0, 0, 0}, a = {0, 0, 0, 0, 0, 0, 0, 0};
    const uint4 wv = *reinterpret_cast<const uint4*>(wp + k / 2 + 16 * h);
    w[0] = wv.x, w[1] = wv.y, w[2] = wv.z, w[3] = wv.w;
    const int sw = wsp[k / 32 + h], sa = asp[k / 32 + h];
    if (FMT == GPTQ_MX_E2M1) {
      const uint4 v = *reinterpret_cast<const uint4*>(ap + k / 2 + 16 * h);
      a[0] = v.x, a[1] = v.y, a[2] = v.z, a[3] = v.w;
      acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, a, acc, 4, 4, 0, sw, 0, sa);
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(ap + k + 16 * h);
      const uint4 u = *reinterpret_cast<const uint4*>(ap + k + 32 + 16 * h);
      a[0] = v.x, a[1] = v.y, a[2] = v.z, a[3] = v.w, a[4] = u.x, a[5] = u.y, a[6] = u.z, a[7] = u.w;
      if (SPLIT) {
        i32x8 hi, lo;
        split_e4m3(a, hi, lo);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, lo, acc, 4, 0, 0, sw, 0, sa);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, hi, acc, 4, 0, 0, sw, 0, sa);
      } else {
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, a, acc, 4, 0, 0, sw, 0, sa);
      }
    }
  }
  // result: register i of the lane holds column (of W's rows) 8 (i / 4) + 4 h + i % 4, token r
  if (t0 + r >= n) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = o0 + 8 * (i >> 2) + 4 * h + (i & 3);
    if (c >= out) continue;
    float y = acc[i];
    if (bias) y += bias[c];
    if (relu) y = relu_nan(y);
    const int64_t at = (int64_t)(t0 + r) * ld + c;
    if (YBF16) static_cast<uint16_t*>(Y)[at] = (uint16_t)bf16_bits(y);
    else static_cast<float*>(Y)[at] = y;
  }
}

}  // namespace

size_t mx_matmul_ws_bytes(int64_t, int64_t, int64_t, int) { return 0; }

hipError_t mx_matmul_launch(const MxMatrix& a, const MxMatrix& w, const float* bias, int relu, void* Y, int y_dtype,
                            int64_t ld_y, void*, hipStream_t stream) {
  const int kp = (int)ceil_div(a.cols, 128) * 128;
  const int64_t tiles_o = ceil_div(w.rows, 64), srow = mx_scale_row(a.cols);
  // at most 2^23 workgroups of 256 a launch
  const int64_t rows_max = std::max<int64_t>(1, ((int64_t)1 << 23) / tiles_o) * 64;
  for (int64_t r = 0; r < a.rows; r += rows_max) {
    const int64_t n = std::min(rows_max, a.rows - r);
    const dim3 grid((unsigned)(tiles_o * ceil_div(n, 64)));
    const uint8_t *ac = a.codes + r * mx_code_row(a.cols, a.fmt), *as = a.scales + r * srow;
    void* y = static_cast<uint8_t*>(Y) + r * ld_y * (y_dtype == GPTQ_BF16 ? 2 : 4);
#define GPTQ_GO(F, S, B)                                                                                              \
  hipLaunchKernelGGL((k_mx_matmul_simple<F, S, B>), grid, dim3(256), 0, stream, ac, as, (int)n, w.codes, w.scales,    \
                     (int)w.rows, kp, srow, bias, relu, y, ld_y)
    if (a.fmt == GPTQ_MX_E2M1) {
      if (y_dtype == GPTQ_BF16) GPTQ_GO(GPTQ_MX_E2M1, false, true);
      else GPTQ_GO(GPTQ_MX_E2M1, false, false);
    } else {
      if (y_dtype == GPTQ_BF16) GPTQ_GO(GPTQ_MX_E4M3, false, true);
      else GPTQ_GO(GPTQ_MX_E4M3, true, false);
    }
#undef GPTQ_GO
  }
  return hipGetLastError();
}

size_t mx_linear_ws_bytes(int64_t n, int64_t in, int64_t out, int act_fmt) {
  return align_up(n * mx_code_row(in, act_fmt), 256) + align_up(n * mx_scale_row(in), 256) +
         mx_matmul_ws_bytes(n, in, out, act_fmt);
}

hipError_t mx_linear_launch(const void* X, int x_dtype, int64_t n, int64_t ld_x, int act_fmt, const MxMatrix& w,
                            const float* bias, int relu, void* Y, int y_dtype, int64_t ld_y, void* ws,
                            hipStream_t stream) {
  uint8_t* codes = static_cast<uint8_t*>(ws);
  uint8_t* scales = codes + align_up(n * mx_code_row(w.cols, act_fmt), 256);
  uint8_t* rest = scales + align_up(n * mx_scale_row(w.cols), 256);
  const hipError_t e = mx_quantize_launch(X, x_dtype, n, w.cols, ld_x, act_fmt, codes, scales, stream);
  if (e != hipSuccess) return e;
  const MxMatrix a = {codes, scales, act_fmt, n, w.cols};
  return mx_matmul_launch(a, w, bias, relu, Y, y_dtype, ld_y, rest, stream);
}

}  // namespace gptq
