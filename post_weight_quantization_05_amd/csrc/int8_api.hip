// C ABI of the 8-bit integer operators and the norm: argument checks and launch. Every check runs on the host before
// anything is launched, so an argument error writes nothing.
#include <cmath>

#include "int8.h"

using namespace gptq;

namespace {

constexpr int64_t MAX_IN = 65536;
constexpr int64_t MAX_OUT = 1 << 20;
constexpr int64_t MAX_N = ((int64_t)1 << 31) - 1;

bool valid_dtype(int t) { return t == GPTQ_F32 || t == GPTQ_BF16; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned_to(const void* p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype == GPTQ_F32 ? 3 : 1)) == 0; }
bool valid_data(const void* p, int dtype) { return p && aligned_to(p, dtype); }
bool valid_codes(const int8_t* codes, const float* scales) {
  return codes && aligned16(codes) && valid_data(scales, GPTQ_F32);
}
bool valid_sizes(int64_t n, int64_t in, int64_t out) {
  return n >= 0 && n <= MAX_N && in >= 1 && in <= MAX_IN && out >= 1 && out <= MAX_OUT;
}
bool ws_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && have >= need && (reinterpret_cast<uintptr_t>(ws) & 255) == 0);
}
int hip_status(hipError_t e) { return e == hipSuccess ? GPTQ_OK : GPTQ_ERR_HIP; }
hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

int64_t gptq_int8_code_bytes_per_row(int64_t cols) { return (cols < 1 || cols > MAX_IN) ? 0 : int8_code_row(cols); }

int gptq_int8_quantize(const void* X, int x_dtype, int64_t n, int64_t in, int64_t ld_x, int8_t* codes, float* scales,
                       void* stream) {
  if (!valid_sizes(n, in, 1) || ld_x < in || !valid_dtype(x_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!valid_data(X, x_dtype) || !valid_codes(codes, scales)) return GPTQ_ERR_INVALID_ARG;
  return hip_status(int8_quantize_launch(X, x_dtype, n, in, ld_x, codes, scales, as_stream(stream)));
}

int gptq_int8_dequantize(const int8_t* codes, const float* scales, int64_t n, int64_t in, void* Y, int y_dtype,
                         int64_t ld_y, void* stream) {
  if (!valid_sizes(n, in, 1) || ld_y < in || !valid_dtype(y_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!valid_data(Y, y_dtype) || !valid_codes(codes, scales)) return GPTQ_ERR_INVALID_ARG;
  return hip_status(int8_dequantize_launch({codes, scales, n, in}, Y, y_dtype, ld_y, as_stream(stream)));
}

int gptq_int8_pad_codes(const int8_t* codes, int64_t out, int64_t in, int8_t* padded, void* stream) {
  if (!valid_sizes(0, in, out) || !codes || !padded || !aligned16(padded)) return GPTQ_ERR_INVALID_ARG;
  return hip_status(int8_pad_launch(codes, out, in, padded, as_stream(stream)));
}

size_t gptq_int8_matmul_workspace_bytes(int64_t n, int64_t in, int64_t out) {
  return valid_sizes(n, in, out) ? int8_matmul_ws_bytes(n, in, out) : 0;
}

int gptq_int8_matmul(const int8_t* a_codes, const float* a_scales, int64_t n, int64_t in, const int8_t* w_codes,
                     const float* w_scales, int64_t out, const float* bias, int relu, void* Y, int y_dtype, int64_t ld_y,
                     void* ws, size_t ws_bytes, void* stream) {
  if (!valid_sizes(n, in, out) || !valid_dtype(y_dtype) || ld_y < out) return GPTQ_ERR_INVALID_ARG;
  if (relu != 0 && relu != 1) return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!valid_codes(a_codes, a_scales) || !valid_codes(w_codes, w_scales) || !valid_data(Y, y_dtype))
    return GPTQ_ERR_INVALID_ARG;
  if (bias && !aligned_to(bias, GPTQ_F32)) return GPTQ_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, int8_matmul_ws_bytes(n, in, out))) return GPTQ_ERR_WORKSPACE;
  return hip_status(int8_matmul_launch({a_codes, a_scales, n, in}, {w_codes, w_scales, out, in}, bias, relu, Y, y_dtype,
                                       ld_y, ws, as_stream(stream)));
}

size_t gptq_int8_linear_workspace_bytes(int64_t n, int64_t in, int64_t out) {
  return valid_sizes(n, in, out) ? int8_linear_ws_bytes(n, in, out) : 0;
}

int gptq_int8_linear(const void* X, int x_dtype, int64_t n, int64_t in, int64_t ld_x, const int8_t* w_codes,
                     const float* w_scales, int64_t out, const float* bias, int relu, void* Y, int y_dtype, int64_t ld_y,
                     void* ws, size_t ws_bytes, void* stream) {
  if (!valid_sizes(n, in, out) || !valid_dtype(x_dtype) || !valid_dtype(y_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (ld_x < in || ld_y < out || (relu != 0 && relu != 1)) return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!valid_data(X, x_dtype) || !valid_codes(w_codes, w_scales) || !valid_data(Y, y_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (bias && !aligned_to(bias, GPTQ_F32)) return GPTQ_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, int8_linear_ws_bytes(n, in, out))) return GPTQ_ERR_WORKSPACE;
  return hip_status(int8_linear_launch(X, x_dtype, n, ld_x, {w_codes, w_scales, out, in}, bias, relu, Y, y_dtype, ld_y, ws,
                                       as_stream(stream)));
}

int gptq_rms_norm(const void* X, int x_dtype, int64_t ld_x, const void* R, int r_dtype, int64_t ld_r, int64_t n, int64_t d,
                  const float* weight, double eps, void* H, int64_t ld_h, int fmt, void* codes, void* scales, float* rstd,
                  void* stream) {
  if (!valid_sizes(n, d, 1) || ld_x < d || !valid_dtype(x_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (fmt != GPTQ_NORM_INT8 && fmt != GPTQ_NORM_E4M3) return GPTQ_ERR_INVALID_ARG;
  if (!(eps >= 1e-30) || !std::isfinite(eps)) return GPTQ_ERR_INVALID_ARG;
  if (R && (!valid_dtype(r_dtype) || ld_r < d || ld_h < d)) return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!valid_data(X, x_dtype) || !valid_data(weight, GPTQ_F32)) return GPTQ_ERR_INVALID_ARG;
  if (R && (!aligned_to(R, r_dtype) || !valid_data(H, r_dtype) || (H == R && ld_h != ld_r))) return GPTQ_ERR_INVALID_ARG;
  if (!codes || !aligned16(codes) || !scales) return GPTQ_ERR_INVALID_ARG;
  if (fmt == GPTQ_NORM_INT8 ? !aligned_to(scales, GPTQ_F32) : !aligned16(scales)) return GPTQ_ERR_INVALID_ARG;
  if (rstd && !aligned_to(rstd, GPTQ_F32)) return GPTQ_ERR_INVALID_ARG;
  const NormArgs a = {X, R, ld_x, ld_r, n, (int)d, weight, eps, H, ld_h, static_cast<uint8_t*>(codes), scales, rstd};
  return hip_status(rms_norm_launch(a, x_dtype, r_dtype, fmt, as_stream(stream)));
}

size_t gptq_rms_norm_grad_workspace_bytes(int64_t n, int64_t d) {
  return valid_sizes(n, d, 1) ? rms_norm_grad_ws_bytes(n, d) : 0;
}

int gptq_rms_norm_grad(const void* dY, int y_dtype, int64_t ld_dy, const void* h, int h_dtype, int64_t ld_h,
                       const float* rstd, const float* weight, const void* dH, int64_t ld_dh, int64_t n, int64_t d,
                       int accumulate, void* dX, int64_t ld_dx, float* dweight, void* ws, size_t ws_bytes, void* stream) {
  if (!valid_sizes(n, d, 1) || !valid_dtype(y_dtype) || !valid_dtype(h_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (ld_dy < d || ld_h < d || ld_dx < d || (dH && ld_dh < d)) return GPTQ_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return GPTQ_ERR_INVALID_ARG;
  if (!valid_data(dweight, GPTQ_F32)) return GPTQ_ERR_INVALID_ARG;
  if (n > 0) {
    if (!valid_data(dY, y_dtype) || !valid_data(h, h_dtype) || !valid_data(dX, h_dtype)) return GPTQ_ERR_INVALID_ARG;
    if (!valid_data(rstd, GPTQ_F32) || !valid_data(weight, GPTQ_F32)) return GPTQ_ERR_INVALID_ARG;
    if (dH && !aligned_to(dH, h_dtype)) return GPTQ_ERR_INVALID_ARG;
  } else if (accumulate) {
    return GPTQ_OK;
  }
  if (!ws_ok(ws, ws_bytes, rms_norm_grad_ws_bytes(n, d))) return GPTQ_ERR_WORKSPACE;
  const NormGradArgs a = {dY, h, dH, ld_dy, ld_h, ld_dh, n, (int)d, rstd, weight, dX, ld_dx, accumulate, dweight,
                          static_cast<double*>(ws)};
  return hip_status(rms_norm_grad_launch(a, y_dtype, h_dtype, as_stream(stream)));
}

}  // extern "C"
