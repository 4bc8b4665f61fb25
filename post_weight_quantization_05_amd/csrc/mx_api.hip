// C ABI of the MX operators: argument checks and launch. Every check runs on the host before anything is
// launched, so an argument error writes nothing.
#include "mx.h"

using namespace gptq;

namespace {

constexpr int64_t MAX_IN = 65536;
constexpr int64_t MAX_OUT = 1 << 20;
constexpr int64_t MAX_N = ((int64_t)1 << 31) - 1;

bool valid_dtype(int t) { return t == GPTQ_F32 || t == GPTQ_BF16; }
bool valid_fmt(int f) { return f == GPTQ_MX_E2M1 || f == GPTQ_MX_E4M3; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool aligned_to(const void* p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype == GPTQ_F32 ? 3 : 1)) == 0; }
bool valid_codes(const uint8_t* codes, const uint8_t* scales) {
  return codes && scales && aligned16(codes) && aligned16(scales);
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

int64_t gptq_mx_code_bytes_per_row(int64_t cols, int fmt) {
  return (cols < 1 || cols > MAX_IN || !valid_fmt(fmt)) ? 0 : mx_code_row(cols, fmt);
}

int64_t gptq_mx_scale_bytes_per_row(int64_t cols) { return (cols < 1 || cols > MAX_IN) ? 0 : mx_scale_row(cols); }

int gptq_mx_quantize(const void* X, int x_dtype, int64_t n, int64_t in, int64_t ld_x, int fmt, uint8_t* codes,
                     uint8_t* scales, void* stream) {
  if (!valid_sizes(n, in, 1) || ld_x < in || !valid_dtype(x_dtype) || !valid_fmt(fmt)) return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!X || !aligned_to(X, x_dtype) || !valid_codes(codes, scales)) return GPTQ_ERR_INVALID_ARG;
  return hip_status(mx_quantize_launch(X, x_dtype, n, in, ld_x, fmt, codes, scales, as_stream(stream)));
}

int gptq_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int fmt, int64_t n, int64_t in, void* Y,
                       int y_dtype, int64_t ld_y, void* stream) {
  if (!valid_sizes(n, in, 1) || ld_y < in || !valid_dtype(y_dtype) || !valid_fmt(fmt)) return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!Y || !aligned_to(Y, y_dtype) || !valid_codes(codes, scales)) return GPTQ_ERR_INVALID_ARG;
  const MxMatrix q = {codes, scales, fmt, n, in};
  return hip_status(mx_dequantize_launch(q, Y, y_dtype, ld_y, as_stream(stream)));
}

size_t gptq_mx_matmul_workspace_bytes(int64_t n, int64_t in, int64_t out, int a_fmt) {
  return (valid_sizes(n, in, out) && valid_fmt(a_fmt)) ? mx_matmul_ws_bytes(n, in, out, a_fmt) : 0;
}

int gptq_mx_matmul(const uint8_t* a_codes, const uint8_t* a_scales, int a_fmt, int64_t n, int64_t in,
                   const uint8_t* w_codes, const uint8_t* w_scales, int64_t out, const float* bias, int relu,
                   void* Y, int y_dtype, int64_t ld_y, void* ws, size_t ws_bytes, void* stream) {
  if (!valid_sizes(n, in, out) || !valid_fmt(a_fmt) || !valid_dtype(y_dtype) || ld_y < out) return GPTQ_ERR_INVALID_ARG;
  if (relu != 0 && relu != 1) return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!valid_codes(a_codes, a_scales) || !valid_codes(w_codes, w_scales) || !Y || !aligned_to(Y, y_dtype))
    return GPTQ_ERR_INVALID_ARG;
  if (bias && !aligned_to(bias, GPTQ_F32)) return GPTQ_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, mx_matmul_ws_bytes(n, in, out, a_fmt))) return GPTQ_ERR_WORKSPACE;
  const MxMatrix a = {a_codes, a_scales, a_fmt, n, in}, w = {w_codes, w_scales, GPTQ_MX_E2M1, out, in};
  return hip_status(mx_matmul_launch(a, w, bias, relu, Y, y_dtype, ld_y, ws, as_stream(stream)));
}

size_t gptq_mx_linear_workspace_bytes(int64_t n, int64_t in, int64_t out, int act_fmt) {
  return (valid_sizes(n, in, out) && valid_fmt(act_fmt)) ? mx_linear_ws_bytes(n, in, out, act_fmt) : 0;
}

int gptq_mx_linear(const void* X, int x_dtype, int64_t n, int64_t in, int64_t ld_x, int act_fmt,
                   const uint8_t* w_codes, const uint8_t* w_scales, int64_t out, const float* bias, int relu,
                   void* Y, int y_dtype, int64_t ld_y, void* ws, size_t ws_bytes, void* stream) {
  if (!valid_sizes(n, in, out) || !valid_fmt(act_fmt) || !valid_dtype(x_dtype) || !valid_dtype(y_dtype))
    return GPTQ_ERR_INVALID_ARG;
  if (ld_x < in || ld_y < out || (relu != 0 && relu != 1)) return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!X || !aligned_to(X, x_dtype) || !valid_codes(w_codes, w_scales) || !Y || !aligned_to(Y, y_dtype))
    return GPTQ_ERR_INVALID_ARG;
  if (bias && !aligned_to(bias, GPTQ_F32)) return GPTQ_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, mx_linear_ws_bytes(n, in, out, act_fmt))) return GPTQ_ERR_WORKSPACE;
  const MxMatrix w = {w_codes, w_scales, GPTQ_MX_E2M1, out, in};
  return hip_status(mx_linear_launch(X, x_dtype, n, ld_x, act_fmt, w, bias, relu, Y, y_dtype, ld_y, ws,
                                     as_stream(stream)));
}

size_t gptq_mx_grad_input_workspace_bytes(int64_t n, int64_t in, int64_t out) {
  return valid_sizes(n, in, out) ? mx_grad_input_ws_bytes(n, in, out) : 0;
}

int gptq_mx_grad_input(const void* dY, int64_t ld_dy, int64_t n, int64_t out, const uint8_t* w_codes,
                       const uint8_t* w_scales, int64_t in, const uint8_t* mask_codes, const uint8_t* mask_scales,
                       int mask_fmt, void* dX, int dx_dtype, int64_t ld_dx, void* ws, size_t ws_bytes, void* stream) {
  if (!valid_sizes(n, in, out) || ld_dy < out || ld_dx < in || !valid_dtype(dx_dtype)) return GPTQ_ERR_INVALID_ARG;
  if (mask_codes && !valid_fmt(mask_fmt)) return GPTQ_ERR_INVALID_ARG;
  if (n == 0) return GPTQ_OK;
  if (!dY || !aligned_to(dY, GPTQ_BF16) || !valid_codes(w_codes, w_scales) || !dX || !aligned_to(dX, dx_dtype))
    return GPTQ_ERR_INVALID_ARG;
  if (mask_codes && !valid_codes(mask_codes, mask_scales)) return GPTQ_ERR_INVALID_ARG;
  if (!ws_ok(ws, ws_bytes, mx_grad_input_ws_bytes(n, in, out))) return GPTQ_ERR_WORKSPACE;
  const MxMatrix w = {w_codes, w_scales, GPTQ_MX_E2M1, out, in}, m = {mask_codes, mask_scales, mask_fmt, n, in};
  return hip_status(mx_grad_input_launch(static_cast<const uint16_t*>(dY), ld_dy, n, w, mask_codes ? &m : nullptr, dX,
                                         dx_dtype, ld_dx, ws, as_stream(stream)));
}

size_t gptq_mx_grad_weight_workspace_bytes(int64_t n, int64_t in, int64_t out) {
  return valid_sizes(n, in, out) ? mx_grad_weight_ws_bytes(n, in, out) : 0;
}

int gptq_mx_grad_weight(const void* dY, int64_t ld_dy, int64_t n, int64_t out, const uint8_t* a_codes,
                        const uint8_t* a_scales, int a_fmt, int64_t in, int accumulate, void* dW, int dw_dtype,
                        int64_t ld_dw, float* db, void* ws, size_t ws_bytes, void* stream) {
  if (!valid_sizes(n, in, out) || ld_dy < out || ld_dw < in || !valid_dtype(dw_dtype) || !valid_fmt(a_fmt))
    return GPTQ_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return GPTQ_ERR_INVALID_ARG;
  if (!dW || !aligned_to(dW, dw_dtype) || (db && !aligned_to(db, GPTQ_F32))) return GPTQ_ERR_INVALID_ARG;
  if (n > 0 && (!dY || !aligned_to(dY, GPTQ_BF16) || !valid_codes(a_codes, a_scales))) return GPTQ_ERR_INVALID_ARG;
  if (accumulate && dw_dtype != GPTQ_F32) return GPTQ_ERR_UNSUPPORTED;
  if (n == 0 && accumulate) return GPTQ_OK;
  if (!ws_ok(ws, ws_bytes, mx_grad_weight_ws_bytes(n, in, out))) return GPTQ_ERR_WORKSPACE;
  const MxMatrix a = {a_codes, a_scales, a_fmt, n, in};
  return hip_status(mx_grad_weight_launch(static_cast<const uint16_t*>(dY), ld_dy, out, a, accumulate, dW, dw_dtype,
                                          ld_dw, db, ws, as_stream(stream)));
}

}  // extern "C"
