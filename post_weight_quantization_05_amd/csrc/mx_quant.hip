// MX quantization and its inverse on gfx950.
//
// For each block of 32 columns of a row: the scale exponent from the block's largest magnitude, then every
// element divided by the scale (a power of two, so exactly) and rounded to nearest-even in its 4 or 8 bits by the
// conversion instructions. Both kernels are one pass over memory: a wave takes units of one row x 512 columns
// (16 blocks), a lane 8 consecutive columns, four lanes a block.
#include <algorithm>

#include "mx_codec.h"

namespace gptq {

namespace {

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
  return v;
}

template <int FMT, bool XBF16>
__global__ __launch_bounds__(256) void k_mx_quantize(const void* __restrict__ X, int64_t ld, int in, int ks,
                                                     int64_t units, uint8_t* __restrict__ codes,
                                                     uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit >= units) return;
  const int64_t row = unit / ks;
  const int seg = (int)(unit - row * ks);
  const int c = seg * UNIT + lane * 8;
  const Chunk<XBF16> x = load_chunk<XBF16>(X, row * ld + c, c, in);
  const uint32_t byte = scale_byte<FMT>(quad_max(max_bits<XBF16>(chunk_max<XBF16>(x))));
  const int kp = (in + 127) / 128 * 128;
  const float scale = __uint_as_float(byte << 23);
  const bool nan = byte == 255u;
  if (c < kp) {
    if (FMT == GPTQ_MX_E2M1) {
      *reinterpret_cast<uint32_t*>(codes + row * (kp / 2) + c / 2) = nan ? 0u : encode4<XBF16>(x, scale);
    } else {
      const uint2 v = encode8<XBF16>(x, scale);
      *reinterpret_cast<uint2*>(codes + row * kp + c) = nan ? make_uint2(0u, 0u) : v;
    }
  }
  if ((lane & 3) == 0) scales[row * (ks * 16) + (c >> 5)] = (uint8_t)(c < in ? byte : 0u);
}

template <int FMT, bool YBF16>
__global__ __launch_bounds__(256) void k_mx_dequantize(const uint8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales, int in, int ks,
                                                       int64_t units, void* __restrict__ Y, int64_t ld) {
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit < units) dequantize_unit<FMT, YBF16>(codes, scales, in, ks, unit, Y, ld);
}

// A launch holds at most this many rows x segments, so that its grid stays below 2^32 work-items.
constexpr int64_t MAX_UNITS = (int64_t)1 << 25;

}  // namespace

hipError_t mx_quantize_launch(const void* X, int x_dtype, int64_t n, int64_t in, int64_t ld_x, int fmt, uint8_t* codes,
                              uint8_t* scales, hipStream_t stream) {
  const int ks = (int)ceil_div(in, UNIT);
  const bool b = x_dtype == GPTQ_BF16;
  const int64_t rows_max = MAX_UNITS / ks;
  for (int64_t r = 0; r < n; r += rows_max) {
    const int64_t units = std::min(rows_max, n - r) * ks;
    const unsigned grid = (unsigned)ceil_div(units, 4);
    const void* x = static_cast<const uint8_t*>(X) + r * ld_x * (b ? 2 : 4);
    uint8_t *c = codes + r * mx_code_row(in, fmt), *s = scales + r * mx_scale_row(in);
    const auto kernel = fmt == GPTQ_MX_E2M1 ? (b ? k_mx_quantize<GPTQ_MX_E2M1, true> : k_mx_quantize<GPTQ_MX_E2M1, false>)
                                            : (b ? k_mx_quantize<GPTQ_MX_E4M3, true> : k_mx_quantize<GPTQ_MX_E4M3, false>);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, stream, x, ld_x, (int)in, ks, units, c, s);
  }
  return hipGetLastError();
}

hipError_t mx_dequantize_launch(const MxMatrix& q, void* Y, int y_dtype, int64_t ld_y, hipStream_t stream) {
  const int ks = (int)ceil_div(q.cols, UNIT);
  const bool b = y_dtype == GPTQ_BF16;
  const int64_t rows_max = MAX_UNITS / ks;
  for (int64_t r = 0; r < q.rows; r += rows_max) {
    MxMatrix p = q;
    p.rows = std::min(rows_max, q.rows - r);
    p.codes += r * mx_code_row(q.cols, q.fmt);
    p.scales += r * mx_scale_row(q.cols);
    void* y = static_cast<uint8_t*>(Y) + r * ld_y * (b ? 2 : 4);
    const int64_t units = p.rows * ks;
    const unsigned grid = (unsigned)ceil_div(units, 4);
    const auto kernel = q.fmt == GPTQ_MX_E2M1
                            ? (b ? k_mx_dequantize<GPTQ_MX_E2M1, true> : k_mx_dequantize<GPTQ_MX_E2M1, false>)
                            : (b ? k_mx_dequantize<GPTQ_MX_E4M3, true> : k_mx_dequantize<GPTQ_MX_E4M3, false>);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, stream, p.codes, p.scales, (int)p.cols, ks, units, y, ld_y);
  }
  return hipGetLastError();
}

}  // namespace gptq
