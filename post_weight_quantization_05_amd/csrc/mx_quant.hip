// MX quantization and its inverse on gfx950.
//
// For each block of 32 columns of a row: the scale exponent from the block's largest magnitude, then every
// element divided by the scale (a power of two, so exactly) and rounded to nearest-even in its 4 or 8 bits by the
// conversion instructions. Both kernels are one pass over memory: a wave takes units of one row x 512 columns
// (16 blocks), a lane 8 consecutive columns, four lanes a block.
//
// The scale comes from integer work on the magnitude bits: they order like the magnitudes, with infinities and NaN
// above every finite value, so one maximum finds both the exponent and the blocks that are not finite.
#include <algorithm>

#include "mx.h"

namespace gptq {

namespace {

constexpr int UNIT = 512;  // columns per wave and unit: 64 lanes x 8

// byte of the block's scale from its largest magnitude's fp32 bits (sign cleared)
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7F800000u) return 255u;
  const int e = (int)(top >> 23);
  if (FMT == GPTQ_MX_E2M1) return (uint32_t)max(e - 2, 2);  // amax in [4, 8) x scale
  return (uint32_t)max(e - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), 10);  // amax in (224, 448] x scale
}

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
  return v;
}

// 8 columns of one lane, as fp32 bit pattern (fp32 input) or packed bf16 pairs
template <bool XBF16>
struct Chunk {
  uint32_t w[XBF16 ? 4 : 8];
};

template <bool XBF16, bool VEC>
__device__ __forceinline__ Chunk<XBF16> load_chunk(const void* __restrict__ X, int64_t off, int c, int in) {
  Chunk<XBF16> r;
  constexpr int W = XBF16 ? 4 : 8;
  if (VEC && c + 8 <= in) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(X) + off * (XBF16 ? 2 : 4));
#pragma unroll
    for (int q = 0; q < W / 4; ++q) {
      const uint4 v = p[q];
      r.w[4 * q] = v.x, r.w[4 * q + 1] = v.y, r.w[4 * q + 2] = v.z, r.w[4 * q + 3] = v.w;
    }
  } else if (XBF16) {
    const uint16_t* p = static_cast<const uint16_t*>(X) + off;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t lo = (c + 2 * q < in) ? p[2 * q] : 0u, hi = (c + 2 * q + 1 < in) ? p[2 * q + 1] : 0u;
      r.w[q] = lo | (hi << 16);
    }
  } else {
    const uint32_t* p = static_cast<const uint32_t*>(X) + off;
#pragma unroll
    for (int q = 0; q < 8; ++q) r.w[q < W ? q : 0] = (c + q < in) ? p[q] : 0u;
  }
  return r;
}

// largest magnitude of the 8 columns, as fp32 bits
template <bool XBF16>
__device__ __forceinline__ uint32_t chunk_top(const Chunk<XBF16>& x) {
  uint32_t t = 0;
  if (XBF16) {
#pragma unroll
    for (int q = 0; q < 4; ++q) t = max(t, max(x.w[q] & 0x7FFF0000u, (x.w[q] & 0x7FFFu) << 16));
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) t = max(t, x.w[XBF16 ? 0 : q] & 0x7FFFFFFFu);
  }
  return t;
}

template <bool XBF16>
__device__ __forceinline__ float chunk_at(const Chunk<XBF16>& x, int q) {
  if (XBF16) return __uint_as_float((q & 1) ? (x.w[q >> 1] & 0xFFFF0000u) : (x.w[q >> 1] << 16));
  return __uint_as_float(x.w[XBF16 ? 0 : q]);
}

// 8 E2M1 codes (one dword) of x / scale
template <bool XBF16>
__device__ __forceinline__ uint32_t encode4(const Chunk<XBF16>& x, float scale) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, chunk_at<XBF16>(x, 0), chunk_at<XBF16>(x, 1), scale, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, chunk_at<XBF16>(x, 2), chunk_at<XBF16>(x, 3), scale, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, chunk_at<XBF16>(x, 4), chunk_at<XBF16>(x, 5), scale, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, chunk_at<XBF16>(x, 6), chunk_at<XBF16>(x, 7), scale, 3);
  return c;
}

// 8 E4M3 codes (two dwords) of x / scale
template <bool XBF16>
__device__ __forceinline__ uint2 encode8(const Chunk<XBF16>& x, float scale) {
  i16x2 lo = {0, 0}, hi = {0, 0};
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, chunk_at<XBF16>(x, 0), chunk_at<XBF16>(x, 1), scale, false);
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, chunk_at<XBF16>(x, 2), chunk_at<XBF16>(x, 3), scale, true);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, chunk_at<XBF16>(x, 4), chunk_at<XBF16>(x, 5), scale, false);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, chunk_at<XBF16>(x, 6), chunk_at<XBF16>(x, 7), scale, true);
  return make_uint2(__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi));
}

template <int FMT, bool XBF16, bool VEC>
__global__ __launch_bounds__(256) void k_mx_quantize(const void* __restrict__ X, int64_t ld, int in, int ks,
                                                     int64_t units, uint8_t* __restrict__ codes,
                                                     uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit >= units) return;
  const int64_t row = unit / ks;
  const int seg = (int)(unit - row * ks);
  const int c = seg * UNIT + lane * 8;
  const Chunk<XBF16> x = load_chunk<XBF16, VEC>(X, row * ld + c, c, in);
  const uint32_t byte = scale_byte<FMT>(quad_max(chunk_top<XBF16>(x)));
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

// 8 codes of a lane to 8 values
template <int FMT>
__device__ __forceinline__ void decode8(const uint2 v, float scale, float (&y)[8]) {
  if (FMT == GPTQ_MX_E2M1) {
#define GPTQ_DEC4(S)                                                           \
  {                                                                            \
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(v.x, scale, S);   \
    y[2 * S] = d[0], y[2 * S + 1] = d[1];                                      \
  }
    GPTQ_DEC4(0) GPTQ_DEC4(1) GPTQ_DEC4(2) GPTQ_DEC4(3)
#undef GPTQ_DEC4
  } else {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(v.x, scale, false);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(v.x, scale, true);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(v.y, scale, false);
    const f32x2 e = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(v.y, scale, true);
    y[0] = a[0], y[1] = a[1], y[2] = b[0], y[3] = b[1], y[4] = d[0], y[5] = d[1], y[6] = e[0], y[7] = e[1];
  }
}

template <int FMT, bool YBF16, bool VEC>
__global__ __launch_bounds__(256) void k_mx_dequantize(const uint8_t* __restrict__ codes,
                                                       const uint8_t* __restrict__ scales, int in, int ks,
                                                       int64_t units, void* __restrict__ Y, int64_t ld) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit >= units) return;
  const int64_t row = unit / ks;
  const int seg = (int)(unit - row * ks);
  const int c = seg * UNIT + lane * 8;
  if (c >= in) return;
  const int kp = (in + 127) / 128 * 128;
  uint2 v = make_uint2(0u, 0u);
  if (FMT == GPTQ_MX_E2M1) v.x = *reinterpret_cast<const uint32_t*>(codes + row * (kp / 2) + c / 2);
  else v = *reinterpret_cast<const uint2*>(codes + row * kp + c);
  const uint32_t byte = scales[row * (ks * 16) + (c >> 5)];
  float y[8];
  decode8<FMT>(v, __uint_as_float(byte << 23), y);
  if (byte == 255u) {
#pragma unroll
    for (int q = 0; q < 8; ++q) y[q] = __uint_as_float(0x7FC00000u);
  }
  if (YBF16) {
    uint16_t* p = static_cast<uint16_t*>(Y) + row * ld + c;
    if (VEC && c + 8 <= in) {
      *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]), bf16_pair(y[4], y[5]),
                                                bf16_pair(y[6], y[7]));
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < in) p[q] = (uint16_t)bf16_bits(y[q]);
    }
  } else {
    float* p = static_cast<float*>(Y) + row * ld + c;
    if (VEC && c + 8 <= in) {
      reinterpret_cast<float4*>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < in) p[q] = y[q];
    }
  }
}

template <int FMT, bool B>
void quantize_go(bool vec, unsigned grid, hipStream_t stream, const void* X, int64_t ld, int in, int ks, int64_t units,
                 uint8_t* codes, uint8_t* scales) {
  if (vec)
    hipLaunchKernelGGL((k_mx_quantize<FMT, B, true>), dim3(grid), dim3(256), 0, stream, X, ld, in, ks, units, codes, scales);
  else
    hipLaunchKernelGGL((k_mx_quantize<FMT, B, false>), dim3(grid), dim3(256), 0, stream, X, ld, in, ks, units, codes, scales);
}

template <int FMT, bool B>
void dequantize_go(bool vec, unsigned grid, hipStream_t stream, const MxMatrix& q, int ks, int64_t units, void* Y,
                   int64_t ld) {
  if (vec)
    hipLaunchKernelGGL((k_mx_dequantize<FMT, B, true>), dim3(grid), dim3(256), 0, stream, q.codes, q.scales, (int)q.cols,
                       ks, units, Y, ld);
  else
    hipLaunchKernelGGL((k_mx_dequantize<FMT, B, false>), dim3(grid), dim3(256), 0, stream, q.codes, q.scales,
                       (int)q.cols, ks, units, Y, ld);
}

// A launch holds at most this many rows x segments, so that its grid stays below 2^32 work-items.
constexpr int64_t MAX_UNITS = (int64_t)1 << 25;

}  // namespace

hipError_t mx_quantize_launch(const void* X, int x_dtype, int64_t n, int64_t in, int64_t ld_x, int fmt, uint8_t* codes,
                              uint8_t* scales, hipStream_t stream) {
  const int ks = (int)ceil_div(in, UNIT);
  const bool vec = vec_rows(X, ld_x, x_dtype), b = x_dtype == GPTQ_BF16;
  const int64_t rows_max = MAX_UNITS / ks;
  for (int64_t r = 0; r < n; r += rows_max) {
    const int64_t units = std::min(rows_max, n - r) * ks;
    const unsigned grid = (unsigned)ceil_div(units, 4);
    const void* x = static_cast<const uint8_t*>(X) + r * ld_x * (b ? 2 : 4);
    uint8_t *c = codes + r * mx_code_row(in, fmt), *s = scales + r * mx_scale_row(in);
    if (fmt == GPTQ_MX_E2M1)
      b ? quantize_go<GPTQ_MX_E2M1, true>(vec, grid, stream, x, ld_x, (int)in, ks, units, c, s)
        : quantize_go<GPTQ_MX_E2M1, false>(vec, grid, stream, x, ld_x, (int)in, ks, units, c, s);
    else
      b ? quantize_go<GPTQ_MX_E4M3, true>(vec, grid, stream, x, ld_x, (int)in, ks, units, c, s)
        : quantize_go<GPTQ_MX_E4M3, false>(vec, grid, stream, x, ld_x, (int)in, ks, units, c, s);
  }
  return hipGetLastError();
}

hipError_t mx_dequantize_launch(const MxMatrix& q, void* Y, int y_dtype, int64_t ld_y, hipStream_t stream) {
  const int ks = (int)ceil_div(q.cols, UNIT);
  const bool vec = vec_rows(Y, ld_y, y_dtype), b = y_dtype == GPTQ_BF16;
  const int64_t rows_max = MAX_UNITS / ks;
  for (int64_t r = 0; r < q.rows; r += rows_max) {
    MxMatrix p = q;
    p.rows = std::min(rows_max, q.rows - r);
    p.codes += r * mx_code_row(q.cols, q.fmt);
    p.scales += r * mx_scale_row(q.cols);
    void* y = static_cast<uint8_t*>(Y) + r * ld_y * (b ? 2 : 4);
    const int64_t units = p.rows * ks;
    const unsigned grid = (unsigned)ceil_div(units, 4);
    if (q.fmt == GPTQ_MX_E2M1)
      b ? dequantize_go<GPTQ_MX_E2M1, true>(vec, grid, stream, p, ks, units, y, ld_y)
        : dequantize_go<GPTQ_MX_E2M1, false>(vec, grid, stream, p, ks, units, y, ld_y);
    else
      b ? dequantize_go<GPTQ_MX_E4M3, true>(vec, grid, stream, p, ks, units, y, ld_y)
        : dequantize_go<GPTQ_MX_E4M3, false>(vec, grid, stream, p, ks, units, y, ld_y);
  }
  return hipGetLastError();
}

}  // namespace gptq
