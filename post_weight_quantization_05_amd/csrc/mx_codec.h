// Encoding and decoding of MX elements, a lane holding 8 consecutive columns of a row.
//
// The scale comes from integer work on the magnitude bits: they order like the magnitudes, with infinities and NaN
// above every finite value, so one maximum finds both the exponent and the blocks that are not finite.
#pragma once

#include "mx.h"

namespace gptq {

// byte of the block's scale from its largest magnitude's fp32 bits (sign cleared)
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  if (top >= 0x7F800000u) return 255u;
  const int e = (int)(top >> 23);
  if (FMT == GPTQ_MX_E2M1) return (uint32_t)max(e - 2, 2);  // amax in [4, 8) x scale
  return (uint32_t)max(e - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), 10);  // amax in (224, 448] x scale
}

// 8 columns of one lane, as fp32 bit pattern (fp32 input) or packed bf16 pairs
template <bool XBF16>
struct Chunk {
  uint32_t w[XBF16 ? 4 : 8];
};

// columns c .. c + 7 of a row of `in`, zeros behind the last
template <bool XBF16>
__device__ __forceinline__ Chunk<XBF16> load_chunk(const void* __restrict__ X, int64_t off, int c, int in) {
  Chunk<XBF16> r;
  constexpr int W = XBF16 ? 4 : 8;
  if (c + 8 <= in) {
    const i32x4_any* p = reinterpret_cast<const i32x4_any*>(static_cast<const uint8_t*>(X) + off * (XBF16 ? 2 : 4));
#pragma unroll
    for (int q = 0; q < W / 4; ++q) {
      const i32x4 v = p[q];
#pragma unroll
      for (int e = 0; e < 4; ++e) r.w[4 * q + e] = (uint32_t)v[e];
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

// largest magnitudes of the 8 columns, packed: fp32 bits, or two bf16 (even and odd columns) side by side
template <bool XBF16>
__device__ __forceinline__ uint32_t chunk_max(const Chunk<XBF16>& x) {
  if constexpr (XBF16) {
    u16x2 t = {0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q) t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, x.w[q] & 0x7FFF7FFFu));
    return __builtin_bit_cast(uint32_t, t);
  } else {
    uint32_t t = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) t = max(t, x.w[q] & 0x7FFFFFFFu);
    return t;
  }
}
template <bool XBF16>
__device__ __forceinline__ uint32_t max_join(uint32_t a, uint32_t b) {
  if constexpr (XBF16)
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
  else
    return max(a, b);
}
// the largest of them as fp32 bits
template <bool XBF16>
__device__ __forceinline__ uint32_t max_bits(uint32_t t) {
  return XBF16 ? max(t & 0xFFFF0000u, t << 16) : t;
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
#define GPTQ_ENC4(S)                                                                                                  \
  if constexpr (XBF16) c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, x.w[S]), scale, S); \
  else c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, chunk_at<XBF16>(x, 2 * S), chunk_at<XBF16>(x, 2 * S + 1), scale, S);
  GPTQ_ENC4(0) GPTQ_ENC4(1) GPTQ_ENC4(2) GPTQ_ENC4(3)
#undef GPTQ_ENC4
  return c;
}

// 8 E4M3 codes (two dwords) of x / scale
template <bool XBF16>
__device__ __forceinline__ uint2 encode8(const Chunk<XBF16>& x, float scale) {
  i16x2 v[2] = {{0, 0}, {0, 0}};
#define GPTQ_ENC8(S, D, HI)                                                                                             \
  if constexpr (XBF16) v[D] = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(v[D], __builtin_bit_cast(bf16x2, x.w[S]), scale, HI); \
  else v[D] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(v[D], chunk_at<XBF16>(x, 2 * S), chunk_at<XBF16>(x, 2 * S + 1), scale, HI);
  GPTQ_ENC8(0, 0, false) GPTQ_ENC8(1, 0, true) GPTQ_ENC8(2, 1, false) GPTQ_ENC8(3, 1, true)
#undef GPTQ_ENC8
  return make_uint2(__builtin_bit_cast(uint32_t, v[0]), __builtin_bit_cast(uint32_t, v[1]));
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

// A wave's unit: 512 columns of a row, 64 lanes x 8. unit = row * ks + 512-column segment.
constexpr int UNIT = 512;
template <int FMT, bool YBF16>
__device__ __forceinline__ void dequantize_unit(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                                                int in, int ks, int64_t unit, void* __restrict__ Y, int64_t ld) {
  const int lane = threadIdx.x & 63;
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
    if (c + 8 <= in) {
      *reinterpret_cast<i32x4_any*>(p) = (i32x4){(int)bf16_pair(y[0], y[1]), (int)bf16_pair(y[2], y[3]),
                                                 (int)bf16_pair(y[4], y[5]), (int)bf16_pair(y[6], y[7])};
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < in) p[q] = (uint16_t)bf16_bits(y[q]);
    }
  } else {
    float* p = static_cast<float*>(Y) + row * ld + c;
    if (c + 8 <= in) {
      reinterpret_cast<f32x4_any*>(p)[0] = (f32x4){y[0], y[1], y[2], y[3]};
      reinterpret_cast<f32x4_any*>(p)[1] = (f32x4){y[4], y[5], y[6], y[7]};
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < in) p[q] = y[q];
    }
  }
}

}  // namespace gptq
