// A row's 8-bit integer codes and scale, a lane holding 8 consecutive columns.
#pragma once

#include "int8.h"
#include "mx_codec.h"

namespace gptq {

// largest magnitude's fp32 bits (infinities and NaN above every finite value) -> the row's scale
__device__ __forceinline__ float int8_scale(uint32_t top) {
  if (top >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  return fmaxf(__uint_as_float(top), 1e-12f) / 127.f;
}

// 8 codes of v / s, the exact quotient rounded to nearest, ties to even; s is finite, |v| <= 127 s (1 + 2^-23), inv is 1 / s
// to 2 ulp. Adding 1.5 * 2^23 rounds v inv to a whole number k, which then stands in the sum's low byte. v inv is off by less
// than 1e-4, so only a value that close to a tie can have been rounded wrongly. There e = v - k s, which one fused multiply-add
// gives exactly (a multiple of ulp(s) / 2 of at most 24 bits), is compared with s / 2: beyond it k is one off, and at it if
// k is odd. Values in bf16 meet ties often (one in 400 is a tie exactly if the largest one is even), so this way is short too.
__device__ __forceinline__ uint2 int8_encode(const float (&v)[8], float s, float inv) {
  constexpr float MAGIC = 12582912.f;
  float f[8], worst = 0.f;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    f[q] = fmaf(v[q], inv, MAGIC);
    worst = fmaxf(worst, fabsf(fmaf(v[q], inv, MAGIC - f[q])));
  }
  if (worst > 0.4999f) {
    const uint32_t half = __float_as_uint(0.5f * s);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint32_t k = __float_as_uint(f[q]);
      const float e = fmaf(MAGIC - f[q], s, v[q]);
      // |e| > half or |e| == half with k odd, as one comparison of whole numbers
      const uint32_t off = (__float_as_uint(e) & 0x7FFFFFFFu) + (k & 1u) > half ? 1u : 0u;
      f[q] = __uint_as_float(k + ((__float_as_uint(e) >> 31) ? 0u - off : off));
    }
  }
  uint32_t w[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(f[4 * q + 1]), __float_as_uint(f[4 * q]), 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(f[4 * q + 3]), __float_as_uint(f[4 * q + 2]), 0x0C0C0400u);
    w[q] = lo | hi << 16;
  }
  return make_uint2(w[0], w[1]);
}

// 8 columns from element `at` on, whatever its alignment
template <bool XBF16>
__device__ __forceinline__ Chunk<XBF16> load_full(const void* __restrict__ X, int64_t at) {
  const i32x4_any* p = reinterpret_cast<const i32x4_any*>(static_cast<const uint8_t*>(X) + at * (XBF16 ? 2 : 4));
  Chunk<XBF16> r;
#pragma unroll
  for (int q = 0; q < (XBF16 ? 1 : 2); ++q) {
    const i32x4 v = p[q];
#pragma unroll
    for (int e = 0; e < 4; ++e) r.w[4 * q + e] = (uint32_t)v[e];
  }
  return r;
}

// The columns moved down by s, zeros behind them
template <bool XBF16>
__device__ __forceinline__ void move_down(Chunk<XBF16>& r, int s) {
  constexpr int W = XBF16 ? 4 : 8;
#pragma unroll
  for (int b = W / 2; b > 0; b /= 2) {
    const bool on = s & (XBF16 ? 2 * b : b);
#pragma unroll
    for (int q = 0; q < W; ++q) {
      const uint32_t next = q + b < W ? r.w[q + b < W ? q + b : 0] : 0u;
      r.w[q] = s >= 8 ? 0u : on ? next : r.w[q];
    }
  }
  if (XBF16 && (s & 1)) {
#pragma unroll
    for (int q = 0; q < W; ++q) r.w[q] = r.w[q] >> 16 | (q + 1 < W ? r.w[q + 1 < W ? q + 1 : 0] << 16 : 0u);
  }
}

// Where a lane reads the last of its pieces of a row of d columns, which may reach past the row's end: there the row's last
// eight columns are read instead, without a branch, and moved down when they are used. (Tails one column at a time: norm of
// 3000 x 1357 14.5 us, so 12.9.) Rows of fewer than eight columns are read one by one.
struct Tail {
  int from, s;
  __device__ __forceinline__ void init(int c, int d) { from = min(c, max(d - 8, 0)), s = c - from; }
  template <bool XBF16>
  __device__ __forceinline__ Chunk<XBF16> load(const void* __restrict__ X, int64_t row, int d) const {
    if (d < 8) return load_chunk<XBF16>(X, row + s, s, d);
    return load_full<XBF16>(X, row + from);
  }
  template <bool XBF16>
  __device__ __forceinline__ void settle(Chunk<XBF16>& r, int d) const {
    if (s > 0 && d >= 8) move_down(r, s);
  }
};

__device__ __forceinline__ void store8(void* Y, bool bf16, int64_t off, int c, int d, const float (&y)[8]) {
  if (bf16) {
    uint16_t* p = static_cast<uint16_t*>(Y) + off;
    if (c + 8 <= d) {
      *reinterpret_cast<i32x4_any*>(p) = (i32x4){(int)bf16_pair(y[0], y[1]), (int)bf16_pair(y[2], y[3]),
                                                 (int)bf16_pair(y[4], y[5]), (int)bf16_pair(y[6], y[7])};
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < d) p[q] = (uint16_t)bf16_bits(y[q]);
    }
  } else {
    float* p = static_cast<float*>(Y) + off;
    if (c + 8 <= d) {
      reinterpret_cast<f32x4_any*>(p)[0] = (f32x4){y[0], y[1], y[2], y[3]};
      reinterpret_cast<f32x4_any*>(p)[1] = (f32x4){y[4], y[5], y[6], y[7]};
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (c + q < d) p[q] = y[q];
    }
  }
}

// 8 columns of fp32 numbers from c on, zeros behind the last
__device__ __forceinline__ void load8(const float* p, int c, int d, float (&v)[8]) {
  if (c + 8 <= d) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const f32x4 t = reinterpret_cast<const f32x4_any*>(p + c)[q];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * q + e] = t[e];
    }
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = c + q < d ? p[c + q] : 0.f;
  }
}

}  // namespace gptq
