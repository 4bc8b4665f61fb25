// Quantization of tokens to 8-bit integers with a scale a row, its inverse, and GPTQ's codes in padded rows.
//
// A row's scale needs the whole row, so a workgroup takes a row and holds it in registers between the maximum and the
// codes: one pass over memory.
#include <algorithm>

#include "int8_codec.h"
#include "rows.h"

namespace gptq {

namespace {

template <bool XBF16, int NCH, int LANES>
__global__ __launch_bounds__(1024) void k_int8_quantize(const void* __restrict__ X, int64_t ld, int64_t n, int d, int kp,
                                                        RowShape rs, int8_t* __restrict__ codes,
                                                        float* __restrict__ scales) {
  __shared__ RowShared shared;
  RowGroup<LANES> g;
  g.init(rs);
  if (LANES < 64 && g.slot >= rs.rows) return;
  Tail tail;
  tail.init(g.column(NCH - 1), d);
  for (int64_t r0 = (int64_t)blockIdx.x * rs.rows; r0 < n; r0 += (int64_t)gridDim.x * rs.rows) {
    const int64_t row = r0 + g.slot;
    Chunk<XBF16> x[NCH];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int64_t at = min(row, n - 1) * ld;
      x[i] = i < NCH - 1 ? load_full<XBF16>(X, at + g.column(i)) : tail.load<XBF16>(X, at, d);
    }
    tail.settle(x[NCH - 1], d);
#pragma unroll
    for (int i = 0; i < NCH; ++i) top = max(top, max_bits<XBF16>(chunk_max<XBF16>(x[i])));
    top = g.max_of_row(top, shared);
    const float s = int8_scale(top);
    const bool finite = top < 0x7F800000u;
    const float inv = __builtin_amdgcn_rcpf(s);
    if (row < n) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int c = g.column(i);
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = chunk_at<XBF16>(x[i], q);
        if (c < kp) *reinterpret_cast<uint2*>(codes + row * kp + c) = finite ? int8_encode(v, s, inv) : make_uint2(0u, 0u);
      }
      if (g.lane == 0) scales[row] = s;
    }
  }
}

// a wave's unit: 512 columns of a row
template <bool YBF16>
__global__ __launch_bounds__(256) void k_int8_dequantize(const int8_t* __restrict__ codes, const float* __restrict__ scales,
                                                         int d, int kp, int ks, int64_t units, void* __restrict__ Y,
                                                         int64_t ld) {
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit >= units) return;
  const int64_t row = unit / ks;
  const int c = (int)(unit - row * ks) * UNIT + (threadIdx.x & 63) * 8;
  if (c >= d) return;
  const uint2 v = *reinterpret_cast<const uint2*>(codes + row * kp + c);
  const float s = scales[row];
  float y[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) y[q] = (float)(int8_t)((q < 4 ? v.x : v.y) >> (8 * (q & 3))) * s;
  store8(Y, YBF16, row * ld + c, c, d, y);
}

// 16 bytes of a padded row a thread, read one by one, since GPTQ's rows start at any byte; a layer is padded once (4096 x 4100
// 25 us, 11008 x 4000 55; the copy's rate 7 and 18)
__global__ __launch_bounds__(256) void k_int8_pad(const int8_t* __restrict__ codes, int d, int kp, int64_t total,
                                                  int8_t* __restrict__ padded) {
  const int per_row = kp / 16;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    const int64_t row = e / per_row;
    const int c = (int)(e - row * per_row) * 16;
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 16; ++q)
      if (c + q < d) w[q >> 2] |= (uint32_t)(uint8_t)codes[row * d + c + q] << (8 * (q & 3));
    *reinterpret_cast<uint4*>(padded + row * kp + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

constexpr int64_t MAX_UNITS = (int64_t)1 << 25;

}  // namespace

hipError_t int8_quantize_launch(const void* X, int x_dtype, int64_t n, int64_t in, int64_t ld_x, int8_t* codes,
                                float* scales, hipStream_t stream) {
  const int kp = (int)int8_code_row(in);
  const RowShape rs = row_shape(in, n, 4);
  const dim3 grid((unsigned)std::min<int64_t>(ceil_div(n, rs.rows), (int64_t)4 * 256 * (2048 / rs.threads()))), block(rs.threads());
  const bool b = x_dtype == GPTQ_BF16;
#define GPTQ_GO(N, L)                                                                                                   \
  hipLaunchKernelGGL((b ? k_int8_quantize<true, N, L> : k_int8_quantize<false, N, L>), grid, block, 0, stream, X, ld_x, n, \
                     (int)in, kp, rs, codes, scales)
  GPTQ_ROW_SHAPE(rs, GPTQ_GO)
#undef GPTQ_GO
  return hipGetLastError();
}

hipError_t int8_dequantize_launch(const Int8Matrix& q, void* Y, int y_dtype, int64_t ld_y, hipStream_t stream) {
  const int ks = (int)ceil_div(q.cols, UNIT);
  const int kp = (int)int8_code_row(q.cols);
  const bool b = y_dtype == GPTQ_BF16;
  const int64_t rows_max = MAX_UNITS / ks;  // a grid stays below 2^32 work-items
  for (int64_t r = 0; r < q.rows; r += rows_max) {
    const int64_t units = std::min(rows_max, q.rows - r) * ks;
    void* y = static_cast<uint8_t*>(Y) + r * ld_y * (b ? 2 : 4);
    hipLaunchKernelGGL(b ? k_int8_dequantize<true> : k_int8_dequantize<false>, dim3((unsigned)ceil_div(units, 4)), dim3(256),
                       0, stream, q.codes + r * kp, q.scales + r, (int)q.cols, kp, ks, units, y, ld_y);
  }
  return hipGetLastError();
}

hipError_t int8_pad_launch(const int8_t* codes, int64_t out, int64_t in, int8_t* padded, hipStream_t stream) {
  const int64_t kp = int8_code_row(in), total = out * (kp / 16);
  hipLaunchKernelGGL(k_int8_pad, dim3((unsigned)std::min<int64_t>(1 << 16, ceil_div(total, 256))), dim3(256), 0, stream,
                     codes, (int)in, (int)kp, total, padded);
  return hipGetLastError();
}

}  // namespace gptq
