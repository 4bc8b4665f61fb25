// Root-mean-square norm with the residual's addition and an output in 8 bits, and its gradient.
//
// Forward, for a row: h = x + r; rstd = (mean h^2 + eps)^(-1/2); u = h w; out = u rstd in 8 bits. As integers the codes are
// those of u and rstd joins the scale, so one reduction gives both the sum of squares and the scale's maximum. The
// sum is held in fp64: what e4m3 rounds then differs from the definition in 64 bits by fp32 roundings that are the same in
// any order of the sum.
//
// Backward: with g = dy w, dx = rstd (g - h rstd^2 mean(g h)) (+ dh), one reduction a row; dw = sum over rows of dy h rstd in
// fp64, first over a workgroup's rows, then over workgroups in their order.
#include <algorithm>

#include "int8_codec.h"
#include "rows.h"

namespace gptq {

namespace {

// 1 / sqrt(x) to fp32 from the hardware's estimate y (2^-23): with e = 1 - x y^2, (1 - e)^(-1/2) = 1 + e / 2 + 3 e^2 / 8 + ...,
// so y (1 + e / 2 + 3 e^2 / 8) is off by about e^3. An infinite x leaves y = 0.
__device__ __forceinline__ float rsqrt_of(double x) {
  const double y = __builtin_amdgcn_rsq(x);
  const double e = fma(-x * y, y, 1.0);
  const double z = fma(y * e, fma(0.375, e, 0.5), y);
  return (float)(y == 0.0 ? 0.0 : z);
}

// h of 8 columns in its stored type, and as fp32
template <bool XBF16, int RES>
__device__ __forceinline__ void add_residual(const Chunk<XBF16>& x, const Chunk<RES == 2>& r, float (&h)[8]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    h[q] = chunk_at<XBF16>(x, q);
    if (RES == 1) h[q] += chunk_at<RES == 2>(r, q);
    if (RES == 2) h[q] = __uint_as_float(bf16_bits(h[q] + chunk_at<RES == 2>(r, q)) << 16);
  }
}

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));  // lanes 1 0 3 2
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));  // lanes 2 3 0 1
  return v;
}

// RES: 0 no residual, 1 fp32, 2 bf16
template <bool XBF16, int RES, int FMT, int NCH>
__global__ __launch_bounds__(1024) void k_rms_norm(const NormArgs a, const RowShape rs, const double inv_d) {
  __shared__ RowShared shared;
  RowGroup g;
  g.init(rs);
  const int kp = (a.d + 127) / 128 * 128, kscale = (a.d + 511) / 512 * 16;
  for (int64_t r0 = (int64_t)blockIdx.x * rs.rows; r0 < a.n; r0 += (int64_t)gridDim.x * rs.rows) {
    const int64_t row = r0 + g.slot;
    const int d = row < a.n ? a.d : 0;
    float h[NCH][8];
    double sum = 0.0;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = g.column(i);
      const Chunk<XBF16> x = load_chunk<XBF16>(a.x, row * a.ldx + c, c, d);
      Chunk<RES == 2> r = {};
      if (RES) r = load_chunk<RES == 2>(a.r, row * a.ldr + c, c, d);
      add_residual<XBF16, RES>(x, r, h[i]);
      float w[8];
      load8(a.weight, c, a.d, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        sum = fma((double)h[i][q], (double)h[i][q], sum);
        if (FMT == GPTQ_NORM_INT8) top = max(top, __float_as_uint(h[i][q] * w[q]) & 0x7FFFFFFFu);
      }
      if (RES) store8(a.h, RES == 2, row * a.ldh + c, c, d, h[i]);
    }
    g.both_of_row(sum, top, shared);
    if (row >= a.n) continue;
    const float rstd = rsqrt_of(fma(sum, inv_d, a.eps));
    if (a.rstd && g.lane_of_row == 0) a.rstd[row] = rstd;
    const float s = int8_scale(top);
    const bool finite = top < 0x7F800000u;
    const float inv = __builtin_amdgcn_rcpf(s);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = g.column(i);
      float w[8], v[8];
      load8(a.weight, c, a.d, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = h[i][q] * w[q];
      if (FMT == GPTQ_NORM_INT8) {
        if (c < kp) *reinterpret_cast<uint2*>(a.codes + row * kp + c) = finite ? int8_encode(v, s, inv) : make_uint2(0u, 0u);
      } else {
        Chunk<false> y;
#pragma unroll
        for (int q = 0; q < 8; ++q) y.w[q] = c + q < a.d ? __float_as_uint(v[q] * rstd) : 0u;
        const uint32_t byte = scale_byte<GPTQ_MX_E4M3>(quad_max(chunk_max<false>(y)));
        const uint2 code = encode8<false>(y, __uint_as_float(byte << 23));
        if (c < kp) *reinterpret_cast<uint2*>(a.codes + row * kp + c) = byte == 255u ? make_uint2(0u, 0u) : code;
        if ((threadIdx.x & 3) == 0 && (c >> 5) < kscale)
          static_cast<uint8_t*>(a.scales)[row * kscale + (c >> 5)] = (uint8_t)(c < a.d ? byte : 0u);
      }
    }
    if (FMT == GPTQ_NORM_INT8 && g.lane_of_row == 0) static_cast<float*>(a.scales)[row] = s * rstd;
  }
}

// HOLD: a row's dy and h stay in registers between its sum and its gradient; long rows are read again
template <bool YBF16, bool HBF16, bool DH, int NCH>
__global__ __launch_bounds__(1024) void k_rms_norm_grad(const NormGradArgs a, const RowShape rs) {
  constexpr bool HOLD = NCH <= 2;
  __shared__ RowShared shared;
  RowGroup g;
  g.init(rs);
  double dw[NCH][8];
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) dw[i][q] = 0.0;
  for (int64_t r0 = (int64_t)blockIdx.x * rs.rows; r0 < a.n; r0 += (int64_t)gridDim.x * rs.rows) {
    const int64_t row = r0 + g.slot;
    const int d = row < a.n ? a.d : 0;
    const float rstd = row < a.n ? a.rstd[row] : 0.f;
    Chunk<YBF16> y[HOLD ? NCH : 1];
    Chunk<HBF16> h[HOLD ? NCH : 1];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = g.column(i), at = HOLD ? i : 0;
      y[at] = load_chunk<YBF16>(a.dy, row * a.ldy + c, c, d);
      h[at] = load_chunk<HBF16>(a.h, row * a.ldh + c, c, d);
      float w[8];
      load8(a.weight, c, a.d, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) dot = fmaf(chunk_at<YBF16>(y[at], q) * w[q], chunk_at<HBF16>(h[at], q), dot);
    }
    dot = g.sum_of_row(dot, shared);
    if (row >= a.n) continue;
    const float mean = dot / (float)a.d * rstd * rstd;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = g.column(i), at = HOLD ? i : 0;
      if (!HOLD) y[at] = load_chunk<YBF16>(a.dy, row * a.ldy + c, c, d), h[at] = load_chunk<HBF16>(a.h, row * a.ldh + c, c, d);
      float w[8], dx[8];
      load8(a.weight, c, a.d, w);
      Chunk<HBF16> s = {};
      if (DH) s = load_chunk<HBF16>(a.dh, row * a.lddh + c, c, d);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float yv = chunk_at<YBF16>(y[at], q), hv = chunk_at<HBF16>(h[at], q);
        dx[q] = rstd * (yv * w[q] - hv * mean);
        if (DH) dx[q] += chunk_at<HBF16>(s, q);
        dw[i][q] += (double)(yv * (hv * rstd));
      }
      store8(a.dx, HBF16, row * a.lddx + c, c, d, dx);
    }
  }
  double* part = a.part + ((int64_t)blockIdx.x * rs.rows + g.slot) * a.d;
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (g.column(i) + q < a.d) part[g.column(i) + q] = dw[i][q];
}

// 32 columns a workgroup, eight groups of partial rows side by side
__global__ __launch_bounds__(256) void k_rms_norm_grad_join(const double* __restrict__ part, int parts, int d, int accumulate,
                                                            float* __restrict__ dw) {
  __shared__ double red[8][32];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  double sum = 0.0;
  if (c < d)
#pragma unroll 4
    for (int p = g; p < parts; p += 8) sum += part[(int64_t)p * d + c];
  red[g][threadIdx.x & 31] = sum;
  __syncthreads();
  if (g == 0 && c < d) {
#pragma unroll
    for (int q = 1; q < 8; ++q) sum += red[q][threadIdx.x];
    dw[c] = (float)(accumulate ? (double)dw[c] + sum : sum);
  }
}

// partial rows of dweight: workgroups of the gradient's launch
unsigned grad_grid(const RowShape& s, int64_t n) {
  return (unsigned)std::min<int64_t>(ceil_div(n, s.rows), 1024 / s.rows);
}

template <bool XBF16, int RES, int FMT>
void norm_go(const NormArgs& a, hipStream_t stream) {
  const RowShape rs = row_shape(ceil_div(a.d, 512), a.n);
  const dim3 grid(row_grid(rs, a.n)), block(rs.threads());
  const double inv_d = 1.0 / a.d;
#define GPTQ_GO(N) hipLaunchKernelGGL((k_rms_norm<XBF16, RES, FMT, N>), grid, block, 0, stream, a, rs, inv_d)
  GPTQ_ROW_CHUNKS(rs.chunks, GPTQ_GO)
#undef GPTQ_GO
}

template <bool XBF16, int RES>
void norm_fmt(const NormArgs& a, int fmt, hipStream_t stream) {
  fmt == GPTQ_NORM_INT8 ? norm_go<XBF16, RES, GPTQ_NORM_INT8>(a, stream) : norm_go<XBF16, RES, GPTQ_NORM_E4M3>(a, stream);
}

template <bool YBF16, bool HBF16, bool DH>
void grad_go(const NormGradArgs& a, hipStream_t stream) {
  const RowShape rs = row_shape(ceil_div(a.d, 512), a.n);
  const dim3 grid(grad_grid(rs, a.n)), block(rs.threads());
#define GPTQ_GO(N) hipLaunchKernelGGL((k_rms_norm_grad<YBF16, HBF16, DH, N>), grid, block, 0, stream, a, rs)
  GPTQ_ROW_CHUNKS(rs.chunks, GPTQ_GO)
#undef GPTQ_GO
}

}  // namespace

hipError_t rms_norm_launch(const NormArgs& a, int x_dtype, int r_dtype, int fmt, hipStream_t stream) {
  const bool b = x_dtype == GPTQ_BF16;
  if (!a.r) b ? norm_fmt<true, 0>(a, fmt, stream) : norm_fmt<false, 0>(a, fmt, stream);
  else if (r_dtype == GPTQ_BF16) b ? norm_fmt<true, 2>(a, fmt, stream) : norm_fmt<false, 2>(a, fmt, stream);
  else b ? norm_fmt<true, 1>(a, fmt, stream) : norm_fmt<false, 1>(a, fmt, stream);
  return hipGetLastError();
}

size_t rms_norm_grad_ws_bytes(int64_t n, int64_t d) {
  if (n == 0) return 0;
  const RowShape rs = row_shape(ceil_div(d, 512), n);
  return align_up((size_t)grad_grid(rs, n) * rs.rows * d * 8, 256);
}

hipError_t rms_norm_grad_launch(const NormGradArgs& a, int y_dtype, int h_dtype, hipStream_t stream) {
  int parts = 0;
  if (a.n > 0) {
    const RowShape rs = row_shape(ceil_div(a.d, 512), a.n);
    parts = (int)grad_grid(rs, a.n) * rs.rows;
    const int kind = (y_dtype == GPTQ_BF16 ? 4 : 0) + (h_dtype == GPTQ_BF16 ? 2 : 0) + (a.dh ? 1 : 0);
    switch (kind) {
      case 0: grad_go<false, false, false>(a, stream); break;
      case 1: grad_go<false, false, true>(a, stream); break;
      case 2: grad_go<false, true, false>(a, stream); break;
      case 3: grad_go<false, true, true>(a, stream); break;
      case 4: grad_go<true, false, false>(a, stream); break;
      case 5: grad_go<true, false, true>(a, stream); break;
      case 6: grad_go<true, true, false>(a, stream); break;
      default: grad_go<true, true, true>(a, stream); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_rms_norm_grad_join, dim3((unsigned)ceil_div(a.d, 32)), dim3(256), 0, stream, a.part, parts, a.d,
                     a.accumulate, a.dweight);
  return hipGetLastError();
}

}  // namespace gptq
