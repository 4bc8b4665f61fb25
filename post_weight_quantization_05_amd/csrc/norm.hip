// Root-mean-square norm with the residual's addition and an output in 8 bits.
//
// For a row: h = x + r; rstd = (mean h^2 + eps)^(-1/2); u = h w; out = u rstd in 8 bits. As integers the codes are those of u and
// rstd joins the scale, so one reduction gives both the sum of squares and the scale's maximum. The sum is held in fp64: what
// e4m3 rounds then differs from the definition in 64 bits by fp32 roundings that are the same in any order of the sum.
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

// RES: 0 no residual, 1 fp32, 2 bf16. A workgroup takes several rows in turn: the weight stays in registers, and the next row
// is on its way while this one is reduced and written (rows of over 12288 columns leave no registers for that). bf16 with a
// bf16 residual, into int8 and E4M3: 8192 x 11008 123 and 128 us (the copy's rate 128), 8192 x 16384 210 and 184 (190), 2048 x
// 65536 432 and 221 (190). Eight chunks a lane, rows of over 32768 columns, spill 39 to 54 registers into int8 and up to 8 into
// E4M3; three chunks spill 6 in one form, fp32 with an fp32 residual into int8 (8192 x 11008 226 us, the copy's rate 237).
template <bool XBF16, int RES, int FMT, int NCH, int LANES>
__global__ __launch_bounds__(1024) void k_rms_norm(const NormArgs a, const RowShape rs, const double inv_d) {
  __shared__ RowShared shared;
  RowGroup<LANES> g;
  g.init(rs);
  if (LANES < 64 && g.slot >= rs.rows) return;
  const int kp = (a.d + 127) / 128 * 128, kscale = (a.d + 511) / 512 * 16;
  const int64_t step = (int64_t)gridDim.x * rs.rows;
  constexpr bool AHEAD = NCH <= 3;
  constexpr int NH = AHEAD ? NCH : 1;
  float w[NH][8];
  Chunk<XBF16> x[NH];
  Chunk<RES == 2> r[NH];
  Tail tail;
  tail.init(g.column(NCH - 1), a.d);
  auto load = [&](int64_t at, int i, int to) {
    const int64_t row = min(at, a.n - 1);
    if (i < NCH - 1) {
      x[to] = load_full<XBF16>(a.x, row * a.ldx + g.column(i));
      if (RES) r[to] = load_full<RES == 2>(a.r, row * a.ldr + g.column(i));
    } else {
      x[to] = tail.load<XBF16>(a.x, row * a.ldx, a.d);
      if (RES) r[to] = tail.load<RES == 2>(a.r, row * a.ldr, a.d);
    }
  };
  if (AHEAD) {
#pragma unroll
    for (int i = 0; i < NH; ++i) load((int64_t)blockIdx.x * rs.rows + g.slot, i, i);
#pragma unroll
    for (int i = 0; i < NH; ++i) load8(a.weight, g.column(i), a.d, w[i]);
  }
  for (int64_t r0 = (int64_t)blockIdx.x * rs.rows; r0 < a.n; r0 += step) {
    const int64_t row = r0 + g.slot;
    float h[NCH][8];
    double sum = 0.0;
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = g.column(i), at = AHEAD ? i : 0;
      if (!AHEAD) load(row, i, 0), load8(a.weight, c, a.d, w[0]);
      if (i == NCH - 1) {
        tail.settle(x[at], a.d);
        if (RES) tail.settle(r[at], a.d);
      }
      add_residual<XBF16, RES>(x[at], r[at], h[i]);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        sum = fma((double)h[i][q], (double)h[i][q], sum);
        if (FMT == GPTQ_NORM_INT8) top = max(top, __float_as_uint(h[i][q] * w[at][q]) & 0x7FFFFFFFu);
      }
      if (RES && row < a.n) store8(a.h, RES == 2, row * a.ldh + c, c, i < NCH - 1 ? c + 8 : a.d, h[i]);
    }
    if (AHEAD && r0 + step < a.n) {
#pragma unroll
      for (int i = 0; i < NH; ++i) load(row + step, i, i);
    }
    g.both_of_row(sum, top, shared);
    if (row >= a.n) continue;
    const float rstd = rsqrt_of(fma(sum, inv_d, a.eps));
    if (a.rstd && g.lane == 0) a.rstd[row] = rstd;
    const float s = int8_scale(top);
    const bool finite = top < 0x7F800000u;
    const float inv = __builtin_amdgcn_rcpf(s);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = g.column(i), at = AHEAD ? i : 0;
      if (!AHEAD) load8(a.weight, c, a.d, w[0]);
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = h[i][q] * w[at][q];
      if (FMT == GPTQ_NORM_INT8) {
        if (c < kp) *reinterpret_cast<uint2*>(a.codes + row * kp + c) = finite ? int8_encode(v, s, inv) : make_uint2(0u, 0u);
      } else {
        Chunk<false> y;
#pragma unroll
        for (int q = 0; q < 8; ++q) y.w[q] = c + q < a.d ? __float_as_uint(v[q] * rstd) : 0u;
        const uint32_t byte = scale_byte<GPTQ_MX_E4M3>(quad_max(chunk_max<false>(y)));
        const uint2 code = encode8<false>(y, __uint_as_float(byte << 23));
        if (c < kp) *reinterpret_cast<uint2*>(a.codes + row * kp + c) = byte == 255u ? make_uint2(0u, 0u) : code;
        if ((threadIdx.x & 3) == 0 && (c >> 5) < kscale) {
          uint8_t* p = static_cast<uint8_t*>(a.scales) + row * kscale + (c >> 5);
          *p = (uint8_t)(c < a.d ? byte : 0u);
#pragma unroll
          for (int z = LANES / 4; z < 16; z += LANES / 4) p[z] = 0;  // parts of a wave: behind their columns
        }
      }
    }
    if (FMT == GPTQ_NORM_INT8 && g.lane == 0) static_cast<float*>(a.scales)[row] = s * rstd;
  }
}

template <bool XBF16, int RES, int FMT>
void norm_go(const NormArgs& a, hipStream_t stream) {
  const RowShape rs = row_shape(a.d, a.n, 4);
  const dim3 grid((unsigned)std::min<int64_t>(ceil_div(a.n, rs.rows), (int64_t)4 * 256 * (2048 / rs.threads()))), block(rs.threads());
  const double inv_d = 1.0 / a.d;
#define GPTQ_GO(N, L) hipLaunchKernelGGL((k_rms_norm<XBF16, RES, FMT, N, L>), grid, block, 0, stream, a, rs, inv_d)
  GPTQ_ROW_SHAPE(rs, GPTQ_GO)
#undef GPTQ_GO
}

template <bool XBF16, int RES>
void norm_fmt(const NormArgs& a, int fmt, hipStream_t stream) {
  fmt == GPTQ_NORM_INT8 ? norm_go<XBF16, RES, GPTQ_NORM_INT8>(a, stream) : norm_go<XBF16, RES, GPTQ_NORM_E4M3>(a, stream);
}

}  // namespace

hipError_t rms_norm_launch(const NormArgs& a, int x_dtype, int r_dtype, int fmt, hipStream_t stream) {
  const bool b = x_dtype == GPTQ_BF16;
  if (!a.r) b ? norm_fmt<true, 0>(a, fmt, stream) : norm_fmt<false, 0>(a, fmt, stream);
  else if (r_dtype == GPTQ_BF16) b ? norm_fmt<true, 2>(a, fmt, stream) : norm_fmt<false, 2>(a, fmt, stream);
  else b ? norm_fmt<true, 1>(a, fmt, stream) : norm_fmt<false, 1>(a, fmt, stream);
  return hipGetLastError();
}

}  // namespace gptq
