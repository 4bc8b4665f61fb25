// The norm's gradient: with g = dy w, dx = rstd (g - h rstd^2 mean(g h)) (+ dh), one reduction a row, and dw = sum over rows of
// dy h rstd in fp64, first over a workgroup's rows, then over workgroups in their order.
//
// What bounds it is memory: dy, h and dh are read once and dx is written.
#include <algorithm>

#include "int8_codec.h"
#include "rows.h"

namespace gptq {

namespace {

// HOLD: a row stays in registers between its sum and its gradient, and the next one is on its way meanwhile; rows of more than
// 12288 columns are read again. Two and three chunks a lane take up to 205 registers: eight waves to a CU, with over 100 KB of
// loads in flight between them (held to 128 registers 8192 x 11008 takes 500 us instead of 150). The longer rows' four and eight
// chunks have up to sixteen waves and so 128 registers, of which their sums of dweight alone take 64 and 128: 138 to 174 and 466
// to 541 registers are spilled, and updated in scratch memory for every row (8192 x 16384 in bf16 with dh 647 us, 2048 x 65536
// 1097, the copy's rate 217 for both).
template <bool YBF16, bool HBF16, bool DH, int NCH, int LANES>
__global__ __launch_bounds__(NCH == 2 || NCH == 3 ? 512 : 1024) void k_rms_norm_grad(const NormGradArgs a, const RowShape rs) {
  constexpr bool HOLD = NCH <= 3;
  constexpr int NH = HOLD ? NCH : 1;
  __shared__ RowShared shared;
  RowGroup<LANES> g;
  g.init(rs);
  const int64_t step = (int64_t)gridDim.x * rs.rows;
  double dw[NCH][8];
  float w[NH][8];
#pragma unroll
  for (int i = 0; i < NCH; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) dw[i][q] = 0.0;
  Chunk<YBF16> y[NH];
  Chunk<HBF16> h[NH], s[NH];
  float rstd = 0.f;
  Tail tail;
  tail.init(g.column(NCH - 1), a.d);
  auto load = [&](int64_t at, int i, int to) {
    const int64_t row = min(at, a.n - 1);
    if (i < NCH - 1) {
      const int c = g.column(i);
      y[to] = load_full<YBF16>(a.dy, row * a.ldy + c);
      h[to] = load_full<HBF16>(a.h, row * a.ldh + c);
      if (DH) s[to] = load_full<HBF16>(a.dh, row * a.lddh + c);
    } else {
      y[to] = tail.load<YBF16>(a.dy, row * a.ldy, a.d);
      h[to] = tail.load<HBF16>(a.h, row * a.ldh, a.d);
      if (DH) s[to] = tail.load<HBF16>(a.dh, row * a.lddh, a.d);
    }
  };
  auto settle = [&](int i, int to) {
    if (i < NCH - 1) return;
    tail.settle(y[to], a.d), tail.settle(h[to], a.d);
    if (DH) tail.settle(s[to], a.d);
  };
  if (HOLD) {
    const int64_t row = (int64_t)blockIdx.x * rs.rows + g.slot;
#pragma unroll
    for (int i = 0; i < NH; ++i) load(row, i, i);
    rstd = a.rstd[min(row, a.n - 1)];
#pragma unroll
    for (int i = 0; i < NH; ++i) load8(a.weight, g.column(i), a.d, w[i]);
  }
  for (int64_t r0 = (int64_t)blockIdx.x * rs.rows; r0 < a.n; r0 += step) {
    const int64_t row = r0 + g.slot;
    const bool live = row < a.n && g.slot < rs.rows;
    if (!HOLD) rstd = a.rstd[min(row, a.n - 1)];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int at = HOLD ? i : 0;
      if (!HOLD) load(row, i, 0), load8(a.weight, g.column(i), a.d, w[0]);
      settle(i, at);
#pragma unroll
      for (int q = 0; q < 8; ++q) dot = fmaf(chunk_at<YBF16>(y[at], q) * w[at][q], chunk_at<HBF16>(h[at], q), dot);
    }
    dot = g.sum_of_row(dot, shared);
    const float mean = dot / (float)a.d * rstd * rstd;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = g.column(i), at = HOLD ? i : 0;
      if (!HOLD) load(row, i, 0), load8(a.weight, c, a.d, w[0]), settle(i, 0);
      if (live) {
        float dx[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float yv = chunk_at<YBF16>(y[at], q), hv = chunk_at<HBF16>(h[at], q);
          dx[q] = rstd * (yv * w[at][q] - hv * mean);
          if (DH) dx[q] += chunk_at<HBF16>(s[at], q);
          dw[i][q] += (double)(yv * (hv * rstd));
        }
        store8(a.dx, HBF16, row * a.lddx + c, c, i < NCH - 1 ? c + 8 : a.d, dx);
      }
      if (HOLD && r0 + step < a.n) load(row + step, i, i);
    }
    if (HOLD) rstd = a.rstd[min(row + step, a.n - 1)];
  }
  // the workgroup's rows added in their order; the only workgroup's sums are the result
  extern __shared__ double sums[];
  const bool only = gridDim.x == 1;
  auto leave = [&](int c, double v) {
    if (only) a.dweight[c] = (float)(a.accumulate ? (double)a.dweight[c] + v : v);
    else a.part[(int64_t)blockIdx.x * a.d + c] = v;
  };
  if (g.slot < rs.rows) {
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const int c = g.column(i) + q;
        if (c >= a.d) continue;
        if (rs.rows > 1) sums[g.slot * a.d + c] = dw[i][q];
        else leave(c, dw[i][q]);
      }
  }
  if (rs.rows == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < a.d; c += blockDim.x) {
    double v = sums[c];
    for (int s = 1; s < rs.rows; ++s) v += sums[s * a.d + c];
    leave(c, v);
  }
}

// 32 columns a workgroup, 32 groups of partial rows side by side
__global__ __launch_bounds__(1024) void k_rms_norm_grad_join(const double* __restrict__ part, int parts, int d, int accumulate,
                                                             float* __restrict__ dw) {
  __shared__ double red[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
  double sum = 0.0;
  if (c < d)
#pragma unroll 8
    for (int p = y; p < parts; p += 32) sum += part[(int64_t)p * d + c];
  red[y][x] = sum;
  __syncthreads();
  if (y == 0 && c < d) {
#pragma unroll 8
    for (int q = 1; q < 32; ++q) sum += red[q][x];
    dw[c] = (float)(accumulate ? (double)dw[c] + sum : sum);
  }
}

// Workgroups of eight waves, of sixteen for rows of up to 2048 columns, and one of them to a CU: every one leaves a row of fp64
// sums (16384 x 4096 with dh: 105 us so, 126 with two to a CU; 16384 x 256: 14.3 and 18). Up to 32768 values in up to four turns
// go to a single one, which saves a call the second launch, 3.3 us on the host (64 x 512: 7.5 us of GPU time, 8 x 4096 10.5;
// 512 x 64 would take eight turns, 14.5).
struct GradPlan {
  RowShape shape;
  unsigned grid;
};
GradPlan grad_plan(int64_t d, int64_t n) {
  const int waves = d <= 2048 ? 16 : 8;
  const RowShape most = row_shape(d, 1 << 20, waves);
  if (n * d <= 32768 && n <= 4 * most.rows) return {most, 1};
  const RowShape s = row_shape(d, n, waves);
  return {s, (unsigned)std::min<int64_t>(ceil_div(n, s.rows), 256)};
}

template <bool YBF16, bool HBF16, bool DH>
void grad_go(const NormGradArgs& a, hipStream_t stream) {
  const GradPlan p = grad_plan(a.d, a.n);
  const RowShape rs = p.shape;
  const dim3 grid(p.grid), block(rs.threads());
  const size_t lds = rs.rows > 1 ? rs.rows * a.d * sizeof(double) : 0;
#define GPTQ_GO(N, L) hipLaunchKernelGGL((k_rms_norm_grad<YBF16, HBF16, DH, N, L>), grid, block, lds, stream, a, rs)
  GPTQ_ROW_SHAPE(rs, GPTQ_GO)
#undef GPTQ_GO
}

}  // namespace

size_t rms_norm_grad_ws_bytes(int64_t n, int64_t d) {
  if (n == 0) return 0;
  const unsigned grid = grad_plan(d, n).grid;
  return grid > 1 ? align_up((size_t)grid * d * 8, 256) : 0;
}

hipError_t rms_norm_grad_launch(const NormGradArgs& a, int y_dtype, int h_dtype, hipStream_t stream) {
  int parts = 0;
  if (a.n > 0) {
    parts = (int)grad_plan(a.d, a.n).grid;
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
    if (e != hipSuccess || parts == 1) return e;
  }
  hipLaunchKernelGGL(k_rms_norm_grad_join, dim3((unsigned)ceil_div(a.d, 32)), dim3(1024), 0, stream, a.part, parts, a.d,
                     a.accumulate, a.dweight);
  return hipGetLastError();
}

}  // namespace gptq
