// Y = A W^T (+ bias) (ReLU) with A (n x in, E2M1 or E4M3) and W (out x in, E2M1) in MX form, on the scaled matrix
// instructions of gfx950: v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 4- and 8-bit elements and applies each
// block's two scale bytes to its 32 products before they are added in fp32.
//
// W is the first operand, so that a lane of the result holds four consecutive columns of Y. Lane l = 32 h + r of an
// operand holds row r: 4-bit elements of columns 32 h .. 32 h + 31 of the 64; 8-bit elements of columns
// 16 h .. 16 h + 15 and 32 + 16 h .. 32 + 16 h + 15; in both cases the scale byte of block h.
// (Found with an in-bounds check of the instruction's layout.)
#include <algorithm>

#include "mx_tile.h"

namespace gptq {

namespace {

struct MatmulArgs {
  const uint8_t *ac, *as, *wc, *ws;
  const float* bias;
  void* Y;
  int64_t n, ld;
  int64_t crow_a, crow_w, srow;  // bytes of a row of codes and of scales
  int out, ta, tb;               // tiles along out and along tokens
  int nk, slice;                 // 128s of columns; those of a slice (a multiple of 4)
  int relu;
};

// bias (may be null) and ReLU
template <int V>
struct StoreLinear {
  const float* bias;
  float low, b[V];
  __device__ __forceinline__ float relu(float v) { return v < low ? low : v; }  // NaN stays
  __device__ __forceinline__ void columns(int c) {
#pragma unroll
    for (int q = 0; q < V; ++q) b[q] = 0.f;
    if (bias) {
#pragma unroll
      for (int q = 0; q < V; ++q) b[q] = bias[c + q];
    }
  }
  __device__ __forceinline__ void row(int, int, int64_t, int) {}
  __device__ __forceinline__ void keep(int, int) {}
  __device__ __forceinline__ void finish(int, int, float (&v)[V]) {
#pragma unroll
    for (int q = 0; q < V; ++q) v[q] = relu(v[q] + b[q]);
  }
  __device__ __forceinline__ float one(int64_t, int c, float v) { return relu(bias ? v + bias[c] : v); }
};

template <int FMT, bool YBF16, int WA, int WB, int MB, int NB, int OCC>
__global__ __launch_bounds__(256, OCC) void k_mx_matmul(const MatmulArgs g) {
  using T = TileProduct<K_E2M1, FMT == GPTQ_MX_E2M1 ? K_E2M1 : K_E4M3, WA, WB, MB, NB>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  TileOrder order;
  order.init(blockIdx.x, gridDim.x, g.ta, g.tb);
  int ia, ib;
  if (!order.get(0, ia, ib)) return;
  const int k0 = blockIdx.y * g.slice, nk = min(g.slice, g.nk - k0);
  const int stages = (nk + 1) / 2;
  const int64_t wk = (int64_t)k0 * 64, ak = (int64_t)k0 * (FMT == GPTQ_MX_E2M1 ? 64 : 128);
  T t;
  t.init(lds, g.srow);
  t.a.init(g.crow_w, t.wave, t.lane, t.wa);
  t.b.init(g.crow_a, t.wave, t.lane, t.wb);
  t.tail = __builtin_amdgcn_readfirstlane(nk & 1);
  auto locate = [&](bool any, Stretch& a, Stretch& b, Stretch& sa, Stretch& sb) {
    const int o0 = ia * WA;
    const int64_t t0 = (int64_t)ib * WB;
    const int ro = min(WA, g.out - o0), rt = (int)min((int64_t)WB, g.n - t0);
    const int n = any ? stages : 0;
    a.init(g.wc + (int64_t)o0 * g.crow_w + wk, ro * g.crow_w - wk, T::A::STEP, n);
    b.init(g.ac + t0 * g.crow_a + ak, rt * g.crow_a - ak, T::B::STEP, n);
    sa.init(g.ws + (int64_t)o0 * g.srow + k0 * 4, ro * g.srow - k0 * 4, 32, n);
    sb.init(g.as + t0 * g.srow + k0 * 4, rt * g.srow - k0 * 4, 32, n);
  };
  locate(true, t.a.mem, t.b.mem, t.sa, t.sb);
  t.start();
  bool more = true;
  for (int r = 1; more; ++r) {
    const int64_t row0 = (int64_t)ib * WB + t.wb;
    const int c0 = ia * WA + t.wa;
    more = order.get(r, ia, ib);
    locate(more, t.an, t.bn, t.san, t.sbn);
    t.multiply((stages + 1) / 2 * 2);
    if (!T::STAYS) wait_and_barrier<0>();
    uint8_t* buf = T::STAYS ? lds + T::LDS - 4 * 4096 * T::PB : lds;
    if (gridDim.y > 1) {
      float* part = static_cast<float*>(g.Y) + blockIdx.y * g.n * (int64_t)g.out;
      store_rows<false, T::PB>(t.acc, buf, part, g.ld, row0, g.n, c0, g.out, false, StoreAsIs());
    } else {
      StoreLinear<YBF16 ? 8 : 4> done;
      done.bias = g.bias, done.low = g.relu ? 0.f : -__builtin_inff();
      store_rows<YBF16, T::PB>(t.acc, buf, g.Y, g.ld, row0, g.n, c0, g.out, false, done);
    }
    if (!T::STAYS) return;
    t.clear();
  }
  wait_and_barrier<0>();  // nothing may still be writing LDS when the workgroup ends
}

// The slices' partial products, added in their order; bias, ReLU and the result's type.
template <bool YBF16>
__global__ __launch_bounds__(256) void k_mx_join(const float* __restrict__ part, int slices, int64_t n, int out,
                                                 const float* __restrict__ bias, int relu, void* __restrict__ Y,
                                                 int64_t ld) {
  const int64_t total = n * out;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    float y = 0.f;
    for (int s = 0; s < slices; ++s) y += part[s * total + e];
    const int64_t row = e / out;
    const int c = (int)(e - row * out);
    if (bias) y += bias[c];
    if (relu) y = relu_nan(y);
    if (YBF16) static_cast<uint16_t*>(Y)[row * ld + c] = (uint16_t)bf16_bits(y);
    else static_cast<float*>(Y)[row * ld + c] = y;
  }
}

// Tile sizes along out and along tokens. A stage of E4M3 tokens is twice that of E2M1 ones, so its large tile has half
// the tokens.
struct MatmulPlan {
  int wa, wb;
  int slices;  // of k
};

MatmulPlan matmul_plan(int64_t n, int64_t in, int64_t out, int fmt) {
  const int64_t nk = ceil_div(in, 128);
  auto tiles = [&](int64_t a, int64_t b) { return ceil_div(out, a) * ceil_div(n, b); };
  // The largest tile that gives (nearly) every CU one. us with tiles of 64 / 128 / 256 (E2M1): 512 x 4096 x 4096 13.1 /
  // 13.8 / 26, 1024 x 4096 x 4096 21.3 / 16.9 / 32, 2048 x 4096 x 4096 37 / 26 / 35, 4096 x 4096 x 4096 67 / 47 / 42; with a
  // short k the results' way out counts more than the products: 8000 x 1024 x 8000 92 / 64 / 74. E4M3: 512 x 4096 x 4096
  // 23 / 19 / 48, 1024 x 4096 x 4096 40 / 31 / 51, 4096 x 4096 x 4096 143 / 115 / 113, 8000 x 1024 x 8000 169 / 138 / 138.
  MatmulPlan p = {64, 64, 1};
  if (fmt == GPTQ_MX_E2M1) {
    if (tiles(256, 256) >= 256 && nk >= 16) p = {256, 256, 1};
    else if (tiles(128, 128) >= 224) p = {128, 128, 1};
  } else {
    if (tiles(256, 128) >= 256) p = {256, 128, 1};
    else if (tiles(128, 64) >= 224) p = {128, 64, 1};
  }
  // Slices of k, joined by another launch, only where few tiles have a long sum each: 512 x 11008 x 512 (64 tiles) takes
  // 13.6 us with 4 of them and over 17 with one, but 64 x 4096 x 4096 (64 tiles) 8.7 with one and 9.8 with two.
  const int64_t t = tiles(p.wa, p.wb);
  if (t > 0 && t < 256) p.slices = (int)std::max<int64_t>(1, std::min<int64_t>({256 / t, nk / 24, 16}));
  return p;
}

template <int FMT, bool YBF16>
void matmul_go(const MatmulPlan& p, dim3 grid, hipStream_t stream, const MatmulArgs& g) {
#define GPTQ_GO(WA, WB, MB, NB, OCC) \
  hipLaunchKernelGGL((k_mx_matmul<FMT, YBF16, WA, WB, MB, NB, OCC>), grid, dim3(256), 0, stream, g)
  if (p.wa == 64) {
    GPTQ_GO(64, 64, 1, 1, 2);
  } else if constexpr (FMT == GPTQ_MX_E2M1) {
    if (p.wa == 256) GPTQ_GO(256, 256, 4, 4, 1);
    else GPTQ_GO(128, 128, 2, 2, 2);
  } else {
    if (p.wa == 256) GPTQ_GO(256, 128, 4, 2, 1);
    else GPTQ_GO(128, 64, 2, 1, 2);
  }
#undef GPTQ_GO
}

}  // namespace

size_t mx_matmul_ws_bytes(int64_t n, int64_t in, int64_t out, int a_fmt) {
  if (n <= MX_FEW) return 0;
  const MatmulPlan p = matmul_plan(n, in, out, a_fmt);
  return p.slices > 1 ? align_up((size_t)p.slices * n * out * 4, 256) : 0;
}

hipError_t mx_matmul_launch(const MxMatrix& a, const MxMatrix& w, const float* bias, int relu, void* Y, int y_dtype,
                            int64_t ld_y, void* ws, hipStream_t stream) {
  if (a.rows <= MX_FEW) return mx_matmul_few_launch(a, w, bias, relu, Y, y_dtype, ld_y, stream);
  const MatmulPlan p = matmul_plan(a.rows, a.cols, w.rows, a.fmt);
  const bool bf16 = y_dtype == GPTQ_BF16;
  const int64_t srow = mx_scale_row(a.cols), crow = mx_code_row(a.cols, a.fmt);
  MatmulArgs g = {};
  g.wc = w.codes, g.ws = w.scales, g.crow_a = crow, g.crow_w = mx_code_row(a.cols, GPTQ_MX_E2M1), g.srow = srow;
  g.out = (int)w.rows, g.ta = (int)ceil_div(w.rows, p.wa), g.nk = (int)ceil_div(a.cols, 128);
  g.slice = p.slices > 1 ? (int)ceil_div(ceil_div(g.nk, p.slices), 4) * 4 : g.nk;
  const int slices = (int)ceil_div(g.nk, g.slice);
  // at most 2^20 tiles a launch
  const int64_t rows_max = p.slices > 1 ? a.rows : std::max<int64_t>(1, ((int64_t)1 << 20) / g.ta) * p.wb;
  for (int64_t r = 0; r < a.rows; r += rows_max) {
    g.n = std::min(rows_max, a.rows - r);
    g.tb = (int)ceil_div(g.n, p.wb);
    g.ac = a.codes + r * crow, g.as = a.scales + r * srow;
    g.bias = bias, g.relu = relu, g.ld = ld_y;
    g.Y = static_cast<uint8_t*>(Y) + r * ld_y * (bf16 ? 2 : 4);
    if (slices > 1) g.Y = ws, g.ld = w.rows;
    const dim3 grid(tile_grid((int64_t)g.ta * g.tb, p.wa == 256 ? 256 : 1 << 30), (unsigned)slices);
    if (a.fmt == GPTQ_MX_E2M1) {
      bf16 ? matmul_go<GPTQ_MX_E2M1, true>(p, grid, stream, g) : matmul_go<GPTQ_MX_E2M1, false>(p, grid, stream, g);
    } else {
      bf16 ? matmul_go<GPTQ_MX_E4M3, true>(p, grid, stream, g) : matmul_go<GPTQ_MX_E4M3, false>(p, grid, stream, g);
    }
  }
  if (slices > 1) {
    const unsigned grid = (unsigned)std::min<int64_t>(2048, ceil_div(a.rows * w.rows, 256));
    if (bf16)
      hipLaunchKernelGGL((k_mx_join<true>), dim3(grid), dim3(256), 0, stream, static_cast<const float*>(ws), slices,
                         a.rows, (int)w.rows, bias, relu, Y, ld_y);
    else
      hipLaunchKernelGGL((k_mx_join<false>), dim3(grid), dim3(256), 0, stream, static_cast<const float*>(ws), slices,
                         a.rows, (int)w.rows, bias, relu, Y, ld_y);
  }
  return hipGetLastError();
}

size_t mx_linear_ws_bytes(int64_t n, int64_t in, int64_t out, int act_fmt) {
  if (mx_few_fused(n, in)) return 0;
  return align_up(n * mx_code_row(in, act_fmt), 256) + align_up(n * mx_scale_row(in), 256) +
         mx_matmul_ws_bytes(n, in, out, act_fmt);
}

hipError_t mx_linear_launch(const void* X, int x_dtype, int64_t n, int64_t ld_x, int act_fmt, const MxMatrix& w,
                            const float* bias, int relu, void* Y, int y_dtype, int64_t ld_y, void* ws,
                            hipStream_t stream) {
  if (mx_few_fused(n, w.cols)) return mx_linear_few_launch(X, x_dtype, n, ld_x, act_fmt, w, bias, relu, Y, y_dtype, ld_y, stream);
  uint8_t* codes = static_cast<uint8_t*>(ws);
  uint8_t* scales = codes + align_up(n * mx_code_row(w.cols, act_fmt), 256);
  uint8_t* rest = scales + align_up(n * mx_scale_row(w.cols), 256);
  const hipError_t e = mx_quantize_launch(X, x_dtype, n, w.cols, ld_x, act_fmt, codes, scales, stream);
  if (e != hipSuccess) return e;
  const MxMatrix a = {codes, scales, act_fmt, n, w.cols};
  return mx_matmul_launch(a, w, bias, relu, Y, y_dtype, ld_y, rest, stream);
}

}  // namespace gptq
