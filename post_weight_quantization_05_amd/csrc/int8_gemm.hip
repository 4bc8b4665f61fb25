// Y = A W^T s_a s_w (+ bias) (ReLU) with A (n x in) and W (out x in) in 8-bit integers, on v_mfma_i32_32x32x32_i8: sums are
// whole numbers of at most 128^2 x 65536 = 2^30 and exact in 32 bits, in any order, so slices of k change no result.
//
// W is the first operand, so that a lane of the result holds four consecutive columns of Y. Lane l of an operand holds row
// l % 32, columns 16 (l / 32) .. + 15 of the 32 (any order of k would do, both operands having the same).
#include <algorithm>
#include <cmath>

#include "int8.h"
#include "mx_tile.h"

namespace gptq {

namespace {

typedef __attribute__((ext_vector_type(4))) unsigned int u32x4;

struct MatmulArgs {
  const int8_t *ac, *wc;
  const float *as, *ws, *bias;
  void* Y;
  int64_t n, ld;
  int kp;            // bytes of a row of codes
  int out, ta, tb;   // tiles along out and along tokens
  int nk, slice;     // 128s of columns; those of a slice
  int relu;
  int past;          // results leave past the caches' reuse
};

// What a wave needs of the scales and the bias for its results, 32 MB columns by 32 NB rows: they come by transfers to LDS
// before the products and into registers behind them, a lane holding every 64th. (Loaded between the stores they
// would wait for them, and before them for memory: with both, 16384 x 4096 x 11008 took 97 us of 659 for its results.)
template <int MB, int NB>
struct WaveScales {
  static constexpr int NC = (32 * MB + 63) / 64, NR = (32 * NB + 63) / 64;
  static constexpr int BYTES = (2 * NC + NR) * 256, TRANSFERS = 2 * NC + NR;
  float w[NC], b[NC], s[NR];

  static __device__ __forceinline__ i32x4 buffer(const float* p, int64_t count) {
    const uint64_t a = (uint64_t)uniform64((int64_t)(uintptr_t)p);
    const int n = p && count > 0 ? (int)min(count, (int64_t)256) * 4 : 0;  // outside: zeros
    return (i32x4){(int)(uint32_t)a, (int)(uint32_t)(a >> 32) & 0xFFFF, __builtin_amdgcn_readfirstlane(n), 0x00020000};
  }
  static __device__ __forceinline__ void fetch(const MatmulArgs& g, uint32_t at, int c0, int64_t row0) {
    const uint32_t off = (threadIdx.x & 63) * 4;
    const i32x4 w = buffer(g.ws + c0, g.out - c0), b = buffer(g.bias ? g.bias + c0 : nullptr, g.out - c0);
    const i32x4 s = buffer(g.as + row0, g.n - row0);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      dma4(w, (uint32_t)__builtin_amdgcn_readfirstlane((int)(at + i * 256)), off + i * 256);
      dma4(b, (uint32_t)__builtin_amdgcn_readfirstlane((int)(at + (NC + i) * 256)), off + i * 256);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) dma4(s, (uint32_t)__builtin_amdgcn_readfirstlane((int)(at + (2 * NC + i) * 256)), off + i * 256);
  }
  __device__ __forceinline__ void take(const uint8_t* at) {
    const float* p = reinterpret_cast<const float*>(at) + (threadIdx.x & 63);
#pragma unroll
    for (int i = 0; i < NC; ++i) w[i] = p[i * 64], b[i] = p[(NC + i) * 64];
#pragma unroll
    for (int i = 0; i < NR; ++i) s[i] = p[(2 * NC + i) * 64];
  }
  // entry i of a row of them, i / 64 the same in all lanes
  template <int N>
  static __device__ __forceinline__ float pick(const float (&v)[N], int part, int lane) {
    return __int_as_float(__builtin_amdgcn_ds_bpermute(lane * 4, __float_as_int(v[part])));
  }
};

// Writes a wave's results: register i of lane l of acc[mb][nb] is row 32 nb + l % 32, column 32 mb + 8 (i / 4) + 4 (l / 32) + i % 4.
// The sums go through LDS, 32 PB columns of 32 rows at a time, so that a store takes runs of 128 bytes of a row or more. Returns
// whether the wave's results lie inside Y, each store then being issued. RAW: the sums themselves, to partial results.
template <bool YBF16, bool RAW, int PB, int MB, int NB>
__device__ __forceinline__ int store_int8(const f32x16 (&acc)[MB][NB], uint8_t* lds, const WaveScales<MB, NB>& sc,
                                          const MatmulArgs& g, void* __restrict__ Y, int64_t ld, int64_t row0, int c0) {
  constexpr int C = 32 * PB, V = YBF16 ? 8 : 4, PER_ROW = C / V, STEP = 64 / PER_ROW, IT = 32 / STEP;
  const int lane = threadIdx.x & 63;
  int* buf = reinterpret_cast<int*>(lds);
  const int r = lane & 31, h = lane >> 5;
  constexpr int ES = YBF16 ? 2 : 4;
  const bool inside = row0 + 32 * NB <= g.n && c0 + 32 * MB <= g.out && ld < (int64_t)1 << 22;
  const __amdgpu_buffer_rsrc_t to = __builtin_amdgcn_make_buffer_rsrc(
      static_cast<uint8_t*>(Y) + uniform64((row0 * ld + c0) * ES), 0, 0x7FFFFFF0, 0x00020000);
  const int step = __builtin_amdgcn_readfirstlane((int)ld * ES);  // used inside only
  const int first = (lane / PER_ROW) * step + (lane % PER_ROW) * 16;
  const float low = g.relu ? 0.f : -__builtin_inff();
  // the 16-byte chunks of row r are permuted by XOR with r, so that neither side's rows meet on the same banks
  auto chunk = [](int row, int q) { return row * C + ((q ^ (row & (C / 4 - 1))) << 2); };
#pragma unroll
  for (int m0 = 0; m0 < MB; m0 += PB) {
    float w[V], b[V];
    if (!RAW) {
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const int at = m0 % 2 * 32 + (lane % PER_ROW) * V + q;
        w[q] = sc.pick(sc.w, m0 / 2, at), b[q] = sc.pick(sc.b, m0 / 2, at);
      }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float s[IT];
#pragma unroll
      for (int it = 0; it < IT; ++it) s[it] = RAW ? 0.f : sc.pick(sc.s, nb / 2, nb % 2 * 32 + lane / PER_ROW + it * STEP);
#pragma unroll
      for (int mb = 0; mb < PB; ++mb)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *reinterpret_cast<float4*>(buf + chunk(r, mb * 8 + 2 * q + h)) =
              make_float4(acc[m0 + mb][nb][4 * q], acc[m0 + mb][nb][4 * q + 1], acc[m0 + mb][nb][4 * q + 2],
                          acc[m0 + mb][nb][4 * q + 3]);
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int it = 0; it < IT; ++it) {
        float v[V];
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
          const i32x4 x = *reinterpret_cast<const i32x4*>(
              buf + chunk(lane / PER_ROW + it * STEP, (lane % PER_ROW) * (V / 4) + q));
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[4 * q + e] = RAW ? __int_as_float(x[e]) : int8_result((float)x[e], s[it], w[4 * q + e], b[4 * q + e], low);
        }
        if (inside) {
          i32x4 o;
          if (YBF16)
            o = (i32x4){(int)bf16_pair(v[0], v[1]), (int)bf16_pair(v[2], v[3]), (int)bf16_pair(v[V - 4], v[V - 3]),
                        (int)bf16_pair(v[V - 2], v[V - 1])};
          else
            o = __builtin_bit_cast(i32x4, (f32x4){v[0], v[1], v[2], v[3]});
          // No scalar offset: behind a 16-byte store with one the compiler leaves out the wait state before a vector
          // instruction that writes its data registers, and here such stores took the new contents now and then.
          const int at = first + ((nb * 32 + it * STEP) * step + 32 * m0 * ES);
          if (g.past) __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o), to, at, 0, 2);
          else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o), to, at, 0, 0);
        } else {
          const int64_t row = row0 + nb * 32 + lane / PER_ROW + it * STEP;
          const int c = c0 + 32 * m0 + (lane % PER_ROW) * V, n = row < g.n ? g.out - c : 0;
#pragma unroll
          for (int q = 0; q < V; ++q) {
            if (q >= n) continue;
            if (YBF16) static_cast<uint16_t*>(Y)[row * ld + c + q] = (uint16_t)bf16_bits(v[q]);
            else static_cast<float*>(Y)[row * ld + c + q] = v[q];
          }
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
  return inside ? 1 : 0;
}

template <bool YBF16, int WA, int WB, int MB, int NB, int RING, int OCC>
__global__ __launch_bounds__(256, OCC) void k_int8_matmul(const MatmulArgs g) {
  using T = TileProduct<K_INT8, K_INT8, WA, WB, MB, NB, RING>;
  using S = WaveScales<MB, NB>;
  constexpr int PB = MB >= 2 ? 2 : 1;
  // results pass through memory of their own (large tiles) or the ring's; the scales wait in the former or behind the ring
  constexpr int RESULTS = T::STAYS ? T::LDS - 4 * 4096 * PB : 0, SCALES = T::STAYS ? RESULTS : T::LDS;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::STAYS ? T::LDS : T::LDS + 4 * S::BYTES];
  TileOrder order;
  order.init(blockIdx.x, gridDim.x, g.ta, g.tb);
  int ia, ib;
  if (!order.get(0, ia, ib)) return;
  const int k0 = blockIdx.y * g.slice, stages = min(g.slice, g.nk - k0);
  T t;
  t.init(lds, 0);
  t.a.init(g.kp, t.wave, t.lane, t.wa);
  t.b.init(g.kp, t.wave, t.lane, t.wb);
  t.tail = 0;
  uint8_t* results = lds + RESULTS + t.wave * (4096 * PB);
  const int scales = SCALES + t.wave * (T::STAYS ? 4096 * PB : S::BYTES);
  auto locate = [&](bool any, Stretch& a, Stretch& b) {
    const int o0 = ia * WA, n = any ? stages : 0;
    const int64_t t0 = (int64_t)ib * WB, kb = (int64_t)k0 * 128;
    a.init(g.wc + (int64_t)o0 * g.kp + kb, (int64_t)min(WA, g.out - o0) * g.kp - kb, T::A::STEP, n);
    b.init(g.ac + t0 * g.kp + kb, min((int64_t)WB, g.n - t0) * g.kp - kb, T::B::STEP, n);
  };
  locate(true, t.a.mem, t.b.mem);
  t.start();
  bool more = true;
  int stored = 0;
  for (int r = 1; more; ++r) {
    const int64_t row0 = (int64_t)ib * WB + t.wb;
    const int c0 = ia * WA + t.wa;
    more = order.get(r, ia, ib);
    locate(more, t.an, t.bn);
    S::fetch(g, t.base + scales, c0, row0);
    constexpr int STORES = MB / PB * NB * (YBF16 ? 4 * PB / 2 : 4 * PB);
    t.template multiply<STORES>(max(2, stages), __builtin_amdgcn_readfirstlane(stored));
    if (!T::STAYS) wait_and_barrier<0>();
    S sc;
    sc.take(lds + scales);
    if (gridDim.y > 1) {
      float* part = static_cast<float*>(g.Y) + blockIdx.y * g.n * (int64_t)g.out;
      store_int8<false, true, PB>(t.acc, results, sc, g, part, g.ld, row0, c0);
      stored = 0;
    } else {
      stored = store_int8<YBF16, false, PB>(t.acc, results, sc, g, g.Y, g.ld, row0, c0);
    }
    if (!T::STAYS) return;
    t.clear();
  }
  wait_and_barrier<0>();  // nothing may still be writing LDS when the workgroup ends
}

// The slices' partial sums added; scales, bias, ReLU and the result's type. V columns of a row a thread.
template <bool YBF16, int V>
__global__ __launch_bounds__(256) void k_int8_join(const MatmulArgs g, const int* __restrict__ part, int slices) {
  const int per_row = (g.out + V - 1) / V;
  const int64_t total = g.n * per_row, stride = g.n * g.out;
  const float low = g.relu ? 0.f : -__builtin_inff();
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    const int64_t row = e / per_row;
    const int c = (int)(e - row * per_row) * V;
    const int* p = part + row * g.out + c;
    int sum[V];
#pragma unroll
    for (int q = 0; q < V; ++q) sum[q] = 0;
#pragma unroll 4
    for (int s = 0; s < slices; ++s) {
      if constexpr (V == 4) {
        const i32x4 v = *reinterpret_cast<const i32x4*>(p + s * stride);
#pragma unroll
        for (int q = 0; q < V; ++q) sum[q] += v[q];
      } else {
        sum[0] += p[s * stride];
      }
    }
    const float t = g.as[row];
#pragma unroll
    for (int q = 0; q < V; ++q) {
      const float y = int8_result((float)sum[q], t, g.ws[c + q], g.bias ? g.bias[c + q] : 0.f, low);
      if (YBF16) static_cast<uint16_t*>(g.Y)[row * g.ld + c + q] = (uint16_t)bf16_bits(y);
      else static_cast<float*>(g.Y)[row * g.ld + c + q] = y;
    }
  }
}

// Tiles (along out, along tokens), stages of the ring, and what a round of 256 of them takes, one to a CU: us for 128 columns
// of k and for the rest. Fitted to 110 sizes from 17 x 65 x 64 to 16384 x 4096 x 11008; the tile that these times choose is 3 %
// slower than the best one on average, 35 % at worst. The large tiles' rest is mostly that of all results leaving at once.
struct Tile {
  int wa, wb, ring;
  double step, rest;
};
constexpr Tile TILES[] = {{64, 64, 4, 0.23, 1.2},   {128, 64, 3, 0.38, 1.6},   {128, 128, 2, 0.56, 3.0}, {128, 128, 4, 0.47, 4.4},
                          {256, 128, 2, 0.75, 7.6}, {256, 192, 2, 0.90, 12.2}, {256, 256, 2, 1.08, 15.8}};

struct MatmulPlan {
  int tile;    // of TILES
  int slices;  // of k
};

// The fastest by the times above. Workgroups of tiles that fit a CU together mix their rounds, so those count in parts. Slices
// of k, joined by another launch of at least 3 us, where few tiles have a long sum each: 64 x 11008 x 4096 takes 17 us with
// 4 of them and 30 with one, but 200 x 4096 x 4096 (256 tiles of 64) 11 with one and 16 with two.
MatmulPlan matmul_plan(int64_t n, int64_t in, int64_t out) {
  MatmulPlan best = {0, 1};
  double least = 1e300;
  for (int i = 0; i < 7; ++i) {
    const Tile& t = TILES[i];
    const int64_t tiles = ceil_div(out, t.wa) * ceil_div(n, t.wb), nk = ceil_div(in, 128);
    for (int s = 1; s <= 8; s *= 2) {
      if (s > 1 && (tiles * s > 512 || nk < 4 * s)) break;
      const double rounds = tiles * s / 256.0;
      double us = (i < 3 ? std::max(1.0, rounds) : std::ceil(rounds)) * (ceil_div(nk, s) * t.step + t.rest);
      if (s > 1) us += 3.2 + (s + 1) * (double)n * out * 1e-6;
      if (us < least) least = us, best = {i, s};
    }
  }
  return best;
}

template <bool YBF16>
void matmul_go(int tile, dim3 grid, hipStream_t stream, const MatmulArgs& g) {
#define GPTQ_GO(I, OCC)                                                                                                    \
  case I:                                                                                                                  \
    hipLaunchKernelGGL((k_int8_matmul<YBF16, TILES[I].wa, TILES[I].wb, TILES[I].wa / 64, TILES[I].wb / 64, TILES[I].ring, OCC>), \
                       grid, dim3(256), 0, stream, g);                                                                     \
    break
  switch (tile) {
    GPTQ_GO(0, 2);
    GPTQ_GO(1, 2);
    GPTQ_GO(2, 2);
    GPTQ_GO(3, 1);
    GPTQ_GO(4, 1);
    GPTQ_GO(5, 1);
    GPTQ_GO(6, 1);
  }
#undef GPTQ_GO
}

}  // namespace

size_t int8_matmul_ws_bytes(int64_t n, int64_t in, int64_t out) {
  if (int8_few(n, in, out)) return 0;
  const MatmulPlan p = matmul_plan(n, in, out);
  return p.slices > 1 ? align_up((size_t)p.slices * n * out * 4, 256) : 0;
}

hipError_t int8_matmul_launch(const Int8Matrix& a, const Int8Matrix& w, const float* bias, int relu, void* Y, int y_dtype,
                              int64_t ld_y, void* ws, hipStream_t stream) {
  if (int8_few(a.rows, a.cols, w.rows)) return int8_matmul_few_launch(a, w, bias, relu, Y, y_dtype, ld_y, stream);
  const MatmulPlan p = matmul_plan(a.rows, a.cols, w.rows);
  const Tile& shape = TILES[p.tile];
  const bool bf16 = y_dtype == GPTQ_BF16;
  MatmulArgs g = {};
  g.kp = (int)int8_code_row(a.cols);
  g.wc = w.codes, g.ws = w.scales, g.bias = bias, g.out = (int)w.rows, g.relu = relu;
  g.ta = (int)ceil_div(w.rows, shape.wa), g.nk = (int)ceil_div(a.cols, 128);
  g.slice = (int)ceil_div(g.nk, p.slices);
  const int slices = (int)ceil_div(g.nk, g.slice);
  // at most 2^20 tiles a launch (sums over slices have far fewer)
  const int64_t rows_max = p.slices > 1 ? a.rows : std::max<int64_t>(1, ((int64_t)1 << 20) / g.ta) * shape.wb;
  for (int64_t r = 0; r < a.rows; r += rows_max) {
    g.n = std::min(rows_max, a.rows - r);
    g.tb = (int)ceil_div(g.n, shape.wb);
    g.ac = a.codes + r * g.kp, g.as = a.scales + r;
    g.Y = static_cast<uint8_t*>(Y) + r * ld_y * (bf16 ? 2 : 4), g.ld = ld_y;
    // Whole lines leave past the caches' reuse (16384 x 4096 x 11008 630 us, with it 636; 8000 x 256 x 8000 49 and 55). Where
    // rows are not aligned to lines, the caches have to join what two stores of the large tiles leave of one (11286 x 914 x
    // 4830 with 256 x 256 tiles 114 us, past them 134).
    const int line = p.tile < 4 ? 4 : 128;
    g.past = slices == 1 && (reinterpret_cast<uintptr_t>(g.Y) | (uintptr_t)(ld_y * (bf16 ? 2 : 4))) % line == 0;
    if (slices > 1) g.Y = ws, g.ld = w.rows;
    const dim3 grid(tile_grid((int64_t)g.ta * g.tb, shape.wa == 256 ? 256 : 1 << 30), (unsigned)slices);
    bf16 ? matmul_go<true>(p.tile, grid, stream, g) : matmul_go<false>(p.tile, grid, stream, g);
  }
  if (slices > 1) {
    g.Y = Y, g.ld = ld_y;
    const bool four = w.rows % 4 == 0;
    const dim3 grid((unsigned)std::min<int64_t>(8192, ceil_div(a.rows * (four ? w.rows / 4 : w.rows), 256)));
    const auto kernel = four ? (bf16 ? k_int8_join<true, 4> : k_int8_join<false, 4>)
                             : (bf16 ? k_int8_join<true, 1> : k_int8_join<false, 1>);
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, g, static_cast<const int*>(ws), slices);
  }
  return hipGetLastError();
}

size_t int8_linear_ws_bytes(int64_t n, int64_t in, int64_t out) {
  if (int8_few_fused(n, in)) return 0;
  return align_up(n * int8_code_row(in), 256) + align_up(n * 4, 256) + int8_matmul_ws_bytes(n, in, out);
}

hipError_t int8_linear_launch(const void* X, int x_dtype, int64_t n, int64_t ld_x, const Int8Matrix& w, const float* bias,
                              int relu, void* Y, int y_dtype, int64_t ld_y, void* ws, hipStream_t stream) {
  if (int8_few_fused(n, w.cols)) return int8_linear_few_launch(X, x_dtype, n, ld_x, w, bias, relu, Y, y_dtype, ld_y, stream);
  int8_t* codes = static_cast<int8_t*>(ws);
  float* scales = reinterpret_cast<float*>(codes + align_up(n * int8_code_row(w.cols), 256));
  uint8_t* rest = reinterpret_cast<uint8_t*>(scales) + align_up(n * 4, 256);
  const hipError_t e = int8_quantize_launch(X, x_dtype, n, w.cols, ld_x, codes, scales, stream);
  if (e != hipSuccess) return e;
  const Int8Matrix a = {codes, scales, n, w.cols};
  return int8_matmul_launch(a, w, bias, relu, Y, y_dtype, ld_y, rest, stream);
}

}  // namespace gptq
