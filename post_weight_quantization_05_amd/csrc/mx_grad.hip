// Backward pass of a quantized linear layer on gfx950: dX = dY W (masked by the ReLU that made the layer's input)
// and dW = dY^T A with db = column sums of dY.
//
// The quantized operand's values (4 significant bits at most, times a power of two) are exact in bf16, so it is first
// written out in bf16 and the products run on the bf16 matrix cores, exact and summed in fp32. It is the first operand,
// so that a lane of the result holds four consecutive columns.
#include <algorithm>

#include "mx_codec.h"
#include "mx_tile.h"

namespace gptq {

namespace {

struct GradArgs {
  const uint16_t *F, *S;       // first operand [k][f]; second [s][k] (dX) or [k][s] (dW)
  int64_t ldf, lds;            // their rows' elements
  int64_t nk, slice;           // k; k of a slice (a multiple of 64)
  int64_t ns;                  // rows of the result
  int nf, ta, tb;              // its columns; tiles along both
  const uint8_t *mc, *ms;      // mask
  int64_t mrow, msrow;
  void* Y;
  int64_t ld;
  int accumulate;
  const double* sums;          // column sums' slices, for db
  int sum_slices;
  float* db;
};

// Codes of the mask's 4 consecutive columns from c on (a multiple of 4, below the row's padding)
template <int MASK>
__device__ __forceinline__ uint32_t mask_codes(const GradArgs& g, int64_t row, int c) {
  if (MASK == 1) return *reinterpret_cast<const uint16_t*>(g.mc + row * g.mrow + (c >> 1));
  return *reinterpret_cast<const uint32_t*>(g.mc + row * g.mrow + c);
}

// whether the mask's value at one of them is > 0, its block being finite
template <int MASK>
__device__ __forceinline__ bool mask_open(uint32_t codes, int q) {
  if (MASK == 1) return (codes >> (4 * q) & 15u) - 1u < 7u;
  return (codes >> (8 * q) & 255u) - 1u < 0x7Eu;
}

// zero where the mask's value is not > 0
template <int MASK>
__device__ __forceinline__ float masked(const GradArgs& g, int64_t row, int c, float v) {
  if constexpr (MASK != 0) {
    const uint32_t codes = mask_codes<MASK>(g, row, c & ~3);
    if (g.ms[row * g.msrow + (c >> 5)] == 255 || !mask_open<MASK>(codes, c & 3)) v = 0.f;
  }
  return v;
}
template <int MASK, int V, int IT, int BLOCKS>
struct StoreMasked {
  static constexpr int J = V / 4;  // groups of four columns of a row; IT J of them fill a word of flags
  static_assert(IT * J <= 8, "a word of flags a block");
  const GradArgs& g;
  uint32_t codes[4][IT][J], scale[4][IT], flags[BLOCKS];
  __device__ __forceinline__ void columns(int) {}
  __device__ __forceinline__ void row(int set, int it, int64_t row, int c) {
    if constexpr (MASK != 0) {
      scale[set][it] = g.ms[row * g.msrow + (c >> 5)];
#pragma unroll
      for (int p = 0; p < J; ++p) codes[set][it][p] = mask_codes<MASK>(g, row, c + 4 * p);
    }
  }
  // Four codes at once: the top bit of each is set in `open` where the value is > 0 and a number. Group j's flags lie j
  // places further down, E2M1's groups 4 to 7 in the upper half.
  __device__ __forceinline__ void keep(int set, int b) {
    if constexpr (MASK != 0) {
      uint32_t f = 0;
#pragma unroll
      for (int it = 0; it < IT; ++it)
#pragma unroll
        for (int p = 0; p < J; ++p) {
          const uint32_t w = codes[set][it][p];
          const int j = it * J + p;
          uint32_t open;
          if (MASK == 1) {
            open = ((w & 0x7777u) + 0x7777u) & ~w & 0x8888u;
          } else {
            const uint32_t m = w & 0x7F7F7F7Fu;
            open = (m + 0x7F7F7F7Fu) & ~(m + 0x01010101u) & ~w & 0x80808080u;
          }
          open = scale[set][it] == 255u ? 0u : open;
          f |= MASK == 1 ? open >> (3 - (j & 3)) << (16 * (j >> 2)) : open >> (7 - j);
        }
      flags[b] = f;
    }
  }
  __device__ __forceinline__ float one(int64_t row, int c, float v) { return masked<MASK>(g, row, c, v); }
  __device__ __forceinline__ void finish(int b, int it, float (&v)[V]) {
    if constexpr (MASK != 0) {
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const int j = it * J + (q >> 2), at = MASK == 1 ? 4 * (q & 3) + (j & 3) + 16 * (j >> 2) : 8 * (q & 3) + j;
        v[q] = __uint_as_float(__float_as_uint(v[q]) & (uint32_t)((int)(flags[b] << (31 - at)) >> 31));
      }
    }
  }
};

template <bool GRAD_INPUT, bool YBF16, int MASK, int WA, int WB, int MB, int NB, int OCC>
__global__ __launch_bounds__(256, OCC) void k_mx_grad(const GradArgs g) {
  using T = TileProduct<K_BF16T, GRAD_INPUT ? K_BF16 : K_BF16T, WA, WB, MB, NB>;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[T::LDS];
  if (!GRAD_INPUT && g.db && blockIdx.y == 0) {
    for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < g.ns; c += (int64_t)gridDim.x * 256) {
      double sum = g.accumulate ? (double)g.db[c] : 0.0;
      for (int s = 0; s < g.sum_slices; ++s) sum += g.sums[s * g.ns + c];
      g.db[c] = (float)sum;
    }
  }
  TileOrder order;
  order.init(blockIdx.x, gridDim.x, g.ta, g.tb);
  int ia, ib;
  if (!order.get(0, ia, ib)) return;
  const int64_t k0 = blockIdx.y * g.slice, nk = min(g.slice, g.nk - k0);
  const int stages = (int)((nk + 63) / 64);
  T t;
  t.init(lds, 0);
  t.a.init(g.ldf * 2, t.wave, t.lane, t.wa);
  t.b.init(g.lds * 2, t.wave, t.lane, t.wb);
  t.tail = 0;
  // bytes from a tile's first element to the end of its last row, rounded up to whole 16-byte chunks; what a tile reads
  // behind a row's end before that only reaches results that are not stored
  auto locate = [&](bool any, Stretch& a, Stretch& b) {
    const int f0 = ia * WA, n = any ? stages : 0;
    const int64_t s0 = (int64_t)ib * WB;
    a.init(g.F + k0 * g.ldf + f0, ((nk - 1) * g.ldf + ((g.nf + 7) / 8 * 8 - f0)) * 2, (int)(64 * g.ldf * 2), n);
    if (GRAD_INPUT) {
      const int64_t rows = min((int64_t)WB, g.ns - s0);
      b.init(g.S + s0 * g.lds + k0, ((rows - 1) * g.lds + (int64_t)stages * 64) * 2, T::B::STEP, n);
    } else {
      b.init(g.S + k0 * g.lds + s0, ((nk - 1) * g.lds + ((g.ns + 7) / 8 * 8 - s0)) * 2, (int)(64 * g.lds * 2), n);
    }
  };
  locate(true, t.a.mem, t.b.mem);
  t.start();
  bool more = true;
  for (int r = 1; more; ++r) {
    const int64_t row0 = (int64_t)ib * WB + t.wb;
    const int c0 = ia * WA + t.wa;
    more = order.get(r, ia, ib);
    locate(more, t.an, t.bn);
    t.multiply(max(2, stages));
    if (!T::STAYS) wait_and_barrier<0>();
    uint8_t* buf = T::STAYS ? lds + T::LDS - 4 * 4096 * T::PB : lds;
    if (gridDim.y > 1) {
      float* part = static_cast<float*>(g.Y) + blockIdx.y * g.ns * (int64_t)g.nf;
      store_rows<false, T::PB>(t.acc, buf, part, g.nf, row0, g.ns, c0, g.nf, false, StoreAsIs());
    } else {
      constexpr int V = YBF16 ? 8 : 4;
      StoreMasked<MASK, V, 16 * T::PB / V, MB / T::PB * NB> done = {g, {}, {}, {}};
      store_rows<YBF16, T::PB>(t.acc, buf, g.Y, g.ld, row0, g.ns, c0, g.nf, g.accumulate, done);
    }
    if (!T::STAYS) return;
    t.clear();
  }
  wait_and_barrier<0>();  // nothing may still be writing LDS when the workgroup ends
}

// The slices' partial products, added in their order; mask, accumulation and the result's type. Four columns a thread.
template <bool YBF16, int MASK>
__global__ __launch_bounds__(256) void k_mx_grad_join(const GradArgs g, const float* __restrict__ part, int slices) {
  const int per_row = (g.nf + 3) / 4;
  const int64_t total = g.ns * per_row, stride = g.ns * (int64_t)g.nf;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (int64_t)gridDim.x * 256) {
    const int64_t row = e / per_row;
    const int c = (int)(e - row * per_row) * 4;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < slices; ++s)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (c + q < g.nf) v[q] += part[s * stride + row * g.nf + c + q];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (c + q >= g.nf) continue;
      v[q] = masked<MASK>(g, row, c + q, v[q]);
      if (YBF16) {
        static_cast<uint16_t*>(g.Y)[row * g.ld + c + q] = (uint16_t)bf16_bits(v[q]);
      } else {
        float* p = static_cast<float*>(g.Y) + row * g.ld + c + q;
        *p = g.accumulate ? *p + v[q] : v[q];
      }
    }
  }
}

// What both products need first, in one launch: workgroups 0 .. nb_values - 1 write the quantized operand's values in
// bf16; the next nb_pad copy dY to rows of kp columns, zeros behind the last; the rest add dY's columns in fp64, each 32
// columns of a slice of rows, eight row groups side by side (the slices are added in their order by the product).
struct PrepArgs {
  const uint8_t *codes, *scales;
  int cols, ks;
  int64_t units;
  uint16_t* F;
  int64_t ldf;
  const uint16_t* dY;
  int64_t ld, n;
  int out, kp;
  uint16_t* pad;
  double* sums;
  int64_t rows;  // of a slice
  unsigned nb_values, nb_pad, nb_cols;
};

template <int FMT>
__global__ __launch_bounds__(256) void k_mx_grad_prep(const PrepArgs a) {
  unsigned b = blockIdx.x;
  if (b < a.nb_values) {
    for (int64_t u = (int64_t)b * 4 + (threadIdx.x >> 6); u < a.units; u += (int64_t)a.nb_values * 4)
      dequantize_unit<FMT, true>(a.codes, a.scales, a.cols, a.ks, u, a.F, a.ldf);
    return;
  }
  b -= a.nb_values;
  if (b < a.nb_pad) {
    const int64_t total = a.n * (a.kp / 8);
    for (int64_t e = (int64_t)b * 256 + threadIdx.x; e < total; e += (int64_t)a.nb_pad * 256) {
      const int64_t row = e / (a.kp / 8);
      const int c = (int)(e - row * (a.kp / 8)) * 8;
      const Chunk<true> x = load_chunk<true>(a.dY, row * a.ld + c, c, a.out);
      *reinterpret_cast<uint4*>(a.pad + row * a.kp + c) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    }
    return;
  }
  b -= a.nb_pad;
  __shared__ double red[8][32];
  const int c = (int)(b % a.nb_cols) * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  const int64_t slice = b / a.nb_cols, r0 = slice * a.rows, r1 = min(a.n, r0 + a.rows);
  double sum = 0.0;
  if (c < a.out)
#pragma unroll 4
    for (int64_t k = r0 + g; k < r1; k += 8) sum += (double)__uint_as_float((uint32_t)a.dY[k * a.ld + c] << 16);
  red[g][threadIdx.x & 31] = sum;
  __syncthreads();
  if (g == 0 && c < a.out) {
#pragma unroll
    for (int q = 1; q < 8; ++q) sum += red[q][threadIdx.x];
    a.sums[slice * a.out + c] = sum;
  }
}

// sums: rows of a slice of the column sums (0: none are wanted)
hipError_t grad_prep(const MxMatrix& q, uint16_t* F, const uint16_t* dY, int64_t ld, int64_t n, int64_t out, uint16_t* pad,
                     double* sums, int64_t rows, hipStream_t stream) {
  PrepArgs a = {};
  a.codes = q.codes, a.scales = q.scales, a.cols = (int)q.cols, a.ks = (int)ceil_div(q.cols, UNIT);
  a.units = q.rows * a.ks, a.F = F, a.ldf = ceil_div(q.cols, 128) * 128;
  a.dY = dY, a.ld = ld, a.n = n, a.out = (int)out, a.kp = (int)ceil_div(out, 128) * 128, a.pad = pad;
  a.sums = sums, a.rows = rows, a.nb_cols = (unsigned)ceil_div(out, 32);
  a.nb_values = (unsigned)std::min<int64_t>((int64_t)1 << 20, ceil_div(a.units, 4));
  a.nb_pad = pad ? (unsigned)std::min<int64_t>(4096, ceil_div(n * (a.kp / 8), 256)) : 0;
  const unsigned nb_sum = rows ? a.nb_cols * (unsigned)ceil_div(n, rows) : 0;
  const dim3 grid(a.nb_values + a.nb_pad + nb_sum);
  if (q.fmt == GPTQ_MX_E2M1) hipLaunchKernelGGL((k_mx_grad_prep<GPTQ_MX_E2M1>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((k_mx_grad_prep<GPTQ_MX_E4M3>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

struct GradPlan {
  int tile;    // 0: 64 x 64, 1: 128 x 128, 2: 256 x 256
  int slices;
  int64_t slice;
};

GradPlan grad_plan(int64_t ns, int64_t nf, int64_t nk) {
  GradPlan p = {0, 1, std::max<int64_t>(64, (int64_t)align_up(nk, 64))};
  auto tiles = [&](int64_t w) { return ceil_div(ns, w) * ceil_div(nf, w); };
  // us with tiles of 64 / 128 / 256 (dX): 512 x 4096 x 4096 48 / 54 / 96, 1024 x 4096 x 4096 66 / 58 / 100,
  // 2048 x 4096 x 4096 109 / 75 / 91, 4096 x 4096 x 4096 200 / 131 / 114, 1500 x 2000 x 3000 (192 tiles of 128) 42 / 50 / -,
  // 8000 x 8000 x 256 87 / 61 / 68, 8000 x 8000 x 1024 224 / 144 / 134
  p.tile = tiles(256) >= 192 && nk >= 512 ? 2 : tiles(128) >= 224 ? 1 : 0;
  // Slices of k, joined by another launch, where the tiles leave places of the chip empty (three 64 x 64 tiles fit a CU)
  // and each slice has a long sum: 200 x 4096 x 4096 takes 37 us with 4 and 47 with one, dW 4096 x 1024 x 1024 36 and 44,
  // but 512 x 1024 x 1024 15.5 with two and 14.0 with one.
  const int64_t t = tiles(64 << p.tile), places = p.tile == 0 ? 768 : p.tile == 1 ? 512 : 256;
  if (t > 0) {
    const int64_t s = std::max<int64_t>(1, std::min<int64_t>({places / t, nk / 1024, 64}));
    p.slice = std::max<int64_t>(64, (int64_t)align_up(ceil_div(nk, s), 64));
  }
  p.slices = (int)std::max<int64_t>(1, ceil_div(nk, p.slice));
  return p;
}

size_t grad_part_bytes(const GradPlan& p, int64_t ns, int64_t nf) {
  return p.slices > 1 ? align_up((size_t)p.slices * ns * nf * 4, 256) : 0;
}

template <bool GI, bool B, int M>
void grad_go(int tile, dim3 grid, hipStream_t stream, const GradArgs& g) {
#define GPTQ_GO(WA, WB, MB, NB, OCC) \
  hipLaunchKernelGGL((k_mx_grad<GI, B, M, WA, WB, MB, NB, OCC>), grid, dim3(256), 0, stream, g)
  if (tile == 2) GPTQ_GO(256, 256, 4, 4, 1);
  else if (tile == 1) GPTQ_GO(128, 128, 2, 2, 2);
  else GPTQ_GO(64, 64, 1, 1, 3);
#undef GPTQ_GO
}

template <bool GI, bool B, int M>
hipError_t grad_run(const GradPlan& p, GradArgs g, float* part, hipStream_t stream) {
  const GradArgs fin = g;
  g.slice = p.slice;
  g.ta = (int)ceil_div(g.nf, 64 << p.tile);
  if (p.slices > 1) g.Y = part, g.ld = g.nf;
  g.tb = (int)ceil_div(g.ns, 64 << p.tile);
  grad_go<GI, B, M>(p.tile, dim3(tile_grid((int64_t)g.ta * g.tb, p.tile == 2 ? 256 : 1 << 30), (unsigned)p.slices), stream, g);
  if (p.slices > 1)
    hipLaunchKernelGGL((k_mx_grad_join<B, M>), dim3((unsigned)std::min<int64_t>(2048, ceil_div(g.ns * ceil_div(g.nf, 4), 256))),
                       dim3(256), 0, stream, fin, part, p.slices);
  return hipGetLastError();
}

// The tile product reads dY with 16-byte loads of whole chunks; where rows are not aligned, or a row's tail would
// bring its neighbour's numbers into the sum (dX), a padded copy is read instead.
bool dy_direct(const uint16_t* dY, int64_t ld, int64_t out, bool sum_over_out) {
  return vec_rows(dY, ld, GPTQ_BF16) && ld <= ((int64_t)1 << 20) && (!sum_over_out || out % 64 == 0);
}

constexpr int64_t ROWS_MAX = (int64_t)1 << 20;  // rows of dX a launch

}  // namespace

size_t mx_grad_input_ws_bytes(int64_t n, int64_t in, int64_t out) {
  const int64_t m = std::min(n, ROWS_MAX);
  return align_up(out * ceil_div(in, 128) * 256, 256) + align_up(m * ceil_div(out, 128) * 256, 256) +
         grad_part_bytes(grad_plan(m, in, out), m, in);
}

hipError_t mx_grad_input_launch(const uint16_t* dY, int64_t ld_dy, int64_t n, const MxMatrix& w, const MxMatrix* mask,
                                void* dX, int dx_dtype, int64_t ld_dx, void* ws, hipStream_t stream) {
  const int64_t in = w.cols, out = w.rows, ldf = ceil_div(in, 128) * 128, kp = ceil_div(out, 128) * 128;
  uint8_t* pad = static_cast<uint8_t*>(ws) + align_up(out * ldf * 2, 256);
  float* part = reinterpret_cast<float*>(pad + align_up(std::min(n, ROWS_MAX) * kp * 2, 256));
  for (int64_t r = 0; r < n; r += ROWS_MAX) {
    GradArgs g = {};
    g.F = static_cast<const uint16_t*>(ws), g.ldf = ldf, g.nk = out;
    g.S = dY + r * ld_dy, g.lds = ld_dy, g.ns = std::min(ROWS_MAX, n - r), g.nf = (int)in;
    const bool direct = dy_direct(g.S, ld_dy, out, true);
    MxMatrix q = w;
    if (r > 0) q.rows = 0;  // its values are there
    if (r == 0 || !direct) {
      const hipError_t e = grad_prep(q, static_cast<uint16_t*>(ws), g.S, ld_dy, g.ns, out,
                                     direct ? nullptr : reinterpret_cast<uint16_t*>(pad), nullptr, 0, stream);
      if (e != hipSuccess) return e;
    }
    if (!direct) g.S = reinterpret_cast<const uint16_t*>(pad), g.lds = kp;
    if (mask) {
      g.mrow = mx_code_row(in, mask->fmt), g.msrow = mx_scale_row(in);
      g.mc = mask->codes + r * g.mrow, g.ms = mask->scales + r * g.msrow;
    }
    g.Y = static_cast<uint8_t*>(dX) + r * ld_dx * (dx_dtype == GPTQ_BF16 ? 2 : 4), g.ld = ld_dx;
    // the plan of the first (largest) piece: its partial products fit the workspace
    const GradPlan p = grad_plan(std::min(n, ROWS_MAX), in, out);
    const int kind = !mask ? 0 : mask->fmt == GPTQ_MX_E2M1 ? 1 : 2;
    hipError_t s;
    if (dx_dtype == GPTQ_BF16)
      s = kind == 0 ? grad_run<true, true, 0>(p, g, part, stream)
                    : kind == 1 ? grad_run<true, true, 1>(p, g, part, stream) : grad_run<true, true, 2>(p, g, part, stream);
    else
      s = kind == 0 ? grad_run<true, false, 0>(p, g, part, stream)
                    : kind == 1 ? grad_run<true, false, 1>(p, g, part, stream) : grad_run<true, false, 2>(p, g, part, stream);
    if (s != hipSuccess) return s;
  }
  return hipSuccess;
}

namespace {
int64_t colsum_rows(int64_t n, int64_t out) {
  const int64_t want = std::max<int64_t>(1, 2048 / ceil_div(out, 32));  // about 2048 workgroups
  return std::max<int64_t>(256, ceil_div(n, std::min<int64_t>(want, 1024)));
}
}  // namespace

size_t mx_grad_weight_ws_bytes(int64_t n, int64_t in, int64_t out) {
  return align_up(n * ceil_div(in, 128) * 256, 256) + align_up(n * ceil_div(out, 128) * 256, 256) +
         grad_part_bytes(grad_plan(out, in, n), out, in) + align_up(ceil_div(n, colsum_rows(n, out)) * out * 8, 256);
}

hipError_t mx_grad_weight_launch(const uint16_t* dY, int64_t ld_dy, int64_t out, const MxMatrix& a, int accumulate,
                                 void* dW, int dw_dtype, int64_t ld_dw, float* db, void* ws, hipStream_t stream) {
  const int64_t n = a.rows, in = a.cols, ldf = ceil_div(in, 128) * 128, kp = ceil_div(out, 128) * 128;
  uint8_t* pad = static_cast<uint8_t*>(ws) + align_up(n * ldf * 2, 256);
  uint8_t* part = pad + align_up(n * kp * 2, 256);
  const GradPlan p = grad_plan(out, in, n);
  double* sums = reinterpret_cast<double*>(part + grad_part_bytes(p, out, in));
  GradArgs g = {};
  g.F = static_cast<const uint16_t*>(ws), g.ldf = ldf, g.nk = n, g.nf = (int)in;
  g.S = dY, g.lds = ld_dy, g.ns = out, g.Y = dW, g.ld = ld_dw, g.accumulate = accumulate;
  const int64_t rows = colsum_rows(n, out);
  if (n > 0) {
    const bool direct = dy_direct(dY, ld_dy, out, false);
    const hipError_t e = grad_prep(a, static_cast<uint16_t*>(ws), dY, ld_dy, n, out,
                                   direct ? nullptr : reinterpret_cast<uint16_t*>(pad), sums, db ? rows : 0, stream);
    if (e != hipSuccess) return e;
    if (!direct) g.S = reinterpret_cast<const uint16_t*>(pad), g.lds = kp;
  }
  g.db = db, g.sums = sums, g.sum_slices = (int)ceil_div(n, rows);
  const hipError_t s = dw_dtype == GPTQ_BF16 ? grad_run<false, true, 0>(p, g, reinterpret_cast<float*>(part), stream)
                                             : grad_run<false, false, 0>(p, g, reinterpret_cast<float*>(part), stream);
  return s;
}

}  // namespace gptq
