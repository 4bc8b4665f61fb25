// Y = A W^T (+ bias) (ReLU) for at most 16 tokens, A in MX form or quantized on its way in: the form for single tokens.
//
// What bounds it is the latency of a launch and of memory (W is read once: 8.9 MB for 4096 x 4096, under 2 us at the rate
// of a large copy). Each workgroup therefore forms 16 rows of W on its own, its waves splitting the sum over k and joining
// their parts in LDS. v_mfma_scale_f32_16x16x128_f8f6f4 multiplies: lane l = 16 g + r of an operand holds row r, E2M1
// elements of columns 32 g .. 32 g + 31 of the 128, or E4M3 elements of columns 16 g .. 16 g + 15 and
// 64 + 16 g .. 64 + 16 g + 15, and block g's scale byte. Waves take every eighth 512 columns, a 16-byte load bringing a
// row's scale bytes for all of them: a load of one byte from each of 16 rows costs as much as one of 16 bytes, and with
// scale bytes loaded for each 128 columns 12 x 11008 x 4096 (E4M3) took 15.0 us, 10.3 of them for the rest.
//
// Few tokens are quantized by every workgroup in registers, in that layout (a lane loads just the columns whose codes it
// holds), which saves a launch; more of them (mx_few_fused) in a launch of their own, since every workgroup would load and
// convert them all. 1 x 4096 x 4096 takes 4.8 us of which an empty kernel takes 2.7, 12 x 11008 x 4096 12.7 us with that.
#include <algorithm>

#include "mx_codec.h"

namespace gptq {

namespace {

constexpr int FEW_WAVES = 8;
enum { FROM_CODES = 0, FROM_F32 = 1, FROM_BF16 = 2 };

struct FewArgs {
  const void* X;      // FROM_CODES: A's codes
  const uint8_t* xs;  // and scale bytes
  int64_t ldx;        // elements of a row of X, or bytes of one of codes
  const uint8_t *wc, *ws;
  int64_t crow, srow;
  const float* bias;
  void* Y;
  int64_t ldy;
  int n, in, out, relu;
};

// what a lane holds of 512 columns: its row's codes and scale bytes, 4 x 32 columns of its token
template <int SRC>
struct FewPart {
  uint4 w[4], s;
  Chunk<SRC == FROM_BF16> x[4][4];
};
template <>
struct FewPart<FROM_CODES> {
  uint4 w[4], s, x[4][2], xs;
};

// The buffers that a workgroup reads, and this lane's places in them. Reads outside give zeros, so nothing branches.
template <int FMT, int SRC>
struct FewSource {
  static constexpr int ES = SRC == FROM_CODES ? 1 : SRC == FROM_BF16 ? 2 : 4;
  __amdgpu_buffer_rsrc_t w, s, x, xs;
  int woff, soff, xoff, xsoff, col;  // col: this lane's first column of each 128

  __device__ __forceinline__ void init(const FewArgs& a, int o0, int r, int g) {
    const int rows = min(16, a.out - o0);
    w = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.wc + o0 * a.crow), 0, (int)(rows * a.crow), 0x00020000);
    s = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.ws + o0 * a.srow), 0, (int)(rows * a.srow), 0x00020000);
    woff = (int)(r * a.crow) + 16 * g, soff = (int)(r * a.srow);
    if constexpr (SRC == FROM_CODES) {
      x = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(a.X), 0, (int)(a.n * a.ldx), 0x00020000);
      xs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.xs), 0, (int)(a.n * a.srow), 0x00020000);
      xoff = (int)(r * a.ldx) + 16 * g, xsoff = soff, col = 0;
    } else {
      x = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(a.X), 0, (int)(((a.n - 1) * a.ldx + a.in) * ES), 0x00020000);
      col = (FMT == GPTQ_MX_E2M1 ? 32 : 16) * g;
      xoff = r < a.n ? (int)(r * a.ldx + col) * ES : (int)0x80000000;
    }
  }
};

__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t r, int off) {
  const i32x4 v = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// Columns 512 u .. 512 u + 511; what lies past the last 128 repeats them and is not used.
// VEC: X's rows are 16-byte aligned, their length a multiple of 8, and all of it lies within 2^31 bytes
template <int FMT, int SRC, bool VEC>
__device__ __forceinline__ void few_load(FewPart<SRC>& p, const FewSource<FMT, SRC>& b, const FewArgs& a, int u, int chunks,
                                         int r) {
  p.s = load16(b.s, b.soff + u * 16);
  if constexpr (SRC == FROM_CODES) p.xs = load16(b.xs, b.xsoff + u * 16);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int c = min(4 * u + j, chunks - 1);
    p.w[j] = load16(b.w, b.woff + c * 64);
    if constexpr (SRC == FROM_CODES) {
      constexpr int ROW = FMT == GPTQ_MX_E2M1 ? 64 : 128;
#pragma unroll
      for (int q = 0; q < (FMT == GPTQ_MX_E2M1 ? 1 : 2); ++q) p.x[j][q] = load16(b.x, b.xoff + c * ROW + q * 64);
    } else {
      constexpr bool XBF16 = SRC == FROM_BF16;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int dc = FMT == GPTQ_MX_E2M1 ? 8 * q : 64 * (q >> 1) + 8 * (q & 1), col = 128 * c + dc;
        Chunk<XBF16>& x = p.x[j][q];
        if constexpr (VEC) {
          const int off = b.col < a.in - col ? b.xoff + col * b.ES : (int)0x80000000;
#pragma unroll
          for (int k = 0; k < (XBF16 ? 1 : 2); ++k) {
            const uint4 v = load16(b.x, off + 16 * k);
            x.w[4 * k] = v.x, x.w[4 * k + 1] = v.y, x.w[4 * k + 2] = v.z, x.w[4 * k + 3] = v.w;
          }
        } else if (r < a.n && b.col + col < a.in) {
          x = load_chunk<XBF16>(a.X, r * a.ldx + b.col + col, b.col + col, a.in);
        } else {
#pragma unroll
          for (int k = 0; k < (XBF16 ? 4 : 8); ++k) x.w[k] = 0u;
        }
      }
    }
  }
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

// the J-th 128 columns of the part
template <int FMT, int SRC, int J>
__device__ __forceinline__ void few_multiply(const FewPart<SRC>& p, int g, f32x4& acc) {
  i32x8 x = {0, 0, 0, 0, 0, 0, 0, 0};
  uint32_t byte;  // in the low 8 bits; 255 makes its products NaN whatever the codes
  if constexpr (SRC == FROM_CODES) {
    byte = word_of(p.xs, J) >> (8 * g);
#pragma unroll
    for (int q = 0; q < (FMT == GPTQ_MX_E2M1 ? 1 : 2); ++q)
      x[4 * q] = (int)p.x[J][q].x, x[4 * q + 1] = (int)p.x[J][q].y, x[4 * q + 2] = (int)p.x[J][q].z, x[4 * q + 3] = (int)p.x[J][q].w;
  } else if constexpr (FMT == GPTQ_MX_E2M1) {
    constexpr bool XBF16 = SRC == FROM_BF16;
    uint32_t top = chunk_max<XBF16>(p.x[J][0]);
#pragma unroll
    for (int q = 1; q < 4; ++q) top = max_join<XBF16>(top, chunk_max<XBF16>(p.x[J][q]));
    byte = scale_byte<FMT>(max_bits<XBF16>(top));
    const float scale = __uint_as_float(byte << 23);
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = (int)encode4<XBF16>(p.x[J][q], scale);
  } else {
    constexpr bool XBF16 = SRC == FROM_BF16;
    // a block lies in two neighbouring groups of 16 lanes: blocks 0 and 1 in their first 16 columns, 2 and 3 in the others
    uint32_t b[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t top = max_join<XBF16>(chunk_max<XBF16>(p.x[J][2 * q]), chunk_max<XBF16>(p.x[J][2 * q + 1]));
      const auto pair = __builtin_amdgcn_permlane16_swap(top, top, false, false);
      b[q] = scale_byte<FMT>(max_bits<XBF16>(max_join<XBF16>(pair[0], pair[1])));
      const float scale = __uint_as_float(b[q] << 23);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint2 v = encode8<XBF16>(p.x[J][2 * q + k], scale);
        x[4 * q + 2 * k] = (int)v.x, x[4 * q + 2 * k + 1] = (int)v.y;
      }
    }
    const auto t = __builtin_amdgcn_permlane32_swap(b[0], b[1], false, false);  // blocks 0 0 2 2 and 1 1 3 3
    byte = (g & 1) ? t[1] : t[0];
  }
  const i32x8 w = {(int)p.w[J].x, (int)p.w[J].y, (int)p.w[J].z, (int)p.w[J].w, 0, 0, 0, 0};
  const int ws = (int)(word_of(p.s, J) >> (8 * g));
  constexpr int FB = FMT == GPTQ_MX_E2M1 ? 4 : 0;
  if constexpr (FMT == GPTQ_MX_E4M3) {
    i32x8 hi, lo;
    split_e4m3(x, hi, lo);
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, lo, acc, 4, FB, 0, ws, 0, (int)byte);
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, hi, acc, 4, FB, 0, ws, 0, (int)byte);
  } else {
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, acc, 4, FB, 0, ws, 0, (int)byte);
  }
}

template <int FMT, int SRC, bool VEC, bool YBF16>
__global__ __launch_bounds__(64 * FEW_WAVES) void k_mx_few(const FewArgs a) {
  __shared__ float red[FEW_WAVES][16][20];
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int o0 = blockIdx.x * 16;
  const int chunks = (a.in + 127) / 128;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const int units = (chunks + 3) / 4;
  FewSource<FMT, SRC> src;
  src.init(a, o0, r, g);
  FewPart<SRC> part;
  for (int u = wave; u < units; u += FEW_WAVES) {
    few_load<FMT, SRC, VEC>(part, src, a, u, chunks, r);
    __builtin_amdgcn_sched_barrier(0);  // all loads first
    few_multiply<FMT, SRC, 0>(part, g, acc);
    if (4 * u + 1 < chunks) few_multiply<FMT, SRC, 1>(part, g, acc);
    if (4 * u + 2 < chunks) few_multiply<FMT, SRC, 2>(part, g, acc);
    if (4 * u + 3 < chunks) few_multiply<FMT, SRC, 3>(part, g, acc);
  }
  // register i of lane 16 g + r: W's row 4 g + i, token r
  *reinterpret_cast<float4*>(&red[wave][r][4 * g]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  if (threadIdx.x < 256) {
    const int tok = threadIdx.x / 16, o = threadIdx.x % 16, c = o0 + o;
    if (tok >= a.n || c >= a.out) return;
    float y = 0.f;
#pragma unroll
    for (int w = 0; w < FEW_WAVES; ++w) y += red[w][tok][o];
    if (a.bias) y += a.bias[c];
    if (a.relu) y = relu_nan(y);
    if (YBF16) static_cast<uint16_t*>(a.Y)[tok * a.ldy + c] = (uint16_t)bf16_bits(y);
    else static_cast<float*>(a.Y)[tok * a.ldy + c] = y;
  }
}

template <int FMT, int SRC>
void few_go(bool vec, bool ybf16, hipStream_t stream, const FewArgs& a) {
  const dim3 grid((unsigned)ceil_div(a.out, 16)), block(64 * FEW_WAVES);
  if (vec || SRC == FROM_CODES) {
    if (ybf16) hipLaunchKernelGGL((k_mx_few<FMT, SRC, true, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((k_mx_few<FMT, SRC, true, false>), grid, block, 0, stream, a);
  } else if constexpr (SRC != FROM_CODES) {
    if (ybf16) hipLaunchKernelGGL((k_mx_few<FMT, SRC, false, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((k_mx_few<FMT, SRC, false, false>), grid, block, 0, stream, a);
  }
}

}  // namespace

hipError_t mx_linear_few_launch(const void* X, int x_dtype, int64_t n, int64_t ld_x, int act_fmt, const MxMatrix& w,
                                const float* bias, int relu, void* Y, int y_dtype, int64_t ld_y, hipStream_t stream) {
  const FewArgs a = {X,  nullptr, ld_x, w.codes, w.scales, mx_code_row(w.cols, GPTQ_MX_E2M1), mx_scale_row(w.cols), bias,
                     Y, ld_y, (int)n, (int)w.cols, (int)w.rows, relu};
  const bool vec = vec_rows(X, ld_x, x_dtype) && w.cols % 8 == 0 && (n - 1) * ld_x + w.cols < (int64_t)1 << 28;
  const bool yb = y_dtype == GPTQ_BF16;
  if (act_fmt == GPTQ_MX_E2M1)
    x_dtype == GPTQ_BF16 ? few_go<GPTQ_MX_E2M1, FROM_BF16>(vec, yb, stream, a) : few_go<GPTQ_MX_E2M1, FROM_F32>(vec, yb, stream, a);
  else
    x_dtype == GPTQ_BF16 ? few_go<GPTQ_MX_E4M3, FROM_BF16>(vec, yb, stream, a) : few_go<GPTQ_MX_E4M3, FROM_F32>(vec, yb, stream, a);
  return hipGetLastError();
}

hipError_t mx_matmul_few_launch(const MxMatrix& x, const MxMatrix& w, const float* bias, int relu, void* Y, int y_dtype,
                                int64_t ld_y, hipStream_t stream) {
  const FewArgs a = {x.codes, x.scales, mx_code_row(x.cols, x.fmt), w.codes, w.scales, mx_code_row(w.cols, GPTQ_MX_E2M1),
                     mx_scale_row(w.cols), bias, Y, ld_y, (int)x.rows, (int)w.cols, (int)w.rows, relu};
  const bool yb = y_dtype == GPTQ_BF16;
  x.fmt == GPTQ_MX_E2M1 ? few_go<GPTQ_MX_E2M1, FROM_CODES>(true, yb, stream, a) : few_go<GPTQ_MX_E4M3, FROM_CODES>(true, yb, stream, a);
  return hipGetLastError();
}

}  // namespace gptq
