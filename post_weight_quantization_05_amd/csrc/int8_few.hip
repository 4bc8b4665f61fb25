// Y = A W^T s_a s_w (+ bias) (ReLU) for few tokens (int8_few), in codes or quantized on their way in: the form for single
// tokens.
//
// What bounds it is the latency of a launch and the reading of W (16.8 MB for 4096 x 4096, 3.4 us at the rate of a large copy).
// A workgroup forms 16 rows of W on its own, its waves splitting the sum over k and joining their parts in LDS.
// v_mfma_i32_16x16x64_i8 multiplies: lane l = 16 g + r of an operand holds row r, columns 16 g .. 16 g + 15 of the 64. A wave
// has its next loads in flight before the first product of those before.
//
// Few tokens are quantized by every workgroup, which saves a launch: its waves share them out, find each token's largest
// magnitude and leave the codes in LDS, while W's first columns are on their way.
#include <algorithm>

#include "int8_codec.h"
#include "rows.h"

namespace gptq {

namespace {

enum { FROM_CODES = 0, FROM_F32 = 1, FROM_BF16 = 2 };

struct FewArgs {
  const void* X;     // FROM_CODES: A's codes
  const float* xs;   // and scales
  int64_t ldx;
  const int8_t* wc;
  const float *ws, *bias;
  void* Y;
  int64_t ldy;
  int n, in, kp, out, relu;
};

__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t r, int off) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}

// The n tokens on their way to codes and scales in LDS, rows of `stride` bytes. n up to 8: 8 waves, or 4, 2, 1, share a token;
// more: a wave takes two. A lane holds at most eight times 8 columns (int8_few_fused) from the token's maximum to its codes.
template <bool XBF16>
struct FewTokens {
  Chunk<XBF16> x[8];
  int per, part, wave, times;  // waves of a token, this one's number, times that it takes 512 columns
  bool two;

  __device__ __forceinline__ int token(int i) const { return two ? wave + (i >> 2) * 8 : wave / per; }
  __device__ __forceinline__ int column(int i) const {
    return (((two ? i & 3 : i) * per + part) * 64 + (int)(threadIdx.x & 63)) * 8;
  }
  __device__ __forceinline__ bool used(const FewArgs& a, int i) const { return (two ? i & 3 : i) < times && token(i) < a.n; }

  __device__ __forceinline__ void load(const FewArgs& a) {
    wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    per = a.n == 1 ? 8 : a.n == 2 ? 4 : a.n <= 4 ? 2 : 1, part = wave % per, two = a.n > 8;
    times = (a.kp + 512 * per - 1) / (512 * per);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (used(a, i)) x[i] = load_full<XBF16>(a.X, token(i) * a.ldx + min(column(i), a.in - 8));
  }
  __device__ __forceinline__ void quantize(const FewArgs& a, int8_t* codes, int stride, float* scales, uint32_t* tops) {
    uint32_t top[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int over = column(i) - (a.in - 8);  // past the row's end: its last eight columns were read
      if (used(a, i) && over > 0) move_down<XBF16>(x[i], over);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (used(a, i)) top[i >> 2] = max(top[i >> 2], max_bits<XBF16>(chunk_max<XBF16>(x[i])));
    if (!two) top[0] = max(top[0], top[1]);
    top[0] = lanes_max<64>(top[0]);
    if (two) top[1] = lanes_max<64>(top[1]);
    if (per > 1) {
      if ((threadIdx.x & 63) == 0) tops[wave] = top[0];
      __syncthreads();
      for (int i = 0; i < per; ++i) top[0] = max(top[0], tops[wave - part + i]);
    }
    if (!two) top[1] = top[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!used(a, i)) continue;
      const int tok = token(i), c = column(i);
      const uint32_t t = top[i >> 2];
      if (c >= a.kp) continue;
      const float s = int8_scale(t);
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = chunk_at<XBF16>(x[i], q);
      *reinterpret_cast<uint2*>(codes + tok * stride + c) =
          t < 0x7F800000u ? int8_encode(v, s, __builtin_amdgcn_rcpf(s)) : make_uint2(0u, 0u);
      if (c == 0) scales[tok] = s;
    }
  }
};

// NT: groups of 16 tokens. NW: waves. UC: 64s of columns that are loaded together. 16 waves and 128 columns for codes: 1 x 4096 x
// 11008 10.9 us, 12 x 11008 x 4096 14.2 (8 waves and 512 columns 12.9 and 15.2, 256 columns 11.5 and 14.3, 64 columns and 16
// waves 12.4 and 16.1; loads of W past the caches' reuse change nothing).
template <int SRC, bool YBF16, int NT, int NW, int UC>
__global__ __launch_bounds__(64 * NW) void k_int8_few(const FewArgs a) {
  extern __shared__ __attribute__((aligned(16))) int8_t codes[];  // FROM_CODES: none
  __shared__ int red[NW][16 * NT][20];
  __shared__ float scales[16];
  __shared__ uint32_t tops[8];
  const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int o0 = blockIdx.x * 16;
  const int chunks = a.kp / 64, stride = a.kp + 16;  // rows of LDS on different banks
  const __amdgpu_buffer_rsrc_t w = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<int8_t*>(a.wc + (int64_t)o0 * a.kp), 0, min(16, a.out - o0) * a.kp, 0x00020000);
  const __amdgpu_buffer_rsrc_t x = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(a.X), 0,
                                                                    SRC == FROM_CODES ? a.n * a.kp : 0, 0x00020000);
  const int off = r * a.kp + 16 * g;
  const int8_t* lds = codes + min(r, a.n - 1) * stride + 16 * g;  // tokens past the last repeat it and are not used
  struct Part {
    i32x4 w[UC], x[NT][UC];
  };
  // columns from the u-th UC 64s on; what lies past the last 64 repeats them and is not used
  auto load = [&](Part& p, int u) {
#pragma unroll
    for (int j = 0; j < UC; ++j) {
      const int c = min(UC * u + j, chunks - 1) * 64;
      p.w[j] = load16(w, off + c);
      if (SRC == FROM_CODES) {
#pragma unroll
        for (int t = 0; t < NT; ++t) p.x[t][j] = load16(x, off + c + t * 16 * a.kp);
      }
    }
  };
  i32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = (i32x4){0, 0, 0, 0};
  auto multiply = [&](Part& p, int u) {
#pragma unroll
    for (int j = 0; j < UC; ++j) {
      if (UC * u + j >= chunks) break;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const i32x4 v = SRC == FROM_CODES ? p.x[t][j] : *reinterpret_cast<const i32x4*>(lds + (UC * u + j) * 64);
        acc[t] = __builtin_amdgcn_mfma_i32_16x16x64_i8(p.w[j], v, acc[t], 0, 0, 0);
      }
    }
  };
  const int units = (chunks + UC - 1) / UC;
  Part even, odd;
  if constexpr (SRC != FROM_CODES) {
    // loads come back in their order: the tokens first, whose codes are made while W is on its way
    FewTokens<SRC == FROM_BF16> tokens;
    tokens.load(a);
    __builtin_amdgcn_sched_barrier(0);
    if (wave < units) load(even, wave);
    __builtin_amdgcn_sched_barrier(0);
    tokens.quantize(a, codes, stride, scales, tops);
    __syncthreads();
  } else if (wave < units) {
    load(even, wave);
  }
  for (int u = wave; u < units; u += 2 * NW) {
    const int v = u + NW;
    if (v < units) load(odd, v);
    __builtin_amdgcn_sched_barrier(0);
    multiply(even, u);
    if (v + NW < units) load(even, v + NW);
    __builtin_amdgcn_sched_barrier(0);
    if (v < units) multiply(odd, v);
  }
  // register i of lane 16 g + r: W's row 4 g + i, token r of its group
#pragma unroll
  for (int t = 0; t < NT; ++t) *reinterpret_cast<i32x4*>(&red[wave][16 * t + r][4 * g]) = acc[t];
  __syncthreads();
  for (int e = threadIdx.x; e < 256 * NT; e += 64 * NW) {
    const int tok = e / 16, o = e % 16, c = o0 + o;
    if (tok >= a.n || c >= a.out) continue;
    int sum = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) sum += red[i][tok][o];
    const float y = int8_result((float)sum, SRC == FROM_CODES ? a.xs[tok] : scales[tok], a.ws[c], a.bias ? a.bias[c] : 0.f,
                                a.relu ? 0.f : -__builtin_inff());
    if (YBF16) static_cast<uint16_t*>(a.Y)[tok * a.ldy + c] = (uint16_t)bf16_bits(y);
    else static_cast<float*>(a.Y)[tok * a.ldy + c] = y;
  }
}

template <int SRC, int NT, int NW, int UC>
hipError_t few_go(const FewArgs& a, int y_dtype, hipStream_t stream) {
  const size_t lds = SRC == FROM_CODES ? 0 : (size_t)a.n * (a.kp + 16);
  hipLaunchKernelGGL((y_dtype == GPTQ_BF16 ? k_int8_few<SRC, true, NT, NW, UC> : k_int8_few<SRC, false, NT, NW, UC>),
                     dim3((unsigned)ceil_div(a.out, 16)), dim3(64 * NW), lds, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t int8_matmul_few_launch(const Int8Matrix& x, const Int8Matrix& w, const float* bias, int relu, void* Y, int y_dtype,
                                  int64_t ld_y, hipStream_t stream) {
  const FewArgs a = {x.codes, x.scales, 0, w.codes, w.scales, bias, Y, ld_y, (int)x.rows, (int)w.cols,
                     (int)int8_code_row(w.cols), (int)w.rows, relu};
  if (x.rows <= 16) return few_go<FROM_CODES, 1, 16, 2>(a, y_dtype, stream);
  return few_go<FROM_CODES, 2, 8, 4>(a, y_dtype, stream);
}

hipError_t int8_linear_few_launch(const void* X, int x_dtype, int64_t n, int64_t ld_x, const Int8Matrix& w, const float* bias,
                                  int relu, void* Y, int y_dtype, int64_t ld_y, hipStream_t stream) {
  const FewArgs a = {X, nullptr, ld_x, w.codes, w.scales, bias, Y, ld_y, (int)n, (int)w.cols,
                     (int)int8_code_row(w.cols), (int)w.rows, relu};
  return x_dtype == GPTQ_BF16 ? few_go<FROM_BF16, 1, 8, 8>(a, y_dtype, stream) : few_go<FROM_F32, 1, 8, 8>(a, y_dtype, stream);
}

}  // namespace gptq
