// Kernels that work on whole rows held in registers. A lane holds `chunks` pieces of 8 consecutive columns; a row is shared by
// `waves` waves of a workgroup or, if it is short, by a part of a wave (`lanes`); a workgroup takes `rows` rows at a time.
#pragma once

#include <algorithm>

#include "common.h"

namespace gptq {

struct RowShape {
  int waves, chunks, lanes, rows;
  unsigned threads() const { return lanes < 64 ? (unsigned)ceil_div(rows * lanes, 64) * 64 : (unsigned)(64 * waves * rows); }
};

// For rows of d columns (at most 65536). Only a lane's last chunk may reach past the row's end. Two chunks a lane from 2049
// columns on (norm of 16384 x 4096 without a residual: 39 us, with one 50), three from 8193 on (8192 x 11008: 65 us, with eight
// in fewer waves 78). Half and quarter waves for short rows, since what is done once a row and wave is most of their work
// (norm of 16384 x 256: 9.4 us, with whole waves 15). waves: those of a workgroup where rows are short enough for several; few
// rows are spread over the chip's CUs first.
static inline RowShape row_shape(int64_t d, int64_t n, int waves) {
  const int64_t segments = ceil_div(d, 512);
  const int chunks = segments <= 4 ? 1 : segments <= 16 ? 2 : segments <= 24 ? 3 : segments <= 64 ? 4 : 8;
  RowShape s = {(int)ceil_div(segments, chunks), chunks, d <= 128 ? 16 : d <= 256 ? 32 : 64, 1};
  const int64_t most = std::max(1, waves / s.waves) * (64 / s.lanes);
  s.rows = (int)std::max<int64_t>(64 / s.lanes, std::min<int64_t>(most, n / 256));
  return s;
}

// GO(chunks, lanes) for a shape's
#define GPTQ_ROW_SHAPE(s, GO)                  \
  switch ((s).chunks) {                        \
    case 1:                                    \
      if ((s).lanes == 16) { GO(1, 16); }      \
      else if ((s).lanes == 32) { GO(1, 32); } \
      else { GO(1, 64); }                      \
      break;                                   \
    case 2: GO(2, 64); break;                  \
    case 3: GO(3, 64); break;                  \
    case 4: GO(4, 64); break;                  \
    default: GO(8, 64);                        \
  }

// Reductions over LANES lanes on the vector unit alone: neighbours, quads, eights, sixteens by DPP, then the halves of 32 and
// of 64 lanes exchanged.
template <int LANES, typename F>
__device__ __forceinline__ uint32_t lanes_join(uint32_t v, F&& f) {
  v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));   // lanes 1 0 3 2
  v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));   // lanes 2 3 0 1
  v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));  // eight lanes reversed
  v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));  // sixteen lanes reversed
  if (LANES > 16) {
    const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = f(a[0], a[1]);
  }
  if (LANES > 32) {
    const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = f(b[0], b[1]);
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  return lanes_join<LANES>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  return __uint_as_float(lanes_join<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int LANES>
__device__ __forceinline__ double lanes_sum(double v) {
  auto moved = [](double x, auto move) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (uint64_t)move((uint32_t)u) | (uint64_t)move((uint32_t)(u >> 32)) << 32);
  };
  v += moved(v, [](uint32_t x) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true); });
  v += moved(v, [](uint32_t x) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true); });
  v += moved(v, [](uint32_t x) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x141, 0xF, 0xF, true); });
  v += moved(v, [](uint32_t x) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x140, 0xF, 0xF, true); });
  if (LANES > 16) {
    const double a = moved(v, [](uint32_t x) { return __builtin_amdgcn_permlane16_swap(x, x, false, false)[0]; });
    const double b = moved(v, [](uint32_t x) { return __builtin_amdgcn_permlane16_swap(x, x, false, false)[1]; });
    v = a + b;
  }
  if (LANES > 32) {
    const double a = moved(v, [](uint32_t x) { return __builtin_amdgcn_permlane32_swap(x, x, false, false)[0]; });
    const double b = moved(v, [](uint32_t x) { return __builtin_amdgcn_permlane32_swap(x, x, false, false)[1]; });
    v = a + b;
  }
  return v;
}

struct RowShared {
  uint32_t top[2][16];
  double sum[2][16];
};

template <int LANES>
struct RowGroup {
  int waves, slot, lane, wave, turn;  // lane: of the row's
  __device__ __forceinline__ void init(const RowShape& s) {
    waves = s.waves;
    wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    slot = LANES < 64 ? (int)threadIdx.x / LANES : wave / waves;
    lane = LANES < 64 ? (int)threadIdx.x % LANES : (int)threadIdx.x - slot * waves * 64;
    turn = 0;
  }
  // first column of this lane's i-th chunk
  __device__ __forceinline__ int column(int i) const { return LANES < 64 ? lane * 8 : (i * waves * 64 + lane) * 8; }

  // The waves' parts meet in LDS, in two buffers in turn: a wave that is one row ahead writes the other one, and no wave can
  // be two ahead, since all pass the barrier between.
  __device__ __forceinline__ uint32_t max_of_row(uint32_t v, RowShared& sh) {
    v = lanes_max<LANES>(v);
    if (LANES < 64 || waves == 1) return v;
    if ((threadIdx.x & 63) == 0) sh.top[turn][wave] = v;
    __syncthreads();
    for (int i = 0; i < waves; ++i) v = max(v, sh.top[turn][slot * waves + i]);
    turn ^= 1;
    return v;
  }
  __device__ __forceinline__ float sum_of_row(float v, RowShared& sh) {
    v = lanes_sum<LANES>(v);
    if (LANES < 64 || waves == 1) return v;
    if ((threadIdx.x & 63) == 0) sh.top[turn][wave] = __float_as_uint(v);
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < waves; ++i) v += __uint_as_float(sh.top[turn][slot * waves + i]);
    turn ^= 1;
    return v;
  }
  __device__ __forceinline__ void both_of_row(double& sum, uint32_t& top, RowShared& sh) {
    sum = lanes_sum<LANES>(sum), top = lanes_max<LANES>(top);
    if (LANES < 64 || waves == 1) return;
    if ((threadIdx.x & 63) == 0) sh.sum[turn][wave] = sum, sh.top[turn][wave] = top;
    __syncthreads();
    sum = 0.0;
    for (int i = 0; i < waves; ++i) sum += sh.sum[turn][slot * waves + i], top = max(top, sh.top[turn][slot * waves + i]);
    turn ^= 1;
  }
};

}  // namespace gptq
