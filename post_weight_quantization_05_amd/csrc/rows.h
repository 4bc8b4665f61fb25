// Kernels that work on whole rows held in registers: a row is shared by `waves` waves of a workgroup, a lane holding
// `chunks` pieces of 8 consecutive columns; a workgroup takes `rows` rows at a time.
#pragma once

#include <algorithm>

#include "common.h"

namespace gptq {

struct RowShape {
  int waves, chunks, rows;
  unsigned threads() const { return (unsigned)(64 * waves * rows); }
};

// segments: 512-column pieces of a row, at most 128
static inline RowShape row_shape(int64_t segments, int64_t n) {
  RowShape s = {(int)segments, 1, 1};
  while (s.waves > 8 && s.chunks < 8) s.chunks *= 2, s.waves = (int)ceil_div(segments, s.chunks);
  if (s.waves == 1 && n > 1) s.rows = 4;
  return s;
}

// workgroups of a launch: up to four times what fits the chip at once
static inline unsigned row_grid(const RowShape& s, int64_t n) {
  return (unsigned)std::min<int64_t>(ceil_div(n, s.rows), (int64_t)4 * 256 * (2048 / s.threads()));
}

// GO(chunks) for the number of chunks a lane holds
#define GPTQ_ROW_CHUNKS(chunks, GO) \
  if ((chunks) == 1) {              \
    GO(1);                          \
  } else if ((chunks) == 2) {       \
    GO(2);                          \
  } else if ((chunks) == 4) {       \
    GO(4);                          \
  } else {                          \
    GO(8);                          \
  }

struct RowShared {
  uint32_t top[2][16];
  double sum[2][16];
};

// Reductions over a wave's 64 lanes on the vector unit alone: neighbours, quads, eights, sixteens by DPP, then the halves
// of 32 and of 64 lanes exchanged.
template <typename F>
__device__ __forceinline__ uint32_t wave_join(uint32_t v, F&& f) {
  v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));   // lanes 1 0 3 2
  v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));   // lanes 2 3 0 1
  v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));  // eight lanes reversed
  v = f(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));  // sixteen lanes reversed
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = f(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return f(b[0], b[1]);
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  return wave_join(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(wave_join(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
__device__ __forceinline__ double wave_sum(double v) {
  auto moved = [](double x, auto move) {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    return __builtin_bit_cast(double, (uint64_t)move((uint32_t)u) | (uint64_t)move((uint32_t)(u >> 32)) << 32);
  };
  v += moved(v, [](uint32_t x) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, true); });
  v += moved(v, [](uint32_t x) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, true); });
  v += moved(v, [](uint32_t x) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x141, 0xF, 0xF, true); });
  v += moved(v, [](uint32_t x) { return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x140, 0xF, 0xF, true); });
  const double a = moved(v, [](uint32_t x) { return __builtin_amdgcn_permlane16_swap(x, x, false, false)[0]; });
  const double b = moved(v, [](uint32_t x) { return __builtin_amdgcn_permlane16_swap(x, x, false, false)[1]; });
  v = a + b;
  const double c = moved(v, [](uint32_t x) { return __builtin_amdgcn_permlane32_swap(x, x, false, false)[0]; });
  const double d = moved(v, [](uint32_t x) { return __builtin_amdgcn_permlane32_swap(x, x, false, false)[1]; });
  return c + d;
}

struct RowGroup {
  int waves, slot, lane_of_row, wave, turn;
  __device__ __forceinline__ void init(const RowShape& s) {
    waves = s.waves;
    wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    slot = wave / waves;
    lane_of_row = (int)threadIdx.x - slot * waves * 64;
    turn = 0;
  }
  // first column of this lane's i-th chunk
  __device__ __forceinline__ int column(int i) const { return (i * waves * 64 + lane_of_row) * 8; }

  // The waves' parts meet in LDS, in two buffers in turn: a wave that is one row ahead writes the other one, and no wave can
  // be two ahead, since all pass the barrier between.
  __device__ __forceinline__ uint32_t max_of_row(uint32_t v, RowShared& sh) {
    v = wave_max(v);
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) sh.top[turn][wave] = v;
    __syncthreads();
    for (int i = 0; i < waves; ++i) v = max(v, sh.top[turn][slot * waves + i]);
    turn ^= 1;
    return v;
  }
  template <typename T>
  __device__ __forceinline__ T sum_of_row(T v, RowShared& sh) {
    v = wave_sum(v);
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) sh.sum[turn][wave] = (double)v;
    __syncthreads();
    T total = 0;
    for (int i = 0; i < waves; ++i) total += (T)sh.sum[turn][slot * waves + i];
    turn ^= 1;
    return total;
  }
  __device__ __forceinline__ void both_of_row(double& sum, uint32_t& top, RowShared& sh) {
    sum = wave_sum(sum), top = wave_max(top);
    if (waves == 1) return;
    if ((threadIdx.x & 63) == 0) sh.sum[turn][wave] = sum, sh.top[turn][wave] = top;
    __syncthreads();
    sum = 0.0;
    for (int i = 0; i < waves; ++i) sum += sh.sum[turn][slot * waves + i], top = max(top, sh.top[turn][slot * waves + i]);
    turn ^= 1;
  }
};

}  // namespace gptq
