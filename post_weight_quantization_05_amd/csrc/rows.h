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

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
  return v;
}
template <typename T>
__device__ __forceinline__ T wave_sum(T v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
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
