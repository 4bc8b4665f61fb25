// The tile product that the MX operators' large kernels share: a workgroup of four waves forms WA x WB of the sum over
// k of a(i, k) b(j, k), operands streaming from memory straight into a ring of LDS stages while the matrix cores work
// on earlier ones.
//
// What bounds it is LDS: a 32 x 32 product of two fragments reads both of them, 2 KB, for 32 cycles of the matrix
// core (bf16 and 4-bit elements). A wave of 128 x 128 reads 8 fragments for 16 products, 16 B per matrix-core cycle and
// wave, half of what 32 x 32 products one by one would take; with 128 x 64 waves it is 24 B, and LDS becomes the limit.
// That leaves one wave to a SIMD (256 accumulators), so nothing but its own instruction order hides latency:
// a stage holds two steps of k; the fragments of the second are read between the products of the first, the next
// stage's first fragments between those of the second, and the wait for the next stage with its barrier lies in the
// middle, where products are queued on both sides.
//
// Stage layout. Operands whose k runs along a row (E2M1, E4M3, bf16) keep each row's piece of the stage (64 or 128
// bytes) together; the 16-byte chunks of row r are permuted by XOR with bits of the Gray code of r, so that the 16
// consecutive rows that one ds_read_b128 takes at one logical chunk lie on different banks. Operands whose k runs
// down the columns (bf16, "T") keep each k's row together and are read by the transposing ds_read_b64_tr_b16;
// chunks are permuted by bits of k.
#pragma once

#include <utility>

#include "mx.h"

namespace gptq {

enum { K_E2M1 = 0, K_E4M3 = 1, K_BF16 = 2, K_BF16T = 3 };

typedef __attribute__((ext_vector_type(2))) int i32x2;
typedef __attribute__((ext_vector_type(4))) int i32x4;

template <int I, int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<I + 1, N>(f);
  }
}

// buffer_load_dwordx4 ... lds: 64 lanes x 16 B to LDS[addr + lane * 16]; out-of-range reads arrive as zeros. Inline asm,
// so that the compiler adds no waits of its own; no register is written, and the ring orders the transfers with
// explicit vmcnt waits and barriers.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is a reserved register; it is named as clobbered all the same
__device__ __forceinline__ void dma16(const i32x4& rsrc, uint32_t lds_addr, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds_addr), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// every LDS read of this wave has its data and at most N transfers are still in flight; then the workgroup's barrier
template <int N>
__device__ __forceinline__ void wait_and_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// A stretch of memory that advances by `step` bytes from stage to stage; reads past its end, and those of stages past
// the last one, give zeros.
struct Stretch {
  uint64_t addr;
  int64_t left;
  int step, stages;
  i32x4 rsrc;
  // every argument is the same in all lanes
  __device__ __forceinline__ void init(const void* p, int64_t bytes, int st, int n) {
    addr = (uint64_t)(uintptr_t)p;
    addr = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)addr) |
           (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(addr >> 32)) << 32;
    left = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)bytes) |
                     (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)bytes >> 32)) << 32);
    step = __builtin_amdgcn_readfirstlane(st), stages = __builtin_amdgcn_readfirstlane(n);
    set();
  }
  __device__ __forceinline__ void set() {
    const int hi = (int)(left >> 31);  // 0 where 0 <= left < 2^31
    const int n = stages <= 0 || hi < 0 ? 0 : hi > 0 ? 0x7FFFFFF0 : (int)left;
    rsrc = (i32x4){(int)(uint32_t)addr, (int)(uint32_t)(addr >> 32) & 0xFFFF, n, 0x00020000};
  }
  __device__ __forceinline__ void advance() {
    addr += (uint64_t)step, left -= step, --stages;
    set();
  }
};

// XOR pattern of a row's 16-byte chunks: 4 chunks (64-byte rows) or 8 (128-byte rows)
__device__ __forceinline__ int swz4(int r) { return ((r >> 1) ^ (r >> 2)) & 3; }
__device__ __forceinline__ int swz8(int r) { return (r ^ (r >> 1)) & 7; }

// One operand: W rows (columns of a T operand) of the tile, transferred by NW waves.
template <int KIND, int W, int NW>
struct Operand {
  static constexpr int ROW = KIND == K_E4M3 ? 128 : 64;   // bytes of a row in a stage (of 32 k of a T column)
  static constexpr int BYTES = ROW * W;
  static constexpr int NI = BYTES / 1024 / NW;            // transfers per wave and stage
  static constexpr int FRAG = KIND == K_E4M3 ? 8 : 4;     // registers of a fragment
  static constexpr int NB = KIND == K_E4M3 ? 4 : KIND == K_BF16T ? 4 : 2;
  static_assert(NI >= 1 && BYTES % (1024 * NW) == 0, "tile too narrow for its waves");
  static_assert(KIND != K_BF16T || W >= 64, "the T layout's permutation needs 8 chunks");

  // XOR pattern of a k row's chunks in the T layout: the four rows that a transposing read touches (64 bytes each) lie
  // on the four quarters of the banks
  static __device__ __forceinline__ int swzt(int k) { return W >= 128 ? (k & 3) << 2 : (k & 2) << 1; }

  Stretch mem;
  uint32_t voff[NI];   // this lane's offsets from mem.addr
  uint32_t roff[NB];   // this lane's fragment offsets within a stage

  // row_bytes: distance of rows (of k rows for T); cols: columns of a T operand from its first one on
  __device__ __forceinline__ void init(int64_t row_bytes, int wave, int lane, int w0, int64_t cols) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int p = wave * NI + i;
      if (KIND == K_BF16T) {
        const int k = p * (512 / W) + lane / (W / 8);
        const int q = (lane % (W / 8)) ^ swzt(k);
        voff[i] = 8 * q < cols ? (uint32_t)(k * row_bytes + q * 16) : 0x80000000u;
      } else if (KIND == K_E4M3) {
        const int row = p * 8 + (lane >> 3);
        voff[i] = (uint32_t)(row * row_bytes + ((lane & 7) ^ swz8(row)) * 16);
      } else {
        const int row = p * 16 + (lane >> 2);
        voff[i] = (uint32_t)(row * row_bytes + ((lane & 3) ^ swz4(row)) * 16);
      }
    }
    const int r = lane & 31, h = lane >> 5;
    if (KIND == K_BF16T) {
      const int g = lane >> 4, s = lane & 15;
      const int k = 8 * (g >> 1) + (s >> 2);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int c = (b * 32) + 16 * (g & 1) + (s & 3) * 4;
        roff[b] = (uint32_t)(k * (2 * W) + ((((w0 + c) >> 3) ^ swzt(k)) << 4) + (c & 7) * 2);
      }
    } else if (KIND == K_E4M3) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int chunk = 4 * (q >> 1) + 2 * (q & 1) + h;
        roff[q] = (uint32_t)((w0 + r) * 128 + (chunk ^ swz8(r)) * 16);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 2; ++q) roff[q] = (uint32_t)((w0 + r) * 64 + ((2 * q + h) ^ swz4(r)) * 16);
    }
  }

  __device__ __forceinline__ void transfer(int i, uint32_t lds_addr, int wave) const {
    dma16(mem.rsrc, (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds_addr + (wave * NI + i) * 1024)), voff[i]);
  }

  // fragment of 32 rows (block b of the wave's) at step J of the stage
  template <int J, int B>
  __device__ __forceinline__ void read(const uint8_t* stage, int (&f)[FRAG]) const {
    if constexpr (KIND == K_BF16T) {
      const uint8_t* p = stage + roff[B] + J * 32 * W;
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)p);
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p + 8 * W));
      const i32x2 l = __builtin_bit_cast(i32x2, lo), u = __builtin_bit_cast(i32x2, hi);
      f[0] = l[0], f[1] = l[1], f[2] = u[0], f[3] = u[1];
    } else {
#pragma unroll
      for (int q = 0; q < FRAG / 4; ++q) {
        const i32x4 v = *reinterpret_cast<const i32x4*>(stage + roff[J * (FRAG / 4) + q] + B * 32 * ROW);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[4 * q + i] = v[i];
      }
    }
  }
};

// Parts of an E4M3 fragment whose exponents differ by at most 7: codes with the top exponent bit set, and the rest.
// The matrix core aligns the products of one instruction to their largest and drops what lies more than about 13
// bits below; with half of the exponents to each part nothing is dropped against E2M1 weights, so the sum is exact
// up to fp32 rounding.
__device__ __forceinline__ void split_e4m3(const i32x8& a, i32x8& hi, i32x8& lo) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint32_t t = (uint32_t)a[q] & 0x40404040u;
    const uint32_t m = (t << 1) - (t >> 6);  // 0x7F in every byte whose top exponent bit is set
    hi[q] = (int)((uint32_t)a[q] & (m | 0x80808080u));
    lo[q] = (int)((uint32_t)a[q] & ~m);
  }
}

template <int KIND, int N>
__device__ __forceinline__ i32x8 as_operand(const int (&f)[N]) {
  i32x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = f[i];
  return v;
}

// A (first operand) x B (second): KA is K_E2M1 with KB K_E2M1 or K_E4M3, or both are bf16 kinds.
// SPLIT: E4M3 fragments in two parts (see split_e4m3).
template <int KA, int KB, int WA, int WB, int MB, int NB, int NSTG, bool SPLIT>
struct TileProduct {
  static constexpr int NW = 4;
  static constexpr bool MX = KA == K_E2M1;
  static constexpr int WAVES_A = WA / (32 * MB), WAVES_B = WB / (32 * NB);
  static_assert(WAVES_A * WAVES_B == NW && NSTG >= 3, "four waves, three stages at least");
  static_assert(!MX || NSTG <= 4, "a scale buffer is refilled NSTG - 1 stages ahead and read four stages long");
  using A = Operand<KA, WA, NW>;
  using B = Operand<KB, WB, NW>;
  static constexpr int STAGE = A::BYTES + B::BYTES;
  static constexpr int SCALES = MX ? (WA + WB) * 16 : 0;         // 512 columns' scale bytes
  static constexpr int STORE = NW * 32 * (32 * MB + 4) * 4;      // what store_rows needs
  static constexpr int LDS = NSTG * STAGE + SCALES > STORE ? NSTG * STAGE + SCALES : STORE;
  static constexpr int SI = MX ? (WA + WB) / 64 : 0;             // scale transfers per 512 columns
  static constexpr int SC = (SI + NW - 1) / NW;                  // per wave (the last ones may repeat the first)
  static constexpr int PER = A::NI + B::NI;
  static constexpr int NM = MB * NB;
  static_assert(!MX || (WA % 64 == 0 && WB % 64 == 0), "scale transfers take 64 rows");

  A a;
  B b;
  Stretch sa, sb;
  int64_t srow;      // bytes of a scale row
  uint8_t* lds;
  uint32_t base;     // LDS address of lds
  int wave, lane, wa, wb;
  uint32_t slot_w, slot_r;
  f32x16 acc[MB][NB];
  int fa[2][MB][A::FRAG], fb[2][NB][B::FRAG];
  int sca[MB][4], scb[NB][4], nca[MB][4], ncb[NB][4];

  __device__ __forceinline__ void init(uint8_t* l) {
    lds = l, base = (uint32_t)(uintptr_t)l;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    wa = (wave / WAVES_B) * (32 * MB), wb = (wave % WAVES_B) * (32 * NB);
    slot_w = slot_r = 0;
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  }

  static __device__ __forceinline__ uint32_t next_slot(uint32_t s) { return s + STAGE == NSTG * STAGE ? 0u : s + STAGE; }

  __device__ __forceinline__ void transfer_scales() {
#pragma unroll
    for (int i = 0; i < SC; ++i) {
      const int t = (wave + NW * i) % (SI ? SI : 1);
      const bool second = t >= WA / 64;
      const uint32_t v = (uint32_t)((64 * (second ? t - WA / 64 : t) + lane) * srow);
      dma16(second ? sb.rsrc : sa.rsrc, (uint32_t)__builtin_amdgcn_readfirstlane((int)(base + NSTG * STAGE + t * 1024)), v);
    }
    sa.advance(), sb.advance();
  }

  // the i-th of a stage's PER transfers
  __device__ __forceinline__ void transfer(int i) {
    if (i < A::NI) a.transfer(i, base + slot_w, wave);
    else b.transfer(i - A::NI, base + slot_w + A::BYTES, wave);
    if (i == PER - 1) {
      a.mem.advance(), b.mem.advance();
      slot_w = next_slot(slot_w);
    }
  }

  // the t-th of the MB + NB fragments of step J of the stage at slot_r into set SET
  template <int SET, int J, int T>
  __device__ __forceinline__ void read_frag() {
    if constexpr (T < MB) a.template read<J, T>(lds + slot_r, fa[SET][T]);
    else b.template read<J, T - MB>(lds + slot_r + A::BYTES, fb[SET][T - MB]);
  }

  template <int T>
  __device__ __forceinline__ void read_scale() {
    const int row = (T < MB ? wa + 32 * T : WA + wb + 32 * (T - MB)) + (lane & 31);
    const i32x4 v = *reinterpret_cast<const i32x4*>(lds + NSTG * STAGE + row * 16);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (T < MB) nca[T][q] = v[q];
      else ncb[T - MB][q] = v[q];
    }
  }

  template <int SET, int Q, int J, int M, int N>
  __device__ __forceinline__ void product() {
    if constexpr (!MX) {
      acc[M][N] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          __builtin_bit_cast(bf16x8, (i32x4){fa[SET][M][0], fa[SET][M][1], fa[SET][M][2], fa[SET][M][3]}),
          __builtin_bit_cast(bf16x8, (i32x4){fb[SET][N][0], fb[SET][N][1], fb[SET][N][2], fb[SET][N][3]}), acc[M][N],
          0, 0, 0);
    } else {
      const i32x8 x = as_operand<KA>(fa[SET][M]), y = as_operand<KB>(fb[SET][N]);
      constexpr int FB = KB == K_E2M1 ? 4 : 0;
      if constexpr (SPLIT) {
        i32x8 hi, lo;
        split_e4m3(y, hi, lo);
        acc[M][N] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, lo, acc[M][N], 4, FB, 2 * J, sca[M][Q], 2 * J,
                                                                    scb[N][Q]);
        acc[M][N] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, hi, acc[M][N], 4, FB, 2 * J, sca[M][Q], 2 * J,
                                                                    scb[N][Q]);
      } else {
        acc[M][N] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc[M][N], 4, FB, 2 * J, sca[M][Q], 2 * J,
                                                                    scb[N][Q]);
      }
    }
  }

  // transfers in flight that may remain when stage Q (mod 4) + 1 is needed: those of the NSTG - 2 stages after it
  static constexpr int pending(int q) {
    int n = 0;
    for (int s = 2; s < NSTG; ++s) n += PER + ((MX && (q + s) % 4 == 0) ? SC : 0);
    return n;
  }

  template <int Q>
  __device__ __forceinline__ void stage() {
    if constexpr (MX && Q == 0) {
      const int sh = 8 * (lane >> 5);  // lanes 32..63 take the odd blocks' bytes
#pragma unroll
      for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int m = 0; m < MB; ++m) sca[m][q] = (int)((uint32_t)nca[m][q] >> sh);
#pragma unroll
        for (int n = 0; n < NB; ++n) scb[n][q] = (int)((uint32_t)ncb[n][q] >> sh);
      }
    }
    if constexpr (MX && (Q + NSTG - 1) % 4 == 0) transfer_scales();
    // first step; between its products the second step's fragments and the transfers of the stage NSTG - 1 ahead
    static_for<0, NM>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      product<0, Q, 0, i / NB, i % NB>();
      static_for<i * (MB + NB) / NM, (i + 1) * (MB + NB) / NM>([&](auto t) { read_frag<1, 1, decltype(t)::value>(); });
      static_for<i * PER / NM, (i + 1) * PER / NM>([&](auto t) { transfer(decltype(t)::value); });
      __builtin_amdgcn_sched_barrier(0);
    });
    wait_and_barrier<pending(Q)>();
    slot_r = next_slot(slot_r);
    static_for<0, NM>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      product<1, Q, 1, i / NB, i % NB>();
      static_for<i * (MB + NB) / NM, (i + 1) * (MB + NB) / NM>([&](auto t) {
        read_frag<0, 0, decltype(t)::value>();
        if constexpr (MX && Q == 3) read_scale<decltype(t)::value>();
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  }

  // nk stages; MX operands take them four at a time (512 columns), those past the last one multiplying zeros (the
  // stretches end there, and the format keeps the scale bytes behind a row's last block at 0)
  __device__ __forceinline__ void run(int nk) {
    static_for<0, NSTG - 1>([&](auto s) {
      if constexpr (MX && decltype(s)::value % 4 == 0) transfer_scales();
#pragma unroll
      for (int i = 0; i < PER; ++i) transfer(i);
    });
    wait_and_barrier<pending(3)>();
    static_for<0, MB + NB>([&](auto t) {
      read_frag<0, 0, decltype(t)::value>();
      if constexpr (MX) read_scale<decltype(t)::value>();
    });
    if constexpr (MX) {
      for (int kt = 0; kt < nk; kt += 4) stage<0>(), stage<1>(), stage<2>(), stage<3>();
    } else {
      for (int kt = 0; kt < nk; ++kt) stage<0>();
    }
    wait_and_barrier<0>();  // nothing may still be writing LDS when the workgroup moves on
  }
};

// Tile of workgroup b of `grid` (a multiple of 8, at least `tiles`), false for the grid's surplus. Workgroup b runs on
// XCD b mod 8: each XCD owns a run of tiles, ordered in strips of up to 8 tiles of the second operand, so that the tiles
// that run together on an XCD share operands in its L2.
__device__ __forceinline__ bool tile_of(int b, int grid, int ta, int tb, int& ia, int& ib) {
  const int p = (b & 7) * (grid >> 3) + (b >> 3);
  if (p >= ta * tb) return false;
  const int strip = p / (8 * ta), rest = p - strip * 8 * ta;
  const int h = min(8, tb - strip * 8);
  ia = rest / h, ib = strip * 8 + rest % h;
  return true;
}

static inline unsigned tile_grid(int64_t tiles) { return (unsigned)((tiles + 7) / 8 * 8); }

// Writes a wave's results, 32 NB rows of Y (from row0 on, of `rows`) by 32 MB columns (from c0 on, of `cols`), through LDS,
// so that a store takes whole runs of a row: register i of lane l of acc[mb][nb] is row 32 nb + l % 32, column
// 32 mb + 8 (i / 4) + 4 (l / 32) + i % 4. finish(row, c, v) completes V consecutive results. vec: Y's rows are 16-byte
// aligned. lds: the workgroup's ring, no longer in use; each wave takes a part of its own.
template <bool YBF16, int MB, int NB, typename F>
__device__ __forceinline__ void store_rows(const f32x16 (&acc)[MB][NB], uint8_t* lds, void* __restrict__ Y, int64_t ld,
                                           int64_t row0, int64_t rows, int c0, int cols, bool vec, bool add,
                                           F&& finish) {
  constexpr int C = 32 * MB, PITCH = C + 4, V = YBF16 ? 8 : 4, PER_ROW = C / V, STEP = 64 / PER_ROW;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* buf = reinterpret_cast<float*>(lds) + wave * (32 * PITCH);
  const int r = lane & 31, h = lane >> 5;
  const int c = c0 + (lane % PER_ROW) * V;
  const bool whole = vec && c + V <= cols;
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<float4*>(buf + r * PITCH + mb * 32 + 8 * g + 4 * h) =
            make_float4(acc[mb][nb][4 * g], acc[mb][nb][4 * g + 1], acc[mb][nb][4 * g + 2], acc[mb][nb][4 * g + 3]);
    __builtin_amdgcn_wave_barrier();
#pragma unroll 2
    for (int i = lane / PER_ROW; i < 32; i += STEP) {
      const int64_t row = row0 + nb * 32 + i;
      if (row >= rows || c >= cols) continue;
      float v[V];
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const float4 x = *reinterpret_cast<const float4*>(buf + i * PITCH + c - c0 + 4 * q);
        v[4 * q] = x.x, v[4 * q + 1] = x.y, v[4 * q + 2] = x.z, v[4 * q + 3] = x.w;
      }
      finish(row, c, v);
      if (YBF16) {
        uint16_t* p = static_cast<uint16_t*>(Y) + row * ld + c;
        if (whole) {
          *reinterpret_cast<uint4*>(p) = make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]),
                                                    bf16_pair(v[V - 4], v[V - 3]), bf16_pair(v[V - 2], v[V - 1]));
        } else {
          for (int q = 0; q < V; ++q)
            if (c + q < cols) p[q] = (uint16_t)bf16_bits(v[q]);
        }
      } else {
        float* p = static_cast<float*>(Y) + row * ld + c;
        if (whole) {
          float4* p4 = reinterpret_cast<float4*>(p);
          const float4 o = add ? *p4 : make_float4(0.f, 0.f, 0.f, 0.f);
          *p4 = add ? make_float4(o.x + v[0], o.y + v[1], o.z + v[2], o.w + v[3]) : make_float4(v[0], v[1], v[2], v[3]);
        } else {
          for (int q = 0; q < V; ++q)
            if (c + q < cols) p[q] = add ? p[q] + v[q] : v[q];
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace gptq
