// The tile product that the MX operators' large kernels share: a workgroup of four waves forms WA x WB of the sum over
// k of a(i, k) b(j, k), operands streaming from memory straight into a ring of LDS stages while the matrix cores work
// on earlier ones.
//
// What bounds it: LDS and the L2. A 32 x 32 product of two fragments reads both of them, 2 KB, for 32 cycles of the
// matrix core (bf16 and 4-bit elements). A wave of 128 x 128 reads 8 fragments for 16 products, 16 B per matrix-core
// cycle and wave, half of what 32 x 32 products one by one would take. That leaves one wave to a SIMD (256 accumulators),
// so nothing but its own instruction order hides latency. The L2 hands out lines of 128 bytes whatever part is asked
// for: a stage therefore takes whole lines, 128 bytes of each row (64 bytes of each row, twice, cost 2.5 times the
// lines of the 4-bit product at 16384 x 4096 x 11008 with its scales, 16 TB/s, which was the limit).
//
// A stage holds four steps of k (64 columns each for MX, 16 for bf16), two stages make the ring. The fragments of a step
// are read between the products of the step before. Before the last step of a stage its buffer has been read by all
// waves and the next stage has arrived (one wait, one barrier); between its products go the first fragments of the next
// stage and the transfers of the stage after that, which have until the next such point to land.
//
// Stage layout. Operands whose k runs along a row (E2M1, E4M3, bf16) keep 128 bytes of each row together (E4M3: two such
// planes); the 16-byte chunks of row r are permuted by XOR with the Gray code of r, so that the consecutive rows that
// one ds_read_b128 takes at one logical chunk lie on different banks. Operands whose k runs down the columns (bf16, "T")
// keep each k's row together and are read by the transposing ds_read_b64_tr_b16; chunks are permuted by bits of k.
#pragma once

#include <utility>

#include "mx.h"

namespace gptq {

enum { K_E2M1 = 0, K_E4M3 = 1, K_BF16 = 2, K_BF16T = 3 };


template <int I, int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    static_for<I + 1, N>(f);
  }
}

// buffer_load_dwordx4 ... lds: 64 lanes x 16 B to LDS[addr + lane * 16]; out-of-range reads arrive as zeros. Inline asm,
// so that the compiler adds no waits of its own; no register is written, and the ring orders the transfers with
// explicit vmcnt waits and barriers. The compiler does not look into the asm for the waits that the hardware leaves to
// software. A load to LDS needs one state after the write of M0: the s_nop (without it a load may take the M0 of the
// transfer before, and its kilobyte lands there). It also needs five after a vector instruction that wrote one of its
// scalar registers, as a spilled one's return does: none comes that close in what is built, which
// tests/test_isa_host.py checks (s_nop 4 would cover it here, but costs dX 8192 x 11008 x 4096 638 us instead of 619).
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // m0 is a reserved register; it is named as clobbered all the same
__device__ __forceinline__ void dma16(const i32x4& rsrc, uint32_t lds_addr, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds_addr), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
// the same where `skip` is 0; a branch of the compiler's would let it move products across the ring's barriers
__device__ __forceinline__ void dma16_unless(int skip, const i32x4& rsrc, uint32_t lds_addr, uint32_t voff) {
  asm volatile("s_cmp_lg_u32 %3, 0\n\ts_cbranch_scc1 .Lno_transfer%=\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\t"
               "buffer_load_dwordx4 %1, %2, 0 offen lds\n.Lno_transfer%=:"
               :
               : "s"(lds_addr), "v"(voff), "s"(rsrc), "s"(skip)
               : "memory", "m0", "scc");
}
#pragma clang diagnostic pop

// every LDS read of this wave has its data and at most N transfers are still in flight; then the workgroup's barrier
template <int N>
__device__ __forceinline__ void wait_and_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v) |
                   (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)((uint64_t)v >> 32)) << 32);
}

// A stretch of memory that advances by `step` bytes from stage to stage; reads past its end, and those of stages past
// the last one, give zeros. All members are the same in all lanes.
struct Stretch {
  uint64_t addr;
  int64_t left;
  int step, stages;
  __device__ __forceinline__ void init(const void* p, int64_t bytes, int st, int n) {
    addr = (uint64_t)uniform64((int64_t)(uintptr_t)p), left = uniform64(bytes);
    step = __builtin_amdgcn_readfirstlane(st), stages = __builtin_amdgcn_readfirstlane(n);
  }
  __device__ __forceinline__ i32x4 rsrc() const {
    const int hi = (int)(left >> 31);  // 0 where 0 <= left < 2^31
    const int n = stages <= 0 || hi < 0 ? 0 : hi > 0 ? 0x7FFFFFF0 : (int)left;
    return (i32x4){(int)(uint32_t)addr, (int)(uint32_t)(addr >> 32) & 0xFFFF, n, 0x00020000};
  }
  __device__ __forceinline__ void advance() { addr += (uint64_t)step, left -= step, --stages; }
  __device__ __forceinline__ void take_if(bool c, const Stretch& s) {
    addr = c ? s.addr : addr, left = c ? s.left : left, stages = c ? s.stages : stages;
  }
  __device__ __forceinline__ Stretch at(int steps) const {
    Stretch s = *this;
    s.addr += (uint64_t)steps * (uint32_t)step, s.left -= (int64_t)steps * step;
    return s;
  }
};

// XOR patterns of a row's 16-byte chunks: 2 chunks (32-byte rows) or 8 (128-byte rows)
__device__ __forceinline__ int swz2(int r) { return (r >> 3) & 1; }
__device__ __forceinline__ int swz8(int r) { return (r ^ (r >> 1)) & 7; }

// One operand: W rows (columns of a T operand) of the tile, transferred by NW waves.
template <int KIND, int W, int NW>
struct Operand {
  static constexpr int PLANES = KIND == K_E4M3 ? 2 : 1;
  static constexpr int BYTES = 128 * PLANES * W;
  static constexpr int NI = BYTES / 1024 / NW;            // transfers per wave and stage
  static constexpr int FRAG = KIND == K_E4M3 ? 8 : 4;     // registers of a fragment
  static constexpr int STEP = 128 * PLANES;               // bytes along a row per stage (not T)
  static_assert(BYTES % (1024 * NW * PLANES) == 0, "tile too narrow for its waves");
  static_assert(KIND != K_BF16T || W >= 64, "the T layout's permutation needs 8 chunks");

  // XOR pattern of a k row's chunks in the T layout: the four rows that a transposing read touches (64 bytes each) lie
  // on the four quarters of the banks
  static __device__ __forceinline__ int swzt(int k) { return W >= 128 ? (k & 3) << 2 : (k & 2) << 1; }

  Stretch mem;
  i32x4 rsrc;          // of the stage whose transfers are being issued
  uint32_t beyond;     // E4M3: set where that stage's second plane lies behind the row's end
  uint32_t voff[NI];   // this lane's offsets from mem.addr
  uint32_t roff[4];    // this lane's fragment offsets within a stage

  // row_bytes: distance of rows (of k rows for T)
  __device__ __forceinline__ void init(int64_t row_bytes, int wave, int lane, int w0) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int p = wave * (NI / PLANES) + i % (NI / PLANES);
      if (KIND == K_BF16T) {
        const int k = p * (512 / W) + lane / (W / 8);
        const int q = (lane % (W / 8)) ^ swzt(k);
        voff[i] = (uint32_t)(k * row_bytes + q * 16);
      } else {
        const int row = p * 8 + (lane >> 3);
        voff[i] = (uint32_t)(row * row_bytes + ((lane & 7) ^ swz8(row)) * 16 + i / (NI / PLANES) * 128);
      }
    }
    const int r = lane & 31, h = lane >> 5;
    const int g = lane >> 4, s = lane & 15, k = 8 * (g >> 1) + (s >> 2);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (KIND == K_BF16T) {  // block q of 32 columns
        const int c = w0 + q * 32 + 16 * (g & 1) + (s & 3) * 4;
        roff[q] = (uint32_t)(k * (2 * W) + (((c >> 3) ^ swzt(k)) << 4) + (c & 7) * 2);
      } else {                // E4M3: step q / 2 of a plane, half q % 2 of the fragment; else step q
        const int chunk = KIND == K_E4M3 ? 4 * (q >> 1) + 2 * (q & 1) + h : 2 * q + h;
        roff[q] = (uint32_t)((w0 + r) * 128 + (chunk ^ swz8(r)) * 16);
      }
    }
  }

  // the next transfers are those of the stage at mem; tail: the last stage's second plane lies behind the row's end
  __device__ __forceinline__ void open(int tail) {
    rsrc = mem.rsrc();
    beyond = mem.stages == 1 && tail ? 0x80000000u : 0u;
  }

  // the i-th transfer of the stage
  __device__ __forceinline__ void transfer(int i, uint32_t lds_addr, int wave) const {
    constexpr int PER_PLANE = NI / PLANES;
    const uint32_t v = KIND == K_E4M3 && i >= PER_PLANE ? voff[i] | beyond : voff[i];
    const int at_lds = (i / PER_PLANE) * (W * 128) + (wave * PER_PLANE + i % PER_PLANE) * 1024;
    dma16(rsrc, (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds_addr + at_lds)), v);
  }

  // fragment of 32 rows (block B of the wave's) at step J of the stage
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
        const int at = KIND == K_E4M3 ? (J >> 1) * (W * 128) : 0;
        const i32x4 v = *reinterpret_cast<const i32x4*>(stage + roff[KIND == K_E4M3 ? (J & 1) * 2 + q : J] + at + B * 4096);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[4 * q + i] = v[i];
      }
    }
  }
};

template <int KIND, int N>
__device__ __forceinline__ i32x8 as_operand(const int (&f)[N]) {
  i32x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = f[i];
  return v;
}

// A (first operand) x B (second): KA is K_E2M1 with KB K_E2M1 or K_E4M3, or both are bf16 kinds.
// E4M3 fragments are multiplied in two parts (see split_e4m3).
template <int KA, int KB, int WA, int WB, int MB, int NB>
struct TileProduct {
  static constexpr int NW = 4;
  static constexpr bool MX = KA == K_E2M1;
  static constexpr int WAVES_A = WA / (32 * MB), WAVES_B = WB / (32 * NB);
  static_assert(WAVES_A * WAVES_B == NW, "four waves");
  using A = Operand<KA, WA, NW>;
  using B = Operand<KB, WB, NW>;
  static constexpr int STAGE = A::BYTES + B::BYTES;
  // Scale bytes are held for 1024 columns (32 bytes of each row), refilled when the last 512 of them are in registers.
  static constexpr int SCALES = MX ? (WA + WB) * 32 : 0;
  // The large tiles' workgroups stay for several tiles, and a tile's results leave through memory of their own while the
  // ring fills with the next one's first stages; the small ones', of which several share a CU, through the ring's.
  static constexpr bool STAYS = MB == 4;
  static constexpr int PB = STAYS && !MX ? 2 : 1;
  static constexpr int LDS = 2 * STAGE + SCALES + (STAYS ? NW * 4096 * PB : 0);
  static constexpr int SI = MX ? ((WA + WB) / 32 + NW - 1) / NW : 0;  // scale transfers per wave (some twice)
  static constexpr int PER = A::NI + B::NI;
  static constexpr int NM = MB * NB;
  // Share of a stage's transfers issued by the end of the last step of the stage two before it, then of the next one's first
  // and second. All of them between the last step's products saturate the L1's 64 bytes a cycle while the matrix cores
  // wait (16384 x 4096 x 11008 in 4 bits: 478 us, against 444); spread over all four steps the last ones arrive late (455).
  static constexpr int D3 = PER * 8 / 16, D0 = PER * 12 / 16, D1 = PER;
  static_assert(!MX || (WA % 64 == 0 && WB % 64 == 0), "scale transfers");

  A a;
  B b;
  Stretch sa, sb;              // scale bytes of the tile
  Stretch an, bn, san, sbn;    // the next tile's operands and scale bytes
  int tail;                    // E4M3: the row's last stage ends after its first plane
  uint8_t* lds;
  uint32_t base;     // LDS address of lds
  int wave, lane, wa, wb;
  uint32_t slot;     // offset of the stage being multiplied
  uint32_t svoff[SI ? SI : 1], soff;
  int stile[SI ? SI : 1];
  f32x16 acc[MB][NB];
  int fa[2][MB][A::FRAG], fb[2][NB][B::FRAG];
  int sca[MB][2], scb[NB][2], nca[MB][4], ncb[NB][4];

  __device__ __forceinline__ void init(uint8_t* l, int64_t srow) {
    lds = l, base = (uint32_t)(uintptr_t)l;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    wa = (wave / WAVES_B) * (32 * MB), wb = (wave % WAVES_B) * (32 * NB);
    slot = 0;
#pragma unroll
    for (int i = 0; i < SI; ++i) {
      stile[i] = (wave * SI + i) % ((WA + WB) / 32);
      const int row = 32 * stile[i] + (lane >> 1);
      svoff[i] = (uint32_t)((row < WA ? row : row - WA) * srow + ((lane & 1) ^ swz2(row)) * 16);
    }
    soff = (uint32_t)(2 * STAGE + (lane & 31) * 32 + swz2(lane) * 16);
    clear();
  }

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  }

  // the scale bytes of 1024 columns, where `skip` is 0
  __device__ __forceinline__ void transfer_scales(int skip, const Stretch& ga, const Stretch& gb) {
    const i32x4 ra = ga.rsrc(), rb = gb.rsrc();
#pragma unroll
    for (int i = 0; i < SI; ++i) {
      dma16_unless(skip, 32 * stile[i] < WA ? ra : rb,
                   (uint32_t)__builtin_amdgcn_readfirstlane((int)(base + 2 * STAGE + stile[i] * 1024)), svoff[i]);
    }
  }

  // the i-th of a stage's PER transfers, into the ring's half at `to`
  __device__ __forceinline__ void transfer(int i, uint32_t to) {
    if (i == 0) a.open(0), b.open(tail);
    if (i < A::NI) a.transfer(i, base + to, wave);
    else b.transfer(i - A::NI, base + to + A::BYTES, wave);
    if (i == PER - 1) a.mem.advance(), b.mem.advance();
  }

  // the t-th of the MB + NB fragments of step J of the stage at `from` into set SET
  template <int SET, int J, int T>
  __device__ __forceinline__ void read_frag(uint32_t from) {
    if constexpr (T < MB) a.template read<J, T>(lds + from, fa[SET][T]);
    else b.template read<J, T - MB>(lds + from + A::BYTES, fb[SET][T - MB]);
  }

  // scale bytes of stages `at` (even) and at + 1, 16 of each row
  __device__ __forceinline__ void read_scales(int at) {
    const uint8_t* p = lds + (soff ^ (uint32_t)((at >> 1 & 1) * 16));
    static_for<0, MB + NB>([&](auto t) {
      constexpr int T = decltype(t)::value;
      const i32x4 v = *reinterpret_cast<const i32x4*>(p + (T < MB ? wa + 32 * T : WA + wb + 32 * (T - MB)) * 32);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (T < MB) nca[T][q] = v[q];
        else ncb[T - MB][q] = v[q];
      }
    });
  }

  // those of the pair's stage P into the products' registers; lanes 32..63 take the odd blocks' bytes
  template <int P>
  __device__ __forceinline__ void take_scales() {
    const int sh = 8 * (lane >> 5);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
#pragma unroll
      for (int m = 0; m < MB; ++m) sca[m][q] = (int)((uint32_t)nca[m][2 * P + q] >> sh);
#pragma unroll
      for (int n = 0; n < NB; ++n) scb[n][q] = (int)((uint32_t)ncb[n][2 * P + q] >> sh);
    }
  }

  template <int SET, int J, int M, int N>
  __device__ __forceinline__ void product() {
    if constexpr (!MX) {
      acc[M][N] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          __builtin_bit_cast(bf16x8, (i32x4){fa[SET][M][0], fa[SET][M][1], fa[SET][M][2], fa[SET][M][3]}),
          __builtin_bit_cast(bf16x8, (i32x4){fb[SET][N][0], fb[SET][N][1], fb[SET][N][2], fb[SET][N][3]}), acc[M][N],
          0, 0, 0);
    } else {
      constexpr int FB = KB == K_E2M1 ? 4 : 0, Q = J >> 1, OS = 2 * (J & 1);
      const i32x8 x = as_operand<KA>(fa[SET][M]), y = as_operand<KB>(fb[SET][N]);
      if constexpr (KB == K_E4M3) {
        i32x8 hi, lo;
        split_e4m3(y, hi, lo);
        acc[M][N] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, lo, acc[M][N], 4, FB, OS, sca[M][Q], OS, scb[N][Q]);
        acc[M][N] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, hi, acc[M][N], 4, FB, OS, sca[M][Q], OS, scb[N][Q]);
      } else {
        acc[M][N] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc[M][N], 4, FB, OS, sca[M][Q], OS, scb[N][Q]);
      }
    }
  }

  // step J; between its products the fragments of the next step (of the stage at `from`) and transfers T0 .. T1 - 1
  // of the stage being brought into `to`
  template <int J, int T0, int T1>
  __device__ __forceinline__ void step(uint32_t from, uint32_t to) {
    static_for<0, NM>([&](auto ic) {
      constexpr int i = decltype(ic)::value;
      product<J & 1, J, i / NB, i % NB>();
      static_for<i * (MB + NB) / NM, (i + 1) * (MB + NB) / NM>(
          [&](auto t) { read_frag<(J + 1) & 1, (J + 1) & 3, decltype(t)::value>(from); });
      static_for<T0 + i * (T1 - T0) / NM, T0 + (i + 1) * (T1 - T0) / NM>([&](auto t) { transfer(decltype(t)::value, to); });
      __builtin_amdgcn_sched_barrier(0);
    });
  }

  // stage `at` of nk, the P-th of a pair
  template <int P>
  __device__ __forceinline__ void stage(int at, int nk) {
    const uint32_t other = STAGE - slot;
    if constexpr (MX) take_scales<P>();
    step<0, D3, D0>(slot, other);
    step<1, D0, D1>(slot, other);
    step<2, D1, D1>(slot, other);
    wait_and_barrier<0>();
    const bool cross = at + 2 == nk;  // the next stage to bring is the next tile's first
    a.mem.take_if(cross, an), b.mem.take_if(cross, bn);
    if constexpr (MX) {
      // Scale bytes are read two stages at a time. Those of the four stages that the buffer holds have all been read
      // when the third's last step begins (the tile's when its last stage but one's does); the next ones arrive before
      // the fourth's.
      if constexpr (P == 1) {
        read_scales(at + 1 == nk ? 0 : at + 1);
      } else {
        Stretch ga = sa.at((at + 2) >> 2), gb = sb.at((at + 2) >> 2);
        ga.take_if(cross, san), gb.take_if(cross, sbn);
        transfer_scales(((at & 3) ^ 2) & (cross ? 0 : -1), ga, gb);
      }
    }
    step<3, 0, D3>(other, slot);
    slot = other;
  }

  // Brings the first tile's first stages and reads its first fragments. nk >= 2 for every tile, and even for MX
  // operands: stages past the operands' last one multiply zeros (their transfers bring zeros, and the format keeps the
  // scale bytes behind a row's last block at 0).
  __device__ __forceinline__ void start() {
    if constexpr (MX) transfer_scales(0, sa, sb);
#pragma unroll
    for (int i = 0; i < PER; ++i) transfer(i, 0);
#pragma unroll
    for (int i = 0; i < D3; ++i) transfer(i, STAGE);
    wait_and_barrier<D3>();
    static_for<0, MB + NB>([&](auto t) { read_frag<0, 0, decltype(t)::value>(0); });
    if constexpr (MX) read_scales(0);
  }

  // A tile; when it ends, the first stages of the next one (an, bn, san, sbn; no stages if there is none) are on their
  // way.
  __device__ __forceinline__ void multiply(int nk) {
    if constexpr (MX) {
      for (int at = 0; at < nk; at += 2) stage<0>(at, nk), stage<1>(at + 1, nk);
      sa = san, sb = sbn;
    } else {
      for (int at = 0; at < nk; ++at) stage<0>(at, nk);
    }
  }
};

// Order of the tiles. A launch has up to one workgroup for each place that the chip has for it, a multiple of 8; workgroup
// b runs on XCD b mod 8. Each XCD owns a run of tiles, ordered in strips of up to 4 tiles of the second operand, and its
// workgroups take them in turn, so that the tiles that run together on an XCD share operands in its L2 (of strips of 4 / 8
// / 16: 16384 x 4096 x 11008 in 4 bits 406 / 407 / 418 us, dW 8192 x 11008 x 4096 628 / 642 / 662).
struct TileOrder {
  static constexpr int STRIP = 4;
  int per_xcd, start, end, step, ta, tb;
  __device__ __forceinline__ void init(int b, int grid, int ta_, int tb_) {
    ta = ta_, tb = tb_, step = grid >> 3;
    per_xcd = (ta * tb + 7) / 8;
    start = (b & 7) * per_xcd + (b >> 3);
    end = min(ta * tb, ((b & 7) + 1) * per_xcd);
  }
  // the r-th tile of this workgroup; false: there is none
  __device__ __forceinline__ bool get(int r, int& ia, int& ib) const {
    const int p = start + r * step;
    if (p >= end) return false;
    const int strip = p / (STRIP * ta), rest = p - strip * STRIP * ta;
    const int h = min(STRIP, tb - strip * STRIP);
    ia = rest / h, ib = strip * STRIP + rest % h;
    return true;
  }
};

// workgroups of a launch of `tiles`, `places` fitting the chip at once
static inline unsigned tile_grid(int64_t tiles, int places) {
  return (unsigned)(tiles < places ? (tiles + 7) / 8 * 8 : places);
}

// Writes a wave's results, 32 NB rows of Y (from row0 on, of `rows`) by 32 MB columns (from c0 on, of `cols`): register i
// of lane l of acc[mb][nb] is row 32 nb + l % 32, column 32 mb + 8 (i / 4) + 4 (l / 32) + i % 4. They go through LDS, so
// that a store takes runs of 32 PB columns of a row (16-byte stores straight from the registers, 32 bytes of a row each,
// took 1.6 times as long for fp32 results of 8192 x 8192 and as long for bf16). lds: 4 PB KB a wave.
//
// The code of this part counts: it runs once a tile, and comes from memory if it is long (with the edges' cases expanded
// for each block it grew to 90 KB, and the 4-bit product at 16384 x 4096 x 11008 took 446 us instead of 390). Blocks
// inside Y take 16-byte stores, a lane completing V consecutive columns of IT rows: done.row(set, it, row, c) fetches what
// a row needs and done.keep(set, b) what remains of it for block b, before the first store; done.columns(c) is called for
// each new c and done.finish(b, it, v) completes the results. Blocks at an edge go one column a lane by
// done.one(row, c, v).
template <bool YBF16, int PB, int MB, int NB, typename D>
__device__ __forceinline__ void store_rows(const f32x16 (&acc)[MB][NB], uint8_t* lds, void* __restrict__ Y, int64_t ld,
                                           int64_t row0, int64_t rows, int c0, int cols, bool add, D&& done) {
  constexpr int C = 32 * PB, V = YBF16 ? 8 : 4, PER_ROW = C / V, STEP = 64 / PER_ROW, IT = 32 / STEP;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float* buf = reinterpret_cast<float*>(lds + wave * (4096 * PB));
  const int r = lane & 31, h = lane >> 5;
  const bool inside = row0 + 32 * NB <= rows && c0 + 32 * MB <= cols;
  // the 16-byte chunks of row r are permuted by XOR with r, so that neither side's rows meet on the same banks
  auto chunk = [](int row, int q) { return row * C + ((q ^ (row & (C / 4 - 1))) << 2); };
  // What the rows need is all fetched before the first store: loads and stores end in their order, so a load behind a store
  // would wait for it.
  if (inside) {
    constexpr int BLOCKS = MB / PB * NB, BATCH = BLOCKS < 4 ? BLOCKS : 4;
#pragma unroll
    for (int b0 = 0; b0 < BLOCKS; b0 += BATCH) {
#pragma unroll
      for (int b = b0; b < b0 + BATCH; ++b)
#pragma unroll
        for (int it = 0; it < IT; ++it)
          done.row(b % BATCH, it, row0 + b % NB * 32 + lane / PER_ROW + it * STEP,
                   c0 + 32 * PB * (b / NB) + (lane % PER_ROW) * V);
#pragma unroll
      for (int b = b0; b < b0 + BATCH; ++b) done.keep(b % BATCH, b);
    }
  }
#pragma unroll
  for (int m0 = 0; m0 < MB; m0 += PB) {
    const int c = c0 + 32 * m0 + (lane % PER_ROW) * V;
    if (inside) done.columns(c);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      const int b = m0 / PB * NB + nb;
      const int64_t first = row0 + nb * 32 + lane / PER_ROW;
#pragma unroll
      for (int mb = 0; mb < PB; ++mb)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<float4*>(buf + chunk(r, mb * 8 + 2 * g + h)) =
              make_float4(acc[m0 + mb][nb][4 * g], acc[m0 + mb][nb][4 * g + 1], acc[m0 + mb][nb][4 * g + 2],
                          acc[m0 + mb][nb][4 * g + 3]);
      __builtin_amdgcn_wave_barrier();
      if (inside) {
#pragma unroll
        for (int it = 0; it < IT; ++it) {
          float v[V];
#pragma unroll
          for (int q = 0; q < V / 4; ++q) {
            const float4 x = *reinterpret_cast<const float4*>(
                buf + chunk(lane / PER_ROW + it * STEP, (lane % PER_ROW) * (V / 4) + q));
            v[4 * q] = x.x, v[4 * q + 1] = x.y, v[4 * q + 2] = x.z, v[4 * q + 3] = x.w;
          }
          done.finish(b, it, v);
          const int64_t at = (first + it * STEP) * ld + c;
          if (YBF16) {
            *reinterpret_cast<i32x4_any*>(static_cast<uint16_t*>(Y) + at) =
                (i32x4){(int)bf16_pair(v[0], v[1]), (int)bf16_pair(v[2], v[3]), (int)bf16_pair(v[V - 4], v[V - 3]),
                        (int)bf16_pair(v[V - 2], v[V - 1])};
          } else {
            f32x4_any* p = reinterpret_cast<f32x4_any*>(static_cast<float*>(Y) + at);
            f32x4 o = {0.f, 0.f, 0.f, 0.f};
            if (add) o = *p;
            *p = o + (f32x4){v[0], v[1], v[2], v[3]};
          }
        }
      } else {
        const int e = c0 + 32 * m0 + (lane & (C - 1));
        const int n = (int)max((int64_t)0, min((int64_t)32, rows - (row0 + nb * 32)));
        if (e < cols) {
#pragma unroll 1
          for (int i = lane / C; i < n; i += 64 / C) {
            const int64_t row = row0 + nb * 32 + i;
            const float v = done.one(row, e, buf[chunk(i, (lane & (C - 1)) >> 2) + (lane & 3)]);
            if (YBF16) {
              static_cast<uint16_t*>(Y)[row * ld + e] = (uint16_t)bf16_bits(v);
            } else {
              float* p = static_cast<float*>(Y) + row * ld + e;
              *p = add ? *p + v : v;
            }
          }
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

// partial products leave as they are
struct StoreAsIs {
  __device__ __forceinline__ void columns(int) {}
  __device__ __forceinline__ void row(int, int, int64_t, int) {}
  __device__ __forceinline__ void keep(int, int) {}
  __device__ __forceinline__ float one(int64_t, int, float v) { return v; }
  template <int V>
  __device__ __forceinline__ void finish(int, int, float (&)[V]) {}
};

}  // namespace gptq
