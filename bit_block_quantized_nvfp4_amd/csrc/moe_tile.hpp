// Tiled matrix product of 16-bit floats or 8-bit integers,
//
//   z[m][n] = sum_k A[m][k] B[n][k],   out = epilogue(z),
//
// for the dense feed-forward block and the 8-bit integer products.  Each operand
// stands in memory with k running fastest, or (16 bits) with its rows running
// fastest: the transposed matrix, as the gradients need it.
//
// A block computes BN columns of BM rows in steps of 128 bytes along K.
// Both operands go from memory to LDS without registers, 16 bytes a lane, A's NA and
// B's NB steps deep; a step's products then run on the 32x32 MFMA with sums in 32 bits.
// B is the MFMA's first operand, so a lane holds four consecutive outputs of a row.
//
// LDS.  k fastest: a row of a step is 128 bytes, its 16-byte chunk c stands at place
// c ^ (row / 2 % 8), so that the 16 rows that one cycle of a 16-byte read serves meet
// all 64 banks.  Rows fastest: a k is a line of BN (BM) values, read with the
// transposing load: 16 lanes get four k of 16 rows; its chunks are permuted so
// that the four lines of such a load meet different banks.  The loads to LDS write
// lanes in order, so both permutations are applied to the addresses they read.
//
// Past the ends of an operand zeros come: rows by the buffer's size, columns and
// the end of K by an offset past it, for both operands, so that nothing that
// stands behind a row (a NaN of the next one) is multiplied.
//
// Large products keep the matrix unit busy 79 % of its cycles, at a clock that falls as it
// fills (MFMAs alone reach 1.7 PFLOP/s; 8192 x 2048 x 8192 in bf16 takes 205 us, 1.34, where
// the library's product takes 170; in 8-bit integers 117 us, 2.36 POP/s): a wave of 128 x 128
// reads the fewest bytes from LDS for its products.  Small ones are bound by the latency of their
// steps, 0.3 to 0.45 us each: hence the deep rings and the groups along K.
#pragma once

#include <algorithm>

#include "moe_dma.hpp"
#include "moe_ffn_common.hpp"
#include "moe_internal.hpp"
#include "moe_vec.hpp"

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t lds_u8;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kElI8 = 16;  // beside MOE_DT_BF16 and MOE_DT_F16

// Lane l of an operand of 32 rows holds row l % 32, the 16 bytes of K from 16 (l / 32)
// on.  Element e of lane l of the product: row 8 (e / 4) + 4 (l / 32) + e % 4 of a, row
// l % 32 of b.
template <int EL>
struct Mma {
  typedef f32x16 Acc;
  typedef f32x4 Four;
  static __device__ __forceinline__ Acc go(u32x4 a, u32x4 b, Acc c) {
    if constexpr (EL == MOE_DT_BF16)
      return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                     __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                    __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
template <>
struct Mma<kElI8> {
  typedef i32x16 Acc;
  typedef i32x4 Four;
  static __device__ __forceinline__ Acc go(u32x4 a, u32x4 b, Acc c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  }
};

struct TileArgs16 {
  const void* a;       // rows of the output (M)
  const void* b;       // columns (N; gated: N gate rows, then N up rows)
  uint32_t lda, ldb;   // bytes from one stored line to the next
  int M, N, K;
  int nt;              // tiles along N
  void* out;
  void* out2;
  const void* aux;
  const float* sm;     // scales of rows and columns (8-bit integers)
  const float* sn;
};

constexpr int SB = 128;  // bytes of a step along K, of each row
// Steps along K of values of es bytes.  K is the rows' number for the weights' gradients:
// up to 2^30, whose bytes pass an int.
constexpr long steps_of(int K, int es) { return ((long)K * es + SB - 1) / SB; }
static_assert(steps_of(1 << 30, 2) == 1 << 24 && steps_of((1 << 30) - 63, 2) == 1 << 24 &&
                  steps_of((1 << 30) - 64, 2) == (1 << 24) - 1 && steps_of(8, 2) == 1 && steps_of(65536, 1) == 512,
              "steps at the limits");
constexpr uint32_t kNowhere = 0x80000000u;  // past the end of every buffer (all below 2^31 bytes)

// Permutation of the 16-byte chunks of a line: rows fastest, a line of CPR chunks.
template <int CPR>
__device__ __forceinline__ int line_swz(int k) {
  return CPR >= 16 ? 4 * (k & 3) : CPR == 8 ? 4 * ((k >> 1) & 1) : 0;
}

// One operand of a block: R rows of it, ROWS fastest or k fastest, brought by NT
// threads.  GATED: the first half of the rows are gate rows, the second the up rows of
// the same columns, which stand `up` bytes behind.
template <int ES, bool ROWS, int R, int NT, bool GATED>
struct Operand {
  static constexpr int kC = SB / 16;           // chunks of a row and step
  static constexpr int kLoads = R * kC / NT;   // per thread and step
  static constexpr int CPR = R / 8;            // chunks of a line (rows fastest)
  static constexpr int KS = SB / ES;           // values of K in a step
  static_assert(R * kC % NT == 0 && NT % 64 == 0 && (!ROWS || (ES == 2 && !GATED)) && (!GATED || kLoads % 2 == 0),
                "operand shape");
  const char* base;
  const char* up;
  uint32_t ld, kbytes, width;                // width: rows' bytes (ROWS) or bytes of the tile
  uint32_t off[kLoads];
  int chunk;

  // first: the tile's first row; left: rows from there on; K values along K
  __device__ __forceinline__ void set(const void* p, uint32_t ld_, long first, int left, int K,
                                      long up_bytes, int tid) {
    ld = ld_;
    kbytes = (uint32_t)K * ES;
    if constexpr (ROWS) {
      base = (const char*)p + first * ES;
      width = (uint32_t)min(left, R) * ES;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int at = i * NT + tid, k = at / CPR, c = (at % CPR) ^ line_swz<CPR>(k);
        off[i] = (uint32_t)c * 16 < width ? (uint32_t)k * ld + c * 16 : kNowhere;
      }
    } else {
      base = (const char*)p + first * (long)ld;
      up = base + up_bytes;
      constexpr int RR = GATED ? R / 2 : R;
      width = (uint32_t)min(left, RR) * ld;
      chunk = 16 * ((tid % kC) ^ ((tid >> 4) % kC));  // of load 0: row / (16 / kC) = tid / 16
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        off[i] = (uint32_t)((i * NT + tid) / kC % RR) * ld + chunk_of(i);
      }
    }
  }
  // The byte of its row's step that load i begins at.
  __device__ __forceinline__ int chunk_of(int i) const { return NT == 64 ? chunk ^ (i % 2 * 64) : chunk; }
  // What the loads of a step share.
  struct Step {
    u32x4 buf, ubuf;
    uint32_t so, ko;
  };
  __device__ __forceinline__ Step begin(int s) const {
    Step t;
    if constexpr (ROWS) {
      const int k0 = s * KS, kn = min((int)(kbytes / ES) - k0, KS);
      t.buf = buf_of(base + (size_t)k0 * ld, kn > 0 ? (uint32_t)(kn - 1) * ld + width : 0u);
      asm volatile("s_nop 4" : "+s"(t.buf));  // as in dma_offset
    } else {
      t.ko = (uint32_t)s * SB;
      t.buf = buf_of(base, width);
      asm volatile("s_nop 4" : "+s"(t.buf));
      if constexpr (GATED) {
        t.ubuf = buf_of(up, width);
        asm volatile("s_nop 4" : "+s"(t.ubuf));
      }
      t.so = dma_offset(min(t.ko, kbytes));
    }
    return t;
  }
  // Load i of a step to the LDS address lds (the wave's share of it).
  __device__ __forceinline__ void load(const Step& t, int i, uint32_t lds) const {
    if constexpr (ROWS)
      dma_b128(t.buf, off[i], 0, lds + i * NT * 16);
    else
      dma_b128(GATED && i >= kLoads / 2 ? t.ubuf : t.buf, t.ko + chunk_of(i) < kbytes ? off[i] : kNowhere, t.so,
               lds + i * NT * 16);
  }
};

// 32 rows from `row` of an operand in LDS, the ks-th 32 bytes of the step.
template <bool ROWS, int R>
__device__ __forceinline__ u32x4 operand_at(const lds_u8* p, int row, int ks, int lane) {
  if constexpr (ROWS) {
    constexpr int CPR = R / 8, LINE = R * 2;
    const int g = lane >> 4, i = lane & 15;
    const int k = 16 * ks + 8 * (g >> 1) + (i >> 2), n = row + 16 * (g & 1) + 4 * (i & 3);
    const lds_u8* q = p + k * LINE + (((n >> 3) ^ line_swz<CPR>(k)) << 4) + 8 * (i & 1);
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)q);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(q + 4 * LINE));
    const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
    return u32x4{a.x, a.y, b.x, b.y};
  } else {
    const int fr = lane & 31, fq = lane >> 5;
    return *(const __attribute__((address_space(3))) u32x4*)(
        p + (row + fr) * SB + (((fq + 2 * ks) ^ (fr / 2 % 8)) << 4));
  }
}

// An epilogue that reads nothing from memory ahead.
struct NoPre {
  __device__ __forceinline__ void get(const TileArgs16&, int, int) {}
};

// EP: the epilogue.  EP::kGated: a wave's columns are TN / 2 gates and the TN / 2 ups of
// the same outputs; EP::put(a, m, n, v, u, pre): outputs n .. n + 7 of row m (both
// inside) from the sums v (and u, the ups) and what EP::Pre::get(a, m, n) has read.
// KG groups of waves with buffers of their own take every KG-th step and join their sums
// at the end, in the groups' order: where there are few tiles, a step costs its
// waiting whatever its size.
template <int BN_, int BM_, int WN_, int WM_, int NA_, int NB_, int KG_ = 1>
struct TileShape {
  static constexpr int BN = BN_, BM = BM_, WN = WN_, WM = WM_, NA = NA_, NB = NB_, KG = KG_;
  static constexpr int kThreads = 64 * WN * WM * KG;
  static constexpr int kGroupLds = (NA * BM + NB * BN) * SB, kLds = KG * kGroupLds;
};

// Block `blk` of the `blocks` of a product.
template <int EL, bool BROWS, bool AROWS, class EP, class TS>
__device__ __forceinline__ void tile_block(const TileArgs16& a, const int blk, const int blocks, lds_u8* const lds) {
  constexpr int BN = TS::BN, BM = TS::BM, WN = TS::WN, WM = TS::WM, NA = TS::NA, NB = TS::NB, KG = TS::KG;
  constexpr int NW = WN * WM, NT = 64 * NW;                  // waves and threads of a group
  constexpr int TN = BN / WN, TM = BM / WM;
  constexpr int FN = TN / 32, FM = TM / 32;
  constexpr int ES = EL == kElI8 ? 1 : 2;
  constexpr int kA = BM * SB, kB = BN * SB, kLds = TS::kGroupLds;  // bytes of a step, of a group
  constexpr int KF = SB / 32;                                // products along K of a step
  constexpr bool G = EP::kGated;
  constexpr int BC = G ? BN / 2 : BN, TC = G ? TN / 2 : TN;  // outputs of a tile and of a wave
  constexpr int CH = TN / 4;                                 // 16-byte chunks of a staged row
  typedef typename Mma<EL>::Acc Acc;
  typedef typename Mma<EL>::Four Four;
  static_assert(TN % 32 == 0 && TM % 32 == 0 && (!G || FN % 2 == 0) && NA >= 2 && NB >= NA, "tile shape");
  constexpr int kStage = 32 * TN * 4;                        // bytes of 32 staged rows
  static_assert(NW * 2 * kStage <= KG * kLds && CH <= 32 && (CH & (CH - 1)) == 0, "staged rows");
  const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane((int)threadIdx.x / NT);
  const int tid = (int)threadIdx.x - kg * NT, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wv % WN, wm = wv / WN;

  // Blocks are dealt to the 8 XCDs in turn: each XCD gets a run of tiles, 8 row tiles
  // deep before the next column tile, so that the blocks that run together on one
  // share the lines of both operands in its L2
  const int mt = (a.M + BM - 1) / BM, per = blocks / 8;
  const int lin = blk < per * 8 ? (blk % 8) * per + blk / 8 : blk;
  const int deep = 8 * a.nt, grp = lin / deep, in = lin % deep;
  const int gm = min(8, mt - grp * 8);
  const int m0 = __builtin_amdgcn_readfirstlane((grp * 8 + in % gm) * BM);
  const int n0 = __builtin_amdgcn_readfirstlane((in / gm) * BC);

  typedef Operand<ES, BROWS, BN, NT, G> OpB;
  typedef Operand<ES, AROWS, BM, NT, false> OpA;
  constexpr int LA = OpA::kLoads, D = LA + OpB::kLoads;
  // loads that a wave may have under way where it waits for the next step's
  constexpr int kAhead = (NA - 2) * D + (NB > NA ? D - LA : 0);
  static_assert(kAhead + D < 64, "loads under way");
  OpB ob;
  OpA oa;
  ob.set(a.b, a.ldb, n0, a.N - n0, a.K, (long)a.N * a.ldb, tid);
  oa.set(a.a, a.lda, m0, a.M - m0, a.K, 0, tid);
  lds_u8* const l0 = lds + kg * kLds;
  const uint32_t ldsw = (uint32_t)(uintptr_t)l0 + wv * 1024;
  const int steps = (int)((steps_of(a.K, ES) + KG - 1) / KG);  // of a group

  // Step s's turn at the buffers that step s - 1 leaves: the loads of A's step s - 1 + NA,
  // then of B's step s - 1 + NB.  Steps past the last one are brought too, as zeros
  // from outside the operands, so that every wave has the same loads under way at
  // every wait.
  int a_at = 0, b_at = 0;
  typename OpB::Step tb;
  typename OpA::Step ta;
  auto begin = [&](int s) __attribute__((always_inline)) {
    ta = oa.begin((s - 1 + NA) * KG + kg);
    tb = ob.begin((s - 1 + NB) * KG + kg);
  };
  auto load = [&](int i) __attribute__((always_inline)) {
    if (i < LA) oa.load(ta, i, ldsw + NB * kB + a_at);
    else ob.load(tb, i - LA, ldsw + b_at);
    if (i == LA - 1) a_at = a_at == (NA - 1) * kA ? 0 : a_at + kA;
    if (i == D - 1) b_at = b_at == (NB - 1) * kB ? 0 : b_at + kB;
  };
  constexpr int L = D / KF;  // loads that go with the first products
#pragma unroll
  for (int s = 1 - NB; s <= 0; ++s) {
    begin(s);
#pragma unroll
    for (int i = s > -NA ? 0 : LA; i < (s < 0 ? D : L); ++i) load(i);
  }

  Acc acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = Acc{};
  struct Frags {
    u32x4 b[FN], a[FM];
  };
  // Operand r of the ks-th 32 bytes of the step at pa and pb: b's first, all of a's, then
  // b's others.
  const lds_u8 *pa = l0 + NB * kB, *pb = l0;
  auto read = [&](Frags& f, int r, int ks) __attribute__((always_inline)) {
    if (r > 0 && r <= FM) f.a[r - 1] = operand_at<AROWS, BM>(pa, wm * TM + 32 * (r - 1), ks, lane);
    else {
      const int i = r ? r - FM : 0;
      // gated: a wave's columns are gates, then the ups of the same outputs
      const int row = !G ? wn * TN + 32 * i : wn * TC + 32 * i + (i < FN / 2 ? 0 : BN / 2 - TC);
      f.b[i] = operand_at<BROWS, BN>(pb, row, ks, lane);
    }
  };
  // The products of f, and between them the reads of g, the operands of the next ones,
  // and the part'th share of the loads of the step under way: any of these in one piece would
  // hold up the wave with its matrix unit idle.
  auto multiply = [&](const Frags& f, Frags& g, int ks, int part) __attribute__((always_inline)) {
    constexpr int M = FN * FM, R = FN + FM;
    const int from = part * D / KF, n = (part + 1) * D / KF - from;
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) {
        const int m = i * FM + j;
        acc[i][j] = Mma<EL>::go(f.b[i], f.a[j], acc[i][j]);
        if (m < R) read(g, m, ks);
        if (m == M - 1)
#pragma unroll
          for (int r = M; r < R; ++r) read(g, r, ks);
#pragma unroll
        for (int d = 0; d < n; ++d)
          if ((2 * d + 1) * M / (2 * n) == m) load(from + d);
        __builtin_amdgcn_sched_barrier(0);
      }
  };
  // A step's buffers are free once every wave has read its last operands.  The waves
  // meet there, before the products of these; from there on the buffers are filled
  // again.  A's, which are wanted sooner, come first.
  wait_step<kAhead + L>();
  Frags f[2];  // of these and of the next products, in turn
#pragma unroll
  for (int r = 0; r < FN + FM; ++r) read(f[0], r, 0);
  for (int s = 0; s < steps; ++s) {
#pragma unroll
    for (int ks = 0; ks < KF; ++ks) {
      const int next = ks + 1 == KF ? 0 : ks + 1;
      if (next == 0) {
        begin(s + 1);
        wait_step<kAhead>();
        pa = pa == l0 + NB * kB + (NA - 1) * kA ? l0 + NB * kB : pa + kA;
        pb = pb == l0 + (NB - 1) * kB ? l0 : pb + kB;
      }
      multiply(f[ks & 1], f[1 - (ks & 1)], next, next);
    }
  }
  wait_step<0>();  // nothing is under way to LDS, nothing is read from it any more
  if constexpr (KG > 1) {
    // lane by lane, 16 bytes at a time, behind the places of the rows below
    lds_u8* const sums = lds + NW * 2 * kStage + tid * 16;
    static_assert(NW * 2 * kStage + (KG - 1) * BN * BM * 4 <= KG * kLds, "the groups' sums fit");
    auto place = [&](int g, int i, int j, int q) __attribute__((always_inline)) {
      return (__attribute__((address_space(3))) Four*)(sums + (((g * FN + i) * FM + j) * 4 + q) * (NT * 16));
    };
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (kg > 0)
            *place(kg - 1, i, j, q) =
                Four{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
    meet();
    if (kg > 0) return;
#pragma unroll
    for (int g = 0; g < KG - 1; ++g)
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const Four w = *place(g, i, j, q);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][4 * q + e] += w[e];
          }
  }

  // The wave's sums, 32 rows at a time, through LDS of its own (two places in turn): a
  // lane then has eight consecutive outputs of a row, and memory is read and written
  // in whole pieces of rows.  Chunk c of a staged row stands at c ^ (row % chunks), for
  // the banks.  A wave's LDS operations keep their order.  What the epilogue reads from
  // memory is asked for 32 rows ahead.
  constexpr int LR = TC / 8, RP = 64 / LR, P = 32 / RP;  // lanes of a row, rows of a pass, passes
  const int fr = lane & 31, fq = lane >> 5;
  const int r0 = lane / LR, c8 = lane % LR, n = n0 + wn * TC + 8 * c8;
  lds_u8* const mine = l0 + wv * (2 * kStage);
  auto stage = [&](int j) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *(__attribute__((address_space(3))) Four*)(mine + j % 2 * kStage + fr * (TN * 4) +
                                                   (((8 * i + 2 * g + fq) ^ (fr & (CH - 1))) << 4)) =
            Four{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
  };
  auto row_of = [&](int j, int q) __attribute__((always_inline)) { return m0 + wm * TM + 32 * j + q * RP + r0; };
  typename EP::Pre pre[2][P];
  auto fetch = [&](int j) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < P; ++q)
      if (row_of(j, q) < a.M && n < a.N) pre[j % 2][q].get(a, row_of(j, q), n);
  };
  fetch(0);
  stage(0);
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    if (j + 1 < FM) {
      fetch(j + 1);
      stage(j + 1);
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int q = 0; q < P; ++q) {
      const int r = q * RP + r0, m = row_of(j, q);
      float v[8], u[8];
      auto row8 = [&](int c, float (&f)[8]) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const Four w = *(const __attribute__((address_space(3))) Four*)(
              mine + j % 2 * kStage + r * (TN * 4) + (((c + h) ^ (r & (CH - 1))) << 4));
#pragma unroll
          for (int e = 0; e < 4; ++e) f[4 * h + e] = (float)w[e];
        }
      };
      row8(2 * c8, v);
      if (G) row8(TC / 4 + 2 * c8, u);
      if (m < a.M && n < a.N) EP::put(a, m, n, v, u, pre[j % 2][q]);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int EL, bool BROWS, bool AROWS, class EP, class TS>
__global__ __launch_bounds__(TS::kThreads) void k_tile(TileArgs16 a) {
  __shared__ __align__(1024) uint8_t lds[TS::kLds];
  tile_block<EL, BROWS, AROWS, EP, TS>(a, blockIdx.x, gridDim.x, (lds_u8*)lds);
}

// ---- host side: the shapes, and which of them a product takes

// f with the shape as a type.
constexpr int kTileShapes16 = 8;
template <typename F>
static void by_shape(int shape, F&& f) {
  if (shape == 0) f(TileShape<256, 256, 2, 2, 2, 3>{});
  if (shape == 1) f(TileShape<256, 128, 2, 2, 2, 3>{});
  if (shape == 2) f(TileShape<128, 128, 2, 2, 4, 4>{});
  if (shape == 3) f(TileShape<128, 128, 2, 2, 2, 2>{});
  if (shape == 4) f(TileShape<128, 64, 2, 2, 3, 3, 2>{});
  if (shape == 5) f(TileShape<64, 64, 1, 2, 4, 4>{});
  if (shape == 6) f(TileShape<64, 64, 1, 2, 4, 4, 2>{});
  if (shape == 7) f(TileShape<64, 32, 1, 1, 3, 3, 4>{});
}

// Tiles of a product in a shape.
static inline long tiles_of(int shape, int M, int cols) {
  long n = 0;
  by_shape(shape, [&](auto s) {
    n = (long)((cols + s.BN - 1) / s.BN) * ((M + s.BM - 1) / s.BM);
  });
  return n;
}

// Time of a round of tiles on the chip, in 10 ns, beyond the launch's 2.5 us: `fixed1` +
// steps * `step1` with one block on each compute unit, the first of them; `fixed` + steps *
// `step` every further one, or with two blocks on each where `places` is 512.  From
// launches of 256 and 1024 tiles, 1 to 64 steps (bf16, in a row in a graph, us; the three
// layouts differ by up to a tenth, 8-bit integers by the writes of as many more outputs
// per byte):
//                        256 tiles                      1024 tiles
//   steps            1     4    16     64         1     4    16     64
//   256 x 256     13.6  17.8  35.8    113      39.7  60.0   135    421
//   256 x 128      8.6  10.8  20.5   65.4      25.0  31.3  86.0    251
//   128 x 128, a   5.7   7.2  13.0   43.5      17.5  21.6  51.1    160
//   128 x 128, b   5.4   7.8  15.7   60.6      12.9  17.1  46.3    151
//   128 x 64, 2    4.7   5.6   8.7   27.0      15.5  17.3  37.1    110
//   64 x 64        3.7   4.7   8.5   23.4       7.6   9.2  17.1   60.4
//   64 x 64, 2     4.2   4.8   7.2   16.6      13.4  15.4  23.7   77.7
//   64 x 32, 4     4.6   4.7   6.2   12.3      14.5  14.9  20.6   55.7
// (a: buffers of four steps, one block on a compute unit; b: two steps, two blocks, which
// pays where steps are few; ", 2": groups along K).
struct TileCost {
  int places, fixed1, step1, fixed, step;
};
static inline TileCost tile_cost(int shape) {
  constexpr TileCost c[kTileShapes16] = {{256, 870, 157, 830, 151}, {256, 460, 91, 400, 93}, {256, 240, 58, 300, 57},
                                         {512, 170, 88, 285, 112},  {256, 165, 36, 240, 40}, {512, 90, 32, 130, 43},
                                         {256, 150, 20, 220, 28},   {256, 175, 13, 260, 18}};
  return c[shape];
}
// The shape in which the rounds of a product's tiles take the least time together.
static inline int tile_shape(int M, int cols, long steps) {
  int best = 0;
  long least = 0;
  for (int s = 0; s < kTileShapes16; ++s) {
    const TileCost c = tile_cost(s);
    const long tiles = tiles_of(s, M, cols), rounds = (tiles + c.places - 1) / c.places, rest = tiles % c.places;
    const long one = c.places == 256 || (rest > 0 && rest <= 256) ? 1 : 0;
    const long t = (rounds - one) * (c.fixed + steps * c.step) + one * (c.fixed1 + steps * c.step1);
    if (least == 0 || t < least) least = t, best = s;
  }
  return best;
}
// Threads of a product's launch.
static inline uint64_t tile_threads(int M, int cols, long steps) {
  const int best = tile_shape(M, cols, steps);
  uint64_t t = 0;
  by_shape(best, [&](auto shape) { t = (uint64_t)tiles_of(best, M, cols) * shape.kThreads; });
  return t;
}

// Eight or four values of a row, rounded once, nearest even.
template <int DT>
__device__ __forceinline__ void put_row(void* p, size_t at, const float (&v)[8]) {
  if constexpr (DT == MOE_DT_F32) {
    f32x4* q = (f32x4*)((float*)p + at);
    q[0] = f32x4{v[0], v[1], v[2], v[3]};
    q[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    *(u32x4*)((uint16_t*)p + at) = Chunk<DT>::pack(v);
  }
}
template <int DT>
__device__ __forceinline__ void put_row(void* p, size_t at, const float (&v)[4]) {
  if constexpr (DT == MOE_DT_F32)
    *(f32x4*)((float*)p + at) = f32x4{v[0], v[1], v[2], v[3]};
  else if constexpr (DT == MOE_DT_BF16)
    *(u32x2*)((uint16_t*)p + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  else
    *(u32x2*)((uint16_t*)p + at) = u32x2{pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3])};
}

}  // namespace moe
