// Tiled matrix product of 16-bit floats or 8-bit integers,
//
//   z[m][n] = sum_k A[m][k] B[n][k],   out = epilogue(z),
//
// for the dense feed-forward block and the 8-bit integer products.  Each operand
// stands in memory with k running fastest, or (16 bits) with its rows running
// fastest: the transposed matrix, as the gradients need it.
//
// A block computes BN columns of BM rows in steps of 128 bytes along K (64 or 128
// values).  Both operands go from memory to LDS without registers, 16 bytes a
// lane, NBUF steps deep; a step's products then run on the 32x32 MFMA with sums in
// 32 bits.  B is the MFMA's first operand, so a lane holds four consecutive outputs
// of a row.
//
// LDS.  k fastest: a row of a step is 128 bytes, its 16-byte chunk c stands at
// place c ^ (row / 2 % 8), so that the 16 rows that one cycle of a 16-byte read
// serves meet all 64 banks.  Rows fastest: a k is a line of BN (BM) values, read with
// the transposing load: 16 lanes get four k of 16 rows; its chunks are permuted so
// that the four lines of such a load meet different banks.  The loads to LDS write
// lanes in order, so both permutations are applied to the addresses they read.
//
// Past the ends of an operand zeros come: rows by the buffer's size, columns and
// the end of K by an offset past it, for both operands, so that nothing that
// stands behind a row (a NaN of the next one) is multiplied.
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

constexpr int kStepBytes = 128;
constexpr uint32_t kNowhere = 0x80000000u;  // past the end of every buffer (all below 2^31 bytes)

// Permutation of the 16-byte chunks of a line: rows fastest, a line of CPR chunks.
template <int CPR>
__device__ __forceinline__ int line_swz(int k) {
  return CPR >= 16 ? 4 * (k & 3) : CPR == 8 ? 4 * ((k >> 1) & 1) : 0;
}

// One operand of a block: R rows of it, ROWS fastest or k fastest, brought by NT
// threads.  GROUP (gated): every run of GROUP rows is half a run of gate rows, half
// the up rows of the same columns, which stand `up` bytes behind.
template <int ES, bool ROWS, int R, int NT, int GROUP>
struct Operand {
  static constexpr int kLoads = R * 8 / NT;  // per thread and step
  static constexpr int CPR = R / 8;          // chunks of a line (rows fastest)
  static constexpr int KS = kStepBytes / ES; // values of K in a step
  static_assert(R * 8 % NT == 0 && (!ROWS || ES == 2), "operand shape");
  const char* base;
  const char* up;
  uint32_t ld, kbytes, width;                // width: rows' bytes (ROWS) or bytes of the tile
  uint32_t off[kLoads];
  int chunk;
  bool upper[kLoads];

  // first: the tile's first row; left: rows from there on; K values along K
  __device__ __forceinline__ void set(const void* p, uint32_t ld_, long first, int left, int K,
                                      long up_bytes, int tid, int wv) {
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
      constexpr int RR = GROUP ? R / 2 : R;
      width = (uint32_t)min(left, RR) * ld;
      chunk = 16 * ((tid & 7) ^ ((tid >> 4) & 7));
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int lr = (i * NT + tid) >> 3;
        int row = lr;
        if constexpr (GROUP > 0) {
          constexpr int HG = GROUP / 2;
          row = lr / GROUP * HG + lr % HG;
          upper[i] = (i * (NT / 8) + wv * 8) % GROUP >= HG;
        }
        off[i] = (uint32_t)row * ld + chunk;
      }
    }
  }
  // The loads of step s to the LDS address lds (the wave's share of it).
  __device__ __forceinline__ void bring(int s, uint32_t lds) const {
    if constexpr (ROWS) {
      const int k0 = s * KS, kn = min((int)(kbytes / ES) - k0, KS);
      u32x4 buf = buf_of(base + (size_t)k0 * ld, kn > 0 ? (uint32_t)(kn - 1) * ld + width : 0u);
      asm volatile("s_nop 4" : "+s"(buf));  // as in dma_offset
#pragma unroll
      for (int i = 0; i < kLoads; ++i) dma_b128(buf, off[i], 0, lds + i * NT * 16);
    } else {
      const uint32_t ko = (uint32_t)s * kStepBytes;
      u32x4 buf = buf_of(base, width);
      asm volatile("s_nop 4" : "+s"(buf));
      u32x4 ubuf;
      if constexpr (GROUP > 0) {
        ubuf = buf_of(up, width);
        asm volatile("s_nop 4" : "+s"(ubuf));
      }
      const bool in = ko + chunk < kbytes;
      const uint32_t so = dma_offset(min(ko, kbytes));
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if constexpr (GROUP > 0)
          dma_b128(upper[i] ? ubuf : buf, in ? off[i] : kNowhere, so, lds + i * NT * 16);
        else
          dma_b128(buf, in ? off[i] : kNowhere, so, lds + i * NT * 16);
      }
    }
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
        p + (row + fr) * kStepBytes + (((fq + 2 * ks) ^ ((fr >> 1) & 7)) << 4));
  }
}

// EP: the epilogue.  EP::kGated: a wave's columns are TN / 2 gates and the TN / 2 ups of
// the same outputs; EP::put(a, m, n, v, u): outputs n .. n + 7 of row m (both inside)
// from the sums v (and u, the ups).
template <int EL, bool BROWS, bool AROWS, class EP, int BN, int BM, int WN, int WM, int NBUF>
__global__ __launch_bounds__(64 * WN * WM) void k_tile(TileArgs16 a) {
  constexpr int NW = WN * WM, NT = 64 * NW;
  constexpr int TN = BN / WN, TM = BM / WM;
  constexpr int FN = TN / 32, FM = TM / 32;
  constexpr int ES = EL == kElI8 ? 1 : 2;
  constexpr int kBuf = (BN + BM) * kStepBytes;
  constexpr bool G = EP::kGated;
  constexpr int BC = G ? BN / 2 : BN, TC = G ? TN / 2 : TN;  // outputs of a tile and of a wave
  constexpr int CH = TN / 4;                                 // 16-byte chunks of a staged row
  typedef typename Mma<EL>::Acc Acc;
  static_assert(TN % 32 == 0 && TM % 32 == 0 && (!G || FN % 2 == 0) && NBUF >= 2, "tile shape");
  static_assert(NW * 16 * TN * 4 <= NBUF * kBuf && (CH & (CH - 1)) == 0, "staged rows");
  __shared__ __align__(1024) uint8_t lds[NBUF * kBuf];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wv % WN, wm = wv / WN;

  // Blocks are dealt to the 8 XCDs in turn: each XCD gets a run of tiles, 8 row tiles
  // deep before the next column tile, so that the blocks that run together on one
  // share the lines of both operands in its L2
  const int mt = (a.M + BM - 1) / BM, per = (int)gridDim.x / 8, blk = blockIdx.x;
  const int lin = blk < per * 8 ? (blk % 8) * per + blk / 8 : blk;
  const int deep = 8 * a.nt, grp = lin / deep, in = lin % deep;
  const int gm = min(8, mt - grp * 8);
  const int m0 = __builtin_amdgcn_readfirstlane((grp * 8 + in % gm) * BM);
  const int n0 = __builtin_amdgcn_readfirstlane((in / gm) * BC);

  typedef Operand<ES, BROWS, BN, NT, G ? TN : 0> OpB;
  typedef Operand<ES, AROWS, BM, NT, 0> OpA;
  constexpr int D = OpB::kLoads + OpA::kLoads;
  static_assert((NBUF - 1) * D < 64, "loads under way");
  OpB ob;
  OpA oa;
  ob.set(a.b, a.ldb, n0, a.N - n0, a.K, (long)a.N * a.ldb, tid, wv);
  oa.set(a.a, a.lda, m0, a.M - m0, a.K, 0, tid, wv);
  lds_u8* const l0 = (lds_u8*)lds;
  const uint32_t ldsw = (uint32_t)(uintptr_t)l0 + wv * 1024;
  const int steps = (a.K * ES + kStepBytes - 1) / kStepBytes;

  // Steps past the last one are brought too, as zeros from outside the buffers, so
  // that every wave has the same loads under way at every wait.
  int d_at = 0;
  auto bring = [&](int s) __attribute__((always_inline)) {
    oa.bring(s, ldsw + d_at + BN * kStepBytes);
    ob.bring(s, ldsw + d_at);
    d_at = d_at == (NBUF - 1) * kBuf ? 0 : d_at + kBuf;
  };
#pragma unroll
  for (int s = 0; s < NBUF - 1; ++s) bring(s);

  Acc acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = Acc{};
  int at = 0;
  for (int s = 0; s < steps; ++s) {
    wait_step<(NBUF - 2) * D>();
    bring(s + NBUF - 1);
    const lds_u8* pb = l0 + at;
    const lds_u8* pa = pb + BN * kStepBytes;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      u32x4 fb[FN], fa[FM];
#pragma unroll
      for (int i = 0; i < FN; ++i) fb[i] = operand_at<BROWS, BN>(pb, wn * TN + 32 * i, ks, lane);
#pragma unroll
      for (int j = 0; j < FM; ++j) fa[j] = operand_at<AROWS, BM>(pa, wm * TM + 32 * j, ks, lane);
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = Mma<EL>::go(fb[i], fa[j], acc[i][j]);
    }
    at = at == (NBUF - 1) * kBuf ? 0 : at + kBuf;
  }
  wait_step<0>();  // nothing is under way to LDS, nothing is read from it any more

  // The wave's sums, 16 rows at a time, through LDS of its own: a lane then has
  // eight consecutive outputs of a row, and memory is read and written in whole
  // pieces of rows.  Chunk c of a staged row stands at c ^ (row % chunks), for the
  // banks.  A wave's LDS operations keep their order.
  uint8_t* mine = lds + wv * (16 * TN * 4);
  constexpr int LR = TC / 8, RP = 64 / LR;  // lanes of a row, rows of a pass
  const int fr = lane & 31, fq = lane >> 5;
  const int c8 = lane % LR, n = n0 + wn * TC + 8 * c8;
#pragma unroll
  for (int jh = 0; jh < 2 * FM; ++jh) {
    const int j = jh / 2;
    if (fr / 16 == jh % 2) {
      const int r = fr & 15;
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *(f32x4*)(mine + r * (TN * 4) + (((8 * i + 2 * g + fq) ^ (r & (CH - 1))) << 4)) =
              f32x4{(float)acc[i][j][4 * g], (float)acc[i][j][4 * g + 1], (float)acc[i][j][4 * g + 2],
                    (float)acc[i][j][4 * g + 3]};
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int r0 = 0; r0 < 16; r0 += RP) {
      const int r = r0 + lane / LR, m = m0 + wm * TM + 16 * jh + r;
      float v[8], u[8];
      auto row8 = [&](int c, float (&f)[8]) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4 w = *(const f32x4*)(mine + r * (TN * 4) + (((c + h) ^ (r & (CH - 1))) << 4));
#pragma unroll
          for (int e = 0; e < 4; ++e) f[4 * h + e] = w[e];
        }
      };
      if (r < 16 && m < a.M && n < a.N) {
        row8(2 * c8, v);
        if (G) row8(TC / 4 + 2 * c8, u);
        EP::put(a, m, n, v, u);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Eight values of a row, rounded once, nearest even.
template <int DT>
__device__ __forceinline__ void put8(void* p, size_t at, const float (&v)[8]) {
  if constexpr (DT == MOE_DT_F32) {
    f32x4* q = (f32x4*)((float*)p + at);
    q[0] = f32x4{v[0], v[1], v[2], v[3]};
    q[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    *(u32x4*)((uint16_t*)p + at) = Chunk<DT>::pack(v);
  }
}
template <int DT>
__device__ __forceinline__ void get8(const void* p, size_t at, float (&v)[8]) {
  Chunk<DT>::unpack(*(const u32x4*)((const uint16_t*)p + at), v);
}

}  // namespace moe
