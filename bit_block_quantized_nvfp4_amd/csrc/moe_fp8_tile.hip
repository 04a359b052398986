// e4m3 products of many rows: quantisation of the rows, then tiles of BN
// weight rows x BM token rows, the codes as f16 on the 32x32x16 f16 MFMA, whose
// f32 sums drop nothing of a product (the f8 MFMAs do: moe_fp8.hpp).
//
//   z[t][n] = sum_b s[t][b] S[n / 128][b] sum_{k in block b} q[t][k] W[n][k]
//
// One K step is one block of 128, so a step's products start from zero and are
// scaled into the f32 accumulators: 16 multiply-adds per 8 MFMAs of 32 cycles.
// Weights are the MFMA's A operand: a lane then has one token per tile column,
// hence one scale, and four consecutive outputs at a time.
//
// Both operands go from memory to LDS as codes, without registers (16 bytes a
// lane, the next step's while this one is computed); a wave converts them as it
// reads them.  A row of a step is 128 bytes, its 16-byte chunk c stands at place
// c ^ (row % 8), so that the reads of 8 rows at one chunk meet every bank once;
// the DMA writes lanes in order, hence the permutation is applied to the
// addresses that it reads.
//
// Measured.  Dense, bf16 rows: 8192 x 4096 x 4096 20 us + 255 us (1.08 PFLOP/s), 8192
// x 8192 x 8192 45 us + 960 us (1.15), where a library's bf16 product of that size
// reaches 1.21 and the MFMAs alone, on data of mixed bits, 1.65: bound by the
// matrix unit, with 128 conversions and 64 multiply-adds a wave beside 32 MFMAs.
// Experts (H = 2048, I = 512, top 10 of 512 and a shared one): T = 4096 8 + 341 + 216
// us for 1.35 GB and 0.68 GB from memory (nearly all of it weights that one row
// tile reads) and 283 GFLOP, neither of which alone takes as long; T = 16384 22 +
// 945 + 548 us (1133 GFLOP, the matrix unit).
#include <math.h>

#include <algorithm>

#include "moe_ffn_common.hpp"
#include "moe_fp8.hpp"
#include "moe_internal.hpp"
#include "moe_prefill_items.hpp"

namespace moe {

// Rows whose scales of one block along K stand together where a dense product
// reads them (a multiple of every row tile).
constexpr int kScaleRows = 256;

// One thread per 8 values, 16 lanes to a block of 128.  ldq: bytes of a code
// row (K, or K rounded up to 128 with zeros behind).  Scale of row t and block
// b: place t nb + b; TILED: b + nb (t / 256) runs of 256, in it place t % 256.
template <int DT, bool TILED>
__device__ __forceinline__ void quant_block(unsigned block, const void* __restrict__ x, int T,
                                            int K, int ldq, int lg, int cb,
                                            uint8_t* __restrict__ codes,
                                            float* __restrict__ scales) {
  constexpr int N = Chunk<DT>::N;
  const int nb = (K + kQB - 1) / kQB;
  int t, c;
  if (!row_chunk(block, lg, cb, T, nb * 16, &t, &c)) return;
  const u32x4* p = (const u32x4*)((const char*)x + (size_t)t * K * (DT == MOE_DT_F32 ? 4 : 2));
  float f[8];
  float am = 0.f;
#pragma unroll
  for (int i = 0; i < 8 / N; ++i) {
    u32x4 v = u32x4{0u, 0u, 0u, 0u};
    if (8 * c < K) v = p[c * (8 / N) + i];
    float g[N];
    Chunk<DT>::unpack(v, g);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      f[i * N + j] = g[j];
      am = fmaxf(am, fabsf(g[j]));
    }
  }
  // max over the 16 lanes of the block
  am = fmaxf(am, __int_as_float((int)dpp<0xB1>((uint32_t)__float_as_int(am))));
  am = fmaxf(am, __int_as_float((int)dpp<0x4E>((uint32_t)__float_as_int(am))));
  am = fmaxf(am, __int_as_float((int)dpp<0x141>((uint32_t)__float_as_int(am))));
  am = fmaxf(am, __int_as_float((int)dpp<0x140>((uint32_t)__float_as_int(am))));
  am = q_floor(am);
  const float m = 448.0f / am;
  if (8 * c < ldq)
    *(u32x2*)(codes + (size_t)t * ldq + 8 * c) =
        u32x2{fp8x4(f[0] * m, f[1] * m, f[2] * m, f[3] * m),
              fp8x4(f[4] * m, f[5] * m, f[6] * m, f[7] * m)};
  if ((c & 15) == 0)
    scales[TILED ? ((size_t)(t / kScaleRows) * nb + c / 16) * kScaleRows + t % kScaleRows
                 : (size_t)t * nb + c / 16] = am / 448.0f;
}

template <int DT, bool TILED>
__global__ __launch_bounds__(256) void k_fp8_quant(const void* __restrict__ x, int T, int K,
                                                   int ldq, int lg, int cb,
                                                   uint8_t* __restrict__ codes,
                                                   float* __restrict__ scales) {
  quant_block<DT, TILED>(blockIdx.x, x, T, K, ldq, lg, cb, codes, scales);
}

// The row tiles of the grouped products: items[0] = their number, then from
// items[4] on {group, first row, rows, 1 if the group has no other tile} of
// each.  Groups of several tiles come first, a group's tiles one after the
// other (its weights are then still near when the next tile reads them: T =
// 16384 gate_up 652 us, 3% more with all full tiles first), then the others by
// the number of 32-row parts, so that the short ones fill the launch's end.
// One block of 256 threads.
__device__ __forceinline__ void write_items(const int32_t* __restrict__ offsets, int G,
                                            int32_t* __restrict__ items) {
  __shared__ unsigned long long wsum[4];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int per = (G + 255) / 256;
  const int lo = min(tid * per, G), hi = min(lo + per, G);
  // a group of more than one tile: all of them in class 0
  auto tiles = [](int cnt) { return (cnt + kPM - 1) / kPM; };
  auto cls = [](int cnt) { return cnt > kPM ? 0 : 4 - (cnt + 31) / 32; };
  auto unit = [&](int cnt) { return cnt > 0 ? (unsigned long long)tiles(cnt) * pf_unit(cls(cnt)) : 0ull; };
  unsigned long long local = 0;
  for (int g = lo; g < hi; ++g) local += unit(max(offsets[g + 1] - offsets[g], 0));
  const unsigned long long incl = pf_wave_incl_scan64(local, lane);
  if (lane == 63) wsum[wv] = incl;
  __syncthreads();
  unsigned long long before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    before += (i < wv) ? wsum[i] : 0ull;
    total += wsum[i];
  }
  unsigned long long run = before + incl - local;
  int first[4], n = 0;
  for (int k = 0; k < 4; ++k) {
    first[k] = n;
    n += pf_field(total, k);
  }
  if (tid == 0) items[0] = n;
  i32x4* list = (i32x4*)(items + 4);
  for (int g = lo; g < hi; ++g) {
    const int p0 = offsets[g], cnt = max(offsets[g + 1] - p0, 0);
    if (cnt == 0) continue;
    const int k = cls(cnt), at = first[k] + pf_field(run, k);
    for (int i = 0; i < tiles(cnt); ++i)
      list[at + i] = i32x4{g, p0 + i * kPM, min(kPM, cnt - i * kPM), cnt <= kPM};
    run += unit(cnt);
  }
}

// Quantisation of the experts' token rows (K a multiple of 128) and, in block
// 0, the list of row tiles.
__global__ __launch_bounds__(256) void k_fp8_prep(const uint16_t* __restrict__ x, int T, int K,
                                                  int lg, int cb, uint8_t* __restrict__ codes,
                                                  float* __restrict__ scales,
                                                  const int32_t* __restrict__ offsets, int G,
                                                  int32_t* __restrict__ items) {
  if (blockIdx.x == 0) write_items(offsets, G, items);
  else quant_block<MOE_DT_BF16, false>(blockIdx.x - 1, x, T, K, K, lg, cb, codes, scales);
}

enum { kTileLinear = 0, kTileGateUp = 1, kTileDown = 2 };

struct TileArgs {
  const uint8_t* codes;    // weights [N][K] (of group 0)
  const float* scales;     // [ceil(N/128)][nb]
  const uint8_t* xq;       // token codes [rows][nb * 128]
  const float* xs;         // token scales: linear [row / 256][nb][256], gate_up
                           // [T][nb], down [item][nb][kPM]
  void* out;
  float* out_scales;       // gate_up: scales of h, as down reads them
  const int32_t* items;    // grouped modes: row tiles (write_items)
  const int32_t* sorted_slot;
  int R;                   // rows (linear)
  int N, K, T, topk, has_shared;
  int nt;                  // tiles along N
  int ntb;                 // of them per block (grouped modes), a divisor of nt
};

// Weight scales of a block's steps in LDS, times the scales of a step: K up to
// 65536 for one tile, or ntb runs of 64 (a bank's K is up to 8192, ntb up to 8).
constexpr int kTileScales = 512;
// Blocks that a grouped launch keeps at least when its blocks take several tiles.
constexpr size_t kStreamBlocks = 2048;

// Buffer descriptor of `bytes` bytes at p (both wave-uniform): loads past the
// end return zeros.
__device__ __forceinline__ u32x4 buf_of(const void* p, uint32_t bytes) {
  const uint64_t a = (uint64_t)(uintptr_t)p;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32)) & 0xFFFFu,
               (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00027000u};
}
// Memory to LDS, 16 (4) bytes a lane: lane l's bytes at voff + soff land at
// lds + 16 l (4 l).  No register is written.  In asm because the compiler
// would wait for every such load before the next LDS read of any buffer; the
// kernel's own waits below order them.  m0 is reserved in the compiler (it may
// not be named as overwritten), which keeps nothing in it between instructions;
// that nothing else touches it is tested on the built code.  A memory instruction
// may read it one state after it was written.  ONCE: the bytes are not read again
// (non-temporal).
// A wave-uniform offset for these, in a scalar register that a memory
// instruction may read: one that a vector instruction wrote needs 5 states.
__device__ __forceinline__ uint32_t dma_offset(uint32_t v) {
  uint32_t s = (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
  asm volatile("s_nop 4" : "+s"(s));
  return s;
}
template <bool ONCE = false>
__device__ __forceinline__ void dma_b128(u32x4 buf, uint32_t voff, uint32_t soff, uint32_t lds) {
  if (ONCE)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds" ::"s"(lds),
                 "v"(voff), "s"(buf), "s"(soff)
                 : "memory");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds),
                 "v"(voff), "s"(buf), "s"(soff)
                 : "memory");
}
__device__ __forceinline__ void dma_b32(u32x4 buf, uint32_t voff, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(lds),
               "v"(voff), "s"(buf), "s"(soff)
               : "memory");
}
// All but the wave's last N memory operations are done, and all its LDS reads;
// then the block's waves meet.
template <int N>
__device__ __forceinline__ void wait_step() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The block's waves meet, each with its LDS reads done.
__device__ __forceinline__ void meet() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// A block computes a.ntb tiles of BN weight rows side by side (grouped modes; one
// in the linear mode) for one tile of BM tokens: a stream of ntb * nb steps,
// one block of 128 along K each, through NBUF buffers.  While step s is
// computed, the steps up to s + NBUF are on their way, across the ends of
// tiles, so the output of a tile is written while the next one's operands come.
// KG > 1 (linear mode): KG groups of waves with buffers of their own take every
// KG-th step and join their sums at the end, in the groups' order; a step costs
// about half a microsecond of waiting whatever its size, which counts where
// there are few tiles.  The grouped modes' registers are held to two waves a SIMD:
// down has two blocks on a compute unit so, with six registers spilled once a tile
// (the experts' call at T = 4096 531 us, with one block 585 us).
template <int MODE, int DT, int BN, int BM, int WN, int WM, int NBUF, int KG = 1>
__global__ __launch_bounds__(64 * WN * WM * KG, MODE == kTileLinear ? 1 : 2) void k_fp8_tile(TileArgs a) {
  constexpr int NW = WN * WM, NT = 64 * NW;    // waves and threads of a group
  constexpr int TN = BN / WN, TM = BM / WM;    // a wave's part of the tile
  constexpr int FN = TN / 32, FM = TM / 32;    // products of 32 x 32
  constexpr int DW = BN * 8 / NT, DX = BM * 8 / NT;  // 16-byte chunks per thread and step
  constexpr int D = DW + DX + 1;               // memory operations per wave and step
  constexpr int kTok = BN * kQB, kScale = kTok + BM * kQB;  // LDS offsets in a buffer
  constexpr int BS = (BM + 63) / 64;           // waves that bring a step's token scales
  constexpr int kBuf = kScale + BS * 256;
  constexpr int ES = DT == MOE_DT_F32 ? 4 : 2;
  constexpr int CR = TN * ES / 16;             // 16-byte chunks of a row of the wave's output
  constexpr int NS = (BN + kQB - 1) / kQB;     // weight scales of a step
  constexpr int BC = MODE == kTileGateUp ? BN / 2 : BN;  // columns of a tile
  static_assert(BN * 8 % NT == 0 && BM * 8 % NT == 0 && TN % 32 == 0 && TM % 32 == 0 &&
                    BS <= NW && NBUF * D < 64 && 64 % CR == 0,
                "tile shape");
  static_assert(MODE == kTileLinear || BM == kPM, "row tiles of the items");
  static_assert(MODE != kTileGateUp || (BC == kQB && FN == 2), "a tile holds one scale of h, a wave a gate and an up row");
  static_assert(KG == 1 || (MODE == kTileLinear && (KG - 1) * BN * BM * 4 + NW * 16 * TN * ES <= KG * NBUF * kBuf),
                "the groups' sums fit");
  __shared__ __align__(1024) uint8_t lds_all[KG * NBUF * kBuf];
  __shared__ float wsc[NS * kTileScales];
  __shared__ float nowhere[64];                // for loads that bring nothing: they write zeros
  __shared__ __align__(16) uint8_t side[MODE == kTileGateUp ? WN * BM * 4
                                        : MODE == kTileDown ? NW * 16 * TN * ES : 16];
  const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane((int)threadIdx.x / NT);
  const int tid = (int)threadIdx.x - kg * NT, lane = tid & 63;
  uint8_t* lds = lds_all + kg * (NBUF * kBuf);
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wv % WN, wm = wv / WN;
  const int nb = (a.K + kQB - 1) / kQB;
  const int steps = (nb + KG - 1) / KG;        // of a group and tile
  const int ntb = MODE == kTileLinear ? 1 : a.ntb;

  const uint8_t* codes = a.codes;
  const float* scales = a.scales;
  size_t item_at = 0;                          // the item's scales of h
  int m0, rows, n0;                            // first token row, rows left, first column
  bool single = false;                         // the group has no other row tile
  if (MODE == kTileLinear) {
    // Blocks are dealt to the 8 XCDs in turn: give each XCD a run of tiles, and
    // let a run go 8 token tiles deep before its next weight tile, so that the
    // blocks that run together on one XCD share rows of both operands in its L2
    const int mt = (a.R + BM - 1) / BM, nblk = gridDim.x, per = nblk / 8;
    const int b = blockIdx.x;
    const int lin = b < per * 8 ? (b % 8) * per + b / 8 : b;
    const int deep = 8 * a.nt, grp = lin / deep, in = lin % deep;
    const int gm = min(8, mt - grp * 8);
    m0 = (grp * 8 + in % gm) * BM;
    n0 = (in / gm) * BN;
    rows = a.R - m0;
  } else {
    // the column tiles of two row tiles back to back on one XCD: the tiles of a
    // group of several share its weights in the L2 (the call at T = 16384 1476 us,
    // in runs of one row tile 1490 us; T = 4096 545 and 546 us)
    const int per = a.nt / ntb;
    const int lin = pf_item_of_block(blockIdx.x, gridDim.x, 2 * per), item = lin / per;
    item_at = (size_t)item * ((MODE == kTileGateUp ? a.N : a.K) / kQB) * kPM;
    const int n = a.items[0];
    const i32x4 e = ((const i32x4*)(a.items + 4))[item];
    if (item >= n) return;
    const int nr = MODE == kTileGateUp ? 2 * a.N : a.N;
    codes += (size_t)e.x * nr * a.K;
    scales += (size_t)e.x * (nr / kQB) * nb;
    m0 = e.y;
    rows = e.z;
    single = __builtin_amdgcn_readfirstlane(e.w) != 0;
    n0 = (lin % per) * ntb * BC;
  }
  m0 = __builtin_amdgcn_readfirstlane(m0);
  n0 = __builtin_amdgcn_readfirstlane(n0);
  rows = __builtin_amdgcn_readfirstlane(min(rows, BM));

  // Weight row (from the buffer's base) of LDS row lr.  gate_up: each wave's TN
  // rows are TN / 2 gate rows and the up rows of the same columns.
  auto wrow_of = [&](int lr) __attribute__((always_inline)) {
    if (MODE == kTileGateUp) {
      const int w = lr / TN, q = lr % TN;
      return n0 + w * (TN / 2) + q % (TN / 2) + (q < TN / 2 ? 0 : a.N);
    }
    return min(lr, a.N - 1 - n0);
  };
  // Row of the token buffer of the tile's row r; past the tile's rows one
  // behind the buffer's end, for which nothing is read.
  auto xrow_of = [&](int r) __attribute__((always_inline)) {
    if (MODE != kTileGateUp) return r;
    if (r >= rows) return a.T;
    return max(slot_token(a.sorted_slot[m0 + r], a.T, a.topk, a.has_shared), 0);
  };
  const uint32_t ldx = (uint32_t)nb * kQB;
  const u32x4 wbuf = MODE == kTileGateUp
                   ? buf_of(codes, (uint32_t)(2 * a.N) * (uint32_t)a.K)
                   : buf_of(codes + (size_t)n0 * a.K,
                            (uint32_t)min(BN * ntb, a.N - n0) * (uint32_t)a.K);
  const u32x4 xbuf = MODE == kTileGateUp ? buf_of(a.xq, (uint32_t)a.T * ldx)
                                   : buf_of(a.xq + (size_t)m0 * ldx, (uint32_t)rows * ldx);
  // Token scales: 64 rows of a step are one load of a wave, 256 bytes in one
  // piece where the row tile is known when they are written: scattered ones take
  // a lookup each, 64 of them as many as 8 KB of codes (with tiles of 256 x 256
  // and products of half the time, 8192 x 8192 x 8192 took 538 us with all eight
  // waves bringing 64 scattered scales, 513 us with the four that have to, 492 us so).
  constexpr int SR = MODE == kTileLinear ? kScaleRows : MODE == kTileDown ? kPM : 1;
  const u32x4 sbuf = MODE == kTileGateUp ? buf_of(a.xs, (uint32_t)a.T * (uint32_t)nb * 4u)
                   : MODE == kTileDown   ? buf_of(a.xs + item_at, (uint32_t)(nb * SR) * 4u)
                   : buf_of(a.xs + (size_t)(m0 / SR) * nb * SR + m0 % SR,
                            (uint32_t)(nb * SR - m0 % SR) * 4u);
  // Chunk i of this thread: LDS row lr, place tid % 8; rows of one thread are
  // NT / 8 apart, a multiple of 8, so its chunk of the row is always the same.
  const int chunk = 16 * ((tid & 7) ^ ((tid >> 3) & 7));
  uint32_t woff[DW], xoff[DX];
#pragma unroll
  for (int i = 0; i < DW; ++i)
    woff[i] = (uint32_t)wrow_of((i * NT + tid) >> 3) * (uint32_t)a.K + chunk;
#pragma unroll
  for (int i = 0; i < DX; ++i) xoff[i] = (uint32_t)xrow_of((i * NT + tid) >> 3) * ldx + chunk;
  // the first waves bring 64 token scales each, the others none
  const bool brings = wv < BS;
  const int srow = 64 * (wv % BS) + lane;
  const uint32_t soff = MODE == kTileGateUp ? (uint32_t)xrow_of(srow) * (uint32_t)nb * 4u : srow * 4u;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  const uint32_t ldsw = lds0 + wv * 1024;
  const uint32_t ldsn = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) float*)nowhere;

  // The weight scales of all steps, one per 128 weight rows of a tile (gate_up:
  // the gate's, then the up's), first to LDS: a load of one in the loop would
  // wait for the DMA under way, and loads through registers here for memory
  // before it begins.
  const int nbp = (nb + 63) & ~63;             // a run of them, zeros behind
  const uint32_t ldsc = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) float*)wsc;
  for (int i = kg * NW + wv; i < ntb * NS * (nbp / 64); i += NW * KG) {
    const int run = i / (nbp / 64), part = i % (nbp / 64);
    const int tile = run / NS, h = run % NS;
    const int row = n0 + tile * BC + (MODE == kTileGateUp ? h * a.N : h * kQB);
    const int band = (MODE == kTileGateUp ? row : min(row, a.N - 1)) / kQB;
    u32x4 run_buf = buf_of(scales + (size_t)band * nb, (uint32_t)nb * 4u);
    asm volatile("s_nop 4" : "+s"(run_buf));   // as in dma_offset
    dma_b32(run_buf, lane * 4, dma_offset(part * 256), ldsc + i * 256);
  }

  // The next step to bring: how many are left, its block along K and buffer.
  // Tokens (with their scales) and weights of a step are asked for at different
  // times, tokens first.  Past the last step the buffers are empty ones, at
  // offset 0 (the range check subtracts the scalar offset from the size), and
  // zeros come, to where nobody reads: every wave then has the same number of
  // operations under way at every wait, and the loop has no branch, behind
  // which the compiler would move the sums of half a step and spill.
  int d_left = KG == 1 ? ntb * nb : (nb - kg + KG - 1) / KG, d_k = kg, d_at = 0;
  uint32_t d_col = 0;                          // offset of the tile's weights
  auto dma_tokens = [&]() __attribute__((always_inline)) {
    u32x4 xb = xbuf, sb = sbuf;
    xb.z = d_left > 0 ? xb.z : 0u;
    sb.z = d_left > 0 && brings ? sb.z : 0u;
    const uint32_t k = d_left > 0 ? (uint32_t)d_k : 0u;
    const uint32_t kx = dma_offset(k * kQB), ks = dma_offset(brings ? k * (SR * 4) : 0u);
#pragma unroll
    for (int i = 0; i < DX; ++i)
      dma_b128(xb, xoff[i], kx, ldsw + d_at + kTok + i * NT * 16);
    dma_b32(sb, soff, ks, brings ? lds0 + d_at + kScale + 256 * wv : ldsn);
  };
  auto dma_weights = [&](auto once) __attribute__((always_inline)) {
    u32x4 wb = wbuf;
    wb.z = d_left > 0 ? wb.z : 0u;
    const uint32_t k = (uint32_t)d_k * kQB;
    // a chunk past the end of a weight row is read from the start of the block
    // instead: the tokens' codes there are zeros
    const uint32_t back = MODE == kTileLinear && (int)k + chunk >= a.K ? (uint32_t)chunk : 0u;
    const uint32_t so = dma_offset(d_left <= 0 ? 0u : MODE == kTileLinear ? k : k + d_col);
#pragma unroll
    for (int i = 0; i < DW; ++i) dma_b128<decltype(once)::value>(wb, woff[i] - back, so, ldsw + d_at + i * NT * 16);
    --d_left;
    d_at = d_at == (NBUF - 1) * kBuf ? 0 : d_at + kBuf;
    d_k += KG;
    if (MODE != kTileLinear) {
      d_col += d_k == nb ? (uint32_t)BC * (uint32_t)a.K : 0u;
      d_k = d_k == nb ? 0 : d_k;
    }
  };
#pragma unroll
  for (int b = 0; b < NBUF; ++b) {
    dma_tokens();
    dma_weights(std::false_type{});
  }

  // rows of this lane's stores that belong to a slot, a bit each
  uint32_t mine_ok = ~0u;
  if (MODE == kTileDown) {
    mine_ok = 0;
#pragma unroll
    for (int i = 0; i < TM * CR / 64; ++i) {
      const int row = wm * TM + i * (64 / CR) + lane / CR;
      if (row < rows && slot_token(a.sorted_slot[m0 + row], a.T, a.topk, a.has_shared) >= 0)
        mine_ok |= 1u << i;
    }
  }

  f32x16 acc[FN][FM];
  // columns of 32 tokens of this wave with rows in them
  const int live = min(FM, max(0, (rows - wm * TM + 31) / 32));
  const int hs = MODE == kTileGateUp ? 0 : wn * TN / kQB;

  // this lane's four chunks of row 32 i + lane % 32
  const int fr = lane & 31, fq = lane >> 5;
  struct Codes {
    u32x4 c[4];
  };
  auto codes_at = [&](const uint8_t* p, int row32) __attribute__((always_inline)) {
    Codes r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r.c[i] = *(const u32x4*)(p + (row32 + fr) * kQB + (((fq + 2 * i) ^ (fr & 7)) << 4));
    return r;
  };
  // The next step's first operands, read while the last products of a step run.
  Codes wnx, tnx;
  auto first = [&](int at, auto count) __attribute__((always_inline)) {
    if (decltype(count)::value == 0) return;
    wnx = codes_at(lds + at + wn * TN * kQB, 0);
    tnx = codes_at(lds + at + kTok + wm * TM * kQB, 0);
  };
  // Step at buffer `at`, whose weight scales are sc[0] and (gate_up: the up
  // rows') sc[nbp].  One barrier, behind the products of the first weight rows:
  // every wave has then read all its operands, so the buffer may be filled again,
  // and the step after has landed (what was asked for later may be under way), so
  // its first operands are read while the last products run.
  auto step = [&](int at, const float* sc, bool some, auto last, auto count, auto once) __attribute__((always_inline)) {
    constexpr int LV = decltype(count)::value;
    constexpr bool kLast = decltype(last)::value;
    const uint8_t* pw = lds + at + wn * TN * kQB;
    const uint8_t* pt = lds + at + kTok + wm * TM * kQB;
    const float* ps = (const float*)(lds + at + kScale) + wm * TM + fr;
    const int next = at == (NBUF - 1) * kBuf ? 0 : at + kBuf;
    Frag<32> wf, tf[FM];
    float s0[FM], s1[FM];
    // a group's step past the end adds zeros
    const float w0 = KG == 1 || some ? sc[0] : 0.f, w1 = MODE == kTileGateUp ? sc[nbp] : 0.f;
    Codes wc, tc;
    if (LV > 0) {
      wf.set(wnx.c);
      tf[0].set(tnx.c);
    }
    if (LV > 1) tc = codes_at(pt, 32);
    if (LV > 0 && FN > 1) wc = codes_at(pw, 32);
#pragma unroll
    for (int j = 0; j < LV; ++j) {
      const float sx = ps[32 * j];
      s0[j] = sx * w0;
      s1[j] = MODE == kTileGateUp ? sx * w1 : s0[j];
    }
    // a product runs while the one before is scaled into the sums
    f32x16 p[2];
    auto add = [&](int b) __attribute__((always_inline)) {
      const int i = b / (LV > 0 ? LV : 1), j = b % (LV > 0 ? LV : 1);
      const float s = i == 0 ? s0[j] : s1[j];
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = fmaf(s, p[b & 1][e], acc[i][j][e]);
    };
#pragma unroll
    for (int i = 0; i < FN; ++i) {
      if (LV > 0 && i > 0) wf.set(wc.c);
#pragma unroll
      for (int j = 0; j < LV; ++j) {
        if (i == 0 && j > 0) tf[j].set(tc.c);
        const int b = i * LV + j;
        p[b & 1] = mfma128(wf, tf[j]);
        if (b > 0) add(b - 1);
      }
      if (i == 0 && !kLast) {
        __builtin_amdgcn_sched_barrier(0);
        wait_step<(NBUF - 2) * D>();
        dma_tokens();
        dma_weights(once);
        first(next, count);
      }
    }
    if constexpr (LV > 0) add(FN * LV - 1);
  };

  // gate_up: h = silu(gate) up in f32, its absmax over the tile's 128 columns
  // (one scale of h), then its codes.  n: the tile's first column.
  auto put_h = [&](int n, auto count) __attribute__((always_inline)) {
    constexpr int LV = decltype(count)::value;
    float* amax = (float*)side;                // [WN][BM]
#pragma unroll
    for (int j = 0; j < LV; ++j) {
      float am = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float h = silu_f32(acc[0][j][e]) * acc[FN - 1][j][e];
        acc[0][j][e] = h;
        am = fmaxf(am, fabsf(h));
      }
      am = fmaxf(am, __shfl_xor(am, 32));
      if (fq == 0) amax[wn * BM + wm * TM + 32 * j + fr] = am;
    }
    meet();
#pragma unroll
    for (int j = 0; j < LV; ++j) {
      const int r = wm * TM + 32 * j + fr;
      float am = amax[r];
#pragma unroll
      for (int w = 1; w < WN; ++w) am = fmaxf(am, amax[w * BM + r]);
      am = q_floor(am);
      const float m = 448.0f / am;
      if (r < rows) {
        uint8_t* dst = (uint8_t*)a.out + (size_t)(m0 + r) * a.N + n + wn * (TN / 2);
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *(uint32_t*)(dst + 8 * g + 4 * fq) =
              fp8x4(acc[0][j][4 * g] * m, acc[0][j][4 * g + 1] * m, acc[0][j][4 * g + 2] * m,
                    acc[0][j][4 * g + 3] * m);
        if (wn == 0 && fq == 0)
          a.out_scales[item_at + (size_t)(n / kQB) * kPM + r] = am / 448.0f;
      }
    }
  };
  // The wave's part of the output, rounded, 16 tokens at a time through LDS of
  // its own: a lane has 4 columns of a token, the stores are whole rows of the
  // part (16 bytes a lane).  The 16-byte chunk c of a row stands at
  // c ^ (row % chunks), for the banks.  A wave's LDS operations keep their order.
  auto put_out = [&](int n, auto count) __attribute__((always_inline)) {
    constexpr int LV = decltype(count)::value;
    uint8_t* mine = (MODE == kTileDown ? side : lds) + (KG > 1 ? (KG - 1) * BN * BM * 4 : 0) + wv * (16 * TN * ES);
    const int c = lane % CR, nc = n + wn * TN + c * (16 / ES);
#pragma unroll
    for (int jh = 0; jh < 2 * LV; ++jh) {
      const int j = jh / 2;
      if (fr / 16 == jh % 2) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int at = (32 * i + 8 * g + 4 * fq) * ES;
            uint8_t* dst = mine + (fr & 15) * (TN * ES) + (((at / 16) ^ (fr & (CR - 1))) << 4) + (at & 15);
            const f32x4 v = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
            if (DT == MOE_DT_F32)
              *(f32x4*)dst = v;
            else if (DT == MOE_DT_BF16)
              *(u32x2*)dst = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            else
              *(u32x2*)dst = u32x2{pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3])};
          }
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int r0 = 0; r0 < 16; r0 += 64 / CR) {
        const int r = r0 + lane / CR, row = wm * TM + 16 * jh + r;
        const bool on = MODE == kTileDown ? (mine_ok >> ((16 * jh + r0) * CR / 64) & 1) : row < rows;
        const u32x4 v = *(const u32x4*)(mine + r * (TN * ES) + ((c ^ (r & (CR - 1))) << 4));
        if (on && nc < a.N && r < 16)
          *(u32x4*)((uint8_t*)a.out + ((size_t)(m0 + row) * a.N + nc) * ES) = v;
      }
      __builtin_amdgcn_wave_barrier();
    }
  };

  wait_step<(NBUF - 1) * D>();
  auto run = [&](auto count, auto once) __attribute__((always_inline)) {
    int at = 0;
    auto on = [&]() __attribute__((always_inline)) { at = at == (NBUF - 1) * kBuf ? 0 : at + kBuf; };
    first(0, count);
    for (int tile = 0; tile < ntb; ++tile) {
      const float* sc = wsc + (tile * NS + hs) * nbp;
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = f32x16{};
      const float* end = sc + nb;
      sc += kg;
      // grouped modes: the last step of the last tile asks for operands too, and
      // gets zeros (a branch there would double the step, and spill)
      for (int b = MODE == kTileLinear; b < steps; ++b, sc += KG, on())
        step(at, sc, true, std::false_type{}, count, once);
      if (MODE == kTileLinear) step(at, sc, sc < end, std::true_type{}, count, once);
      if (MODE == kTileLinear || tile + 1 == ntb) wait_step<0>();  // nothing is under way to LDS any more
      if (KG > 1) {
        // lane by lane, 16 bytes at a time
        f32x4* mine = (f32x4*)lds_all + tid;
        if (kg > 0) {
#pragma unroll
          for (int i = 0; i < FN * FM; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const f32x16& v = acc[i / FM][i % FM];
              mine[(((kg - 1) * FN * FM + i) * 4 + g) * NT] = f32x4{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
            }
        }
        meet();
        if (kg > 0) return;
#pragma unroll
        for (int o = 0; o < KG - 1; ++o)
#pragma unroll
          for (int i = 0; i < FN * FM; ++i)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const f32x4 v = mine[((o * FN * FM + i) * 4 + g) * NT];
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i / FM][i % FM][4 * g + e] += v[e];
            }
      }
      if (MODE == kTileGateUp) put_h(n0 + tile * BC, count);
      else put_out(n0 + tile * BC, count);
    }
  };
  // A wave computes only its columns of 32 tokens with rows in them, in a loop
  // made for their number: a test at each product would break up the schedule.
  // Every such loop has the same barriers.  The weights of a group with one row
  // tile are read once (the call at T = 512 takes 270 us, with ordinary loads 286
  // us; at T = 1024 311 and 320 us).
  if constexpr (MODE == kTileLinear) {
    run(IntC<FM>{}, std::false_type{});
  } else {
    static_assert(FM == 2, "the loops below");
    auto by_live = [&](auto once) __attribute__((always_inline)) {
      if (live == 2) run(IntC<2>{}, once);
      else if (live == 1) run(IntC<1>{}, once);
      else run(IntC<0>{}, once);
    };
    if (single) by_live(std::true_type{});
    else by_live(std::false_type{});
  }
}

// The linear mode's tiles, largest first: f with the kernel, BN, BM and threads.
constexpr int kTileShapes = 6;
template <int DT, typename F>
static void by_linear_tile(int shape, F&& f) {
  if (shape == 0) f(&k_fp8_tile<kTileLinear, DT, 256, 128, 4, 2, 3>, 256, 128, 512);
  if (shape == 1) f(&k_fp8_tile<kTileLinear, DT, 128, 128, 2, 2, 2, 2>, 128, 128, 512);
  if (shape == 2) f(&k_fp8_tile<kTileLinear, DT, 128, 64, 2, 2, 3, 2>, 128, 64, 512);
  if (shape == 3) f(&k_fp8_tile<kTileLinear, DT, 64, 64, 2, 2, 4, 2>, 64, 64, 512);
  if (shape == 4) f(&k_fp8_tile<kTileLinear, DT, 32, 64, 1, 2, 3, 4>, 32, 64, 512);
  if (shape == 5) f(&k_fp8_tile<kTileLinear, DT, 32, 32, 1, 1, 4, 4>, 32, 32, 256);
}

// The shape whose rounds of 256 blocks (a block's LDS leaves a compute unit no
// second one) take the least time together; a round's relative time hardly
// depends on how full it is.  The whole call with each shape (us, in a row in a
// graph; * the one taken):
//   rows x N x K, bf16    256x128  128x128  128x64  64x64  32x64  32x32
//   8192 x 4096 x 4096       269*     294     355    447    571    891
//   8192 x 8192 x 8192      1028*    1054    1306   1635   1977   2903
//   2600 x 4096 x 4096       117      105*    130    158    191    288
//   2048 x 4096 x 4096        70*      74      91    118    149    228
//   1024 x 4096 x 4096        59       40*     48     63     78    117
//   640 x 4096 x 4096         58       35*     45     47     50     74
//   512 x 4096 x 4096         57       35      27*    34     41     61
//   333 x 4168 x 2064         34       23      18*    22     30     36
//   512 x 2048 x 2048         32       21      16     13*    16     23
//   256 x 4096 x 4096         55       32      24     19*    22     32
//   128 x 4096 x 4096         54       32      23     18     13*    18
//   64 x 4096 x 4096          53       31      23     17     12     11*
//   32 x 8192 x 8192         100       55      39     28     20     17*
// f32 rows take up to a tenth longer with the larger tiles, in the same order.
template <int DT>
static int linear_tile(int T, int N) {
  int best = 0;
  long least = 0;
  for (int s = 0; s < kTileShapes; ++s)
    by_linear_tile<DT>(s, [&](auto, int bn, int bm, int) {
      constexpr int cost[kTileShapes] = {58, 34, 24, 16, 11, 8};
      const long tiles = (long)((N + bn - 1) / bn) * ((T + bm - 1) / bm);
      const long t = (tiles + 255) / 256 * cost[s];
      if (least == 0 || t < least) least = t, best = s;
    });
  return best;
}

void register_fp8_tile_kernels(std::vector<const void*>& k) {
  auto add = [&](auto D) {
    constexpr int DT = decltype(D)::value;
    k.push_back((const void*)&k_fp8_quant<DT, false>);
    k.push_back((const void*)&k_fp8_quant<DT, true>);
    for (int s = 0; s < kTileShapes; ++s)
      by_linear_tile<DT>(s, [&](auto kernel, int, int, int) { k.push_back((const void*)kernel); });
  };
  for (int dt = MOE_DT_BF16; dt <= MOE_DT_F32; ++dt) by_dtype(dt, add);
  k.push_back((const void*)&k_fp8_prep);
  k.push_back((const void*)&k_fp8_tile<kTileGateUp, MOE_DT_BF16, 256, 128, 4, 2, 3>);
  k.push_back((const void*)&k_fp8_tile<kTileDown, MOE_DT_BF16, 128, 128, 2, 2, 2>);
}

template <bool TILED>
static hipError_t quantise(const void* x, int T, int K, int dtype, int ldq, uint8_t* codes,
                           float* scales, hipStream_t s) {
  const RowGrid g = row_grid(T, (K + kQB - 1) / kQB * 16);
  by_dtype(dtype, [&](auto D) {
    MOE_LAUNCH("fp8_quant", s, (k_fp8_quant<decltype(D)::value, TILED>), dim3(g.blocks), dim3(256), 0, s, x,
               T, K, ldq, g.lg, g.cb, codes, scales);
  });
  return hipGetLastError();
}

hipError_t launch_fp8_quant(const void* x, int T, int K, int dtype, uint8_t* codes, float* scales,
                            hipStream_t s) {
  return quantise<false>(x, T, K, dtype, K, codes, scales, s);
}

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
static int blocks_of(int K) { return (K + kQB - 1) / kQB; }

// Up to 16 rows stream the weights in one launch; but where both N and K are
// large the tiles' longer runs of loads are worth the launch of their quantisation
// (both in a row in a graph, us, streamed against tiles: 1 row of 4096 x 4096 6.5
// against 9.5, 16 rows 8.5 against 9.9; 1 row of 4096 x 8192 10.6 against 14.4, 16
// rows 14.2 against 14.7; 1 row of 65536 x 512 8.3 against 12.6, 16 rows 11.1
// against 13.6; 16 rows of 2048 x 8192 13.5 against 14.2; 16 rows of 6144 x 4096
// 13.3 against 9.9, 1 row of 8192 x 8192 18.3 against 15.9, of 8192 x 4096 9.2
// against 10.1).
static bool fp8_linear_streams(int T, int N, int K) {
  if (T > 16) return false;
  return N <= 4096 || K < 2048 || (long)N * K < 3L << 23;
}

uint64_t fp8_quant_threads(int T, int K) { return row_grid_threads(T, blocks_of(K) * 16); }

uint64_t fp8_linear_threads(int T, int N, int K) {
  if (fp8_linear_streams(T, N, K)) return 0;  // at most 65536 / 16 blocks
  uint64_t t = fp8_quant_threads(T, K);
  by_linear_tile<MOE_DT_BF16>(linear_tile<MOE_DT_BF16>(T, N), [&](auto, int bn, int bm, int threads) {
    t = std::max(t, (uint64_t)((N + bn - 1) / bn) * ((T + bm - 1) / bm) * threads);
  });
  return t;
}

size_t fp8_linear_workspace_bytes(int T, int N, int K) {
  if (fp8_linear_streams(T, N, K)) return 0;
  return up256((size_t)T * blocks_of(K) * kQB) +
         ((size_t)T + kScaleRows - 1) / kScaleRows * kScaleRows * blocks_of(K) * sizeof(float);
}

hipError_t launch_fp8_linear(const moe_fp8_matrix& M, const void* x, int T, int dtype, void* out,
                             void* ws, hipStream_t s) {
  if (fp8_linear_streams(T, M.N, M.K)) return launch_fp8_stream_linear(M, x, T, dtype, out, s);
  const int nb = blocks_of(M.K);
  uint8_t* xq = (uint8_t*)ws;
  float* xs = (float*)(xq + up256((size_t)T * nb * kQB));
  hipError_t e = quantise<true>(x, T, M.K, dtype, nb * kQB, xq, xs, s);
  if (e != hipSuccess) return e;
  TileArgs a{};
  a.codes = M.codes;
  a.scales = M.scales;
  a.xq = xq;
  a.xs = xs;
  a.out = out;
  a.R = T;
  a.N = M.N;
  a.K = M.K;
  by_dtype(dtype, [&](auto D) {
    by_linear_tile<decltype(D)::value>(linear_tile<decltype(D)::value>(T, M.N), [&](auto kernel, int bn, int bm, int threads) {
      a.nt = (M.N + bn - 1) / bn;
      MOE_LAUNCH("fp8_tile", s, kernel, dim3((unsigned)a.nt * (unsigned)((T + bm - 1) / bm)),
                 dim3(threads), 0, s, a);
    });
  });
  return hipGetLastError();
}

// Row tiles of S rows in G groups, at most: the full ones and a partial one per
// group, none without a row.
static size_t max_tiles(size_t S, int G) { return std::min(S, S / kPM + (size_t)G); }

// Column tiles that one block takes in a row: a longer stream hides more of a
// block's start and of its outputs, as long as there are blocks enough to share
// the chip out evenly.
static int tiles_per_block(size_t S, int G, int nt) {
  const size_t tiles = (S < (size_t)G ? S : (size_t)G) + S / kPM;
  int n = 1;
  while (n < 8 && nt % (2 * n) == 0 && tiles * (size_t)(nt / (2 * n)) >= kStreamBlocks) n *= 2;
  return n;
}

// Few tokens stream the experts' weights (16 rows of a group are one pass): the
// layer's own switch, and a few more where the matrices are small and a group's
// start counts.  Streams against tiles, us, the same routing (bf16, a shared
// expert): H = 2048, I = 512, top 10 of 512, T = 8 49 and 66, 10 58 and 70, 12 67
// and 73, 13 79 and 80, 16 87 and 84; H = 1024, I = 256, T = 8 20 and 25, 12 23 and
// 28; H = 2048, I = 1408, top 6 of 64, T = 8 83 and 88, 12 73 and 75; H = 2048, I =
// 1024, top 8 of 256, T = 4 43 and 43, 8 77 and 72, 10 89 and 77; H = 4096, I =
// 1536, top 8 of 128, T = 1 43 and 54, 4 126 and 115, 8 206 and 204, 12 248 and 220.
static bool fp8_experts_stream(int T, int H, int I) {
  return T <= kDecodeMaxT || (T <= 12 && (long)H * I <= 1L << 20);
}

size_t fp8_expert_ffn_workspace_bytes(int T, int K, int H, int I, int has_shared) {
  const size_t S = (size_t)T * K + (has_shared ? T : 0);
  if (fp8_experts_stream(T, H, I)) return up256(S * I * sizeof(float));
  const size_t tiles = max_tiles(S, kPMaxG);
  return up256((size_t)T * H) + up256((size_t)T * (H / kQB) * sizeof(float)) + up256(S * I) +
         up256(tiles * (I / kQB) * kPM * sizeof(float)) + 16 * (tiles + 1);
}

uint64_t fp8_expert_ffn_threads(const moe_fp8_weights& W, int T, int K) {
  if (fp8_experts_stream(T, W.H, W.I)) return 0;  // at most 12 * 32 + 1 groups
  const size_t S = (size_t)T * K + (W.has_shared ? T : 0), mt = max_tiles(S, W.E + W.has_shared);
  const int ngu = W.I / 128, ndn = W.H / 128, G = W.E + W.has_shared;
  return std::max({(uint64_t)mt * (ngu / tiles_per_block(S, G, ngu)) * 512,
                   (uint64_t)mt * (ndn / tiles_per_block(S, G, ndn)) * 256,
                   row_grid_threads(T, W.H / kQB * 16) + 256});
}

hipError_t launch_fp8_expert_ffn(const moe_fp8_weights& W, const uint16_t* x, int T, int K,
                                 const int32_t* offsets, const int32_t* sorted_slot,
                                 const int32_t* groups, uint16_t* y, void* ws, hipStream_t s) {
  if (fp8_experts_stream(T, W.H, W.I))
    return launch_fp8_stream_experts(W, x, T, K, offsets, sorted_slot, groups, (float*)ws, y, s);
  const size_t S = (size_t)T * K + (W.has_shared ? T : 0);
  const int G = W.E + W.has_shared;
  uint8_t* xq = (uint8_t*)ws;
  float* xs = (float*)(xq + up256((size_t)T * W.H));
  uint8_t* hq = (uint8_t*)xs + up256((size_t)T * (W.H / kQB) * sizeof(float));
  float* hs = (float*)(hq + up256(S * W.I));
  int32_t* items = (int32_t*)((uint8_t*)hs + up256(max_tiles(S, G) * (W.I / kQB) * kPM * sizeof(float)));
  const RowGrid g = row_grid(T, W.H / kQB * 16);
  MOE_LAUNCH("fp8_prep", s, k_fp8_prep, dim3(g.blocks + 1), dim3(256), 0, s, x, T, W.H, g.lg, g.cb,
             xq, xs, offsets, G, items);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  TileArgs a{};
  a.items = items;
  a.sorted_slot = sorted_slot;
  a.T = T;
  a.topk = K;
  a.has_shared = W.has_shared;
  const unsigned mt = (unsigned)max_tiles(S, G);
  a.codes = W.gu_codes;
  a.scales = W.gu_scales;
  a.xq = xq;
  a.xs = xs;
  a.out = hq;
  a.out_scales = hs;
  a.N = W.I;
  a.K = W.H;
  a.nt = W.I / 128;
  a.ntb = tiles_per_block(S, G, a.nt);
  MOE_LAUNCH("fp8_tile_gate_up", s, (k_fp8_tile<kTileGateUp, MOE_DT_BF16, 256, 128, 4, 2, 3>),
             dim3(mt * (a.nt / a.ntb)), dim3(512), 0, s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.codes = W.dn_codes;
  a.scales = W.dn_scales;
  a.xq = hq;
  a.xs = hs;
  a.out = y;
  a.out_scales = nullptr;
  a.N = W.H;
  a.K = W.I;
  a.nt = W.H / 128;
  a.ntb = tiles_per_block(S, G, a.nt);
  MOE_LAUNCH("fp8_tile_down", s, (k_fp8_tile<kTileDown, MOE_DT_BF16, 128, 128, 2, 2, 2>),
             dim3(mt * (a.nt / a.ntb)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
