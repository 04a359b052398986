// Product of few rows (up to 16) with 16-bit or 8-bit integer weights that stream once
// from memory to registers,
//
//   z[m][n] = sum_k x[m][k] W[n][k],   out = epilogue(z),
//
// bound by the bytes of W.  A wave owns RT tiles of 16 weight rows (gated: a gate tile and
// the up tile of the same outputs) and every KW-th piece of 128 bytes along K; it asks for U
// pieces of each before it multiplies the U before.  It does not multiply beside them: loads
// complete in order, and those of x's operand come behind them, so that its wait for the one
// is a wait for the others; what hides the latency is the other waves.  The KW waves of a
// tile join through LDS in wave order.  16 rows are one MFMA operand whatever their number.
//
// HALF, for up to 8 rows: a tile is 8 weight rows, the operands' upper halves are the same
// rows at the next piece, and the product's two diagonal quarters are added in the end.
// Twice the blocks, for matrices whose tiles of 16 would leave compute units idle.
//
// 8-bit integers: with XDT a row type the rows are quantised on the way.  Each block then
// reads all rows once for their largest magnitudes, behind the first pieces of the weights,
// and again for their codes, which saves a launch where they are few (moe_int8.hip);
// otherwise x holds codes and sm their scales.
#pragma once

#include "moe_int8.hpp"
#include "moe_tile.hpp"

namespace moe {

constexpr int kStreamRows = 16;
// Outputs up to which up to 8 rows take HALF: tiles of 16 leave half the compute units
// idle there, or (gated, two tiles a wave) with too few waves.  bf16, weights from memory,
// in a row in a graph, us, tiles of 16 and HALF:
//   plain, N x K     256 x 512        2.8   2.4                  gated, N outputs, K = 2048
//   2048 x 512       3.3   2.8                                  512     6.4   4.5
//   2048 x 2048      4.9   4.3                                  2048    7.7   5.8
//   2048 x 8192     13.0   9.7                                  4096   11.2   8.4
//   4096 x 2048      5.6   5.5  (8 rows 6.3, 6.8)
// 8-bit integers in the same way, each with a launch of about 2 us for the rows' codes:
//   1024 x 512       4.9   4.9  (8 rows 5.3, 5.5)               1024    6.9   7.0
//   1024 x 2048      6.5   5.9                                  2048    7.5   7.5
//   2048 x 2048      6.6   6.0  (8 rows 7.3, 6.5)               4096    8.3   9.5
//   2048 x 8192     11.8  10.3  (8 rows 13.1, 12.0)             4096, K = 8192  20.9  18.0
//   4096 x 2048      7.2   7.3  (8 rows 8.0, 8.3)               8192   11.4  14.5
// where gated HALF wins for long K alone (2048 outputs, K = 8192: 17.0 and 13.3).
constexpr bool takes_half(int rows, int outputs, bool gated) { return rows <= 8 && outputs <= (gated ? 4096 : 2048); }

// One product of 128 bytes along K: lane l holds chunks l / 16 and l / 16 + 4 of row l % 16,
// so that a load of a wave takes whole halves of 16 lines.  Element e of lane l of the
// result: row 4 (l / 16) + e of a, row l % 16 of b.
template <int EL>
struct Mma16 {
  typedef f32x4 Acc;
  static __device__ __forceinline__ Acc go(u32x4 a, u32x4 b, Acc c) {
    if constexpr (EL == MOE_DT_BF16)
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                     __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                    __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
template <>
struct Mma16<kElI8> {
  typedef i32x4 Acc;
  static __device__ __forceinline__ Acc go(u32x4 a, u32x4 b, Acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a),
                                                 __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
  }
};

constexpr int kXOperand = -1;  // XDT: x holds operands already

// EP as in moe_tile.hpp, with four outputs of a row at a time.
template <int EL, int XDT, class EP, int RT, int KW, int U, bool HALF = false>
__global__ __launch_bounds__(64 * KW) void k_stream(TileArgs16 a) {
  constexpr bool G = EP::kGated;
  constexpr int ES = EL == kElI8 ? 1 : 2;
  constexpr int OT = G ? 1 : RT;             // tiles of outputs of a block
  constexpr int TR = HALF ? 8 : 16, PB = HALF ? 256 : 128;  // a tile's rows; bytes of a piece (HALF: two)
  typedef typename Mma16<EL>::Acc Acc;
  static_assert(!G || RT == 2, "a gate tile and an up tile");
  __shared__ f32x4 red[KW][RT][64];
  __shared__ float amax[XDT == kXOperand ? 1 : KW][kStreamRows];
  const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, q = lane >> 4;
  const int kw = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = (int)blockIdx.x * OT * TR;
  const uint32_t kb = (uint32_t)a.K * ES;
  const int pieces = (int)((kb + PB - 1) / PB);

  const char* wrow[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
    wrow[i] = (const char*)a.b + (size_t)(min(n0 + (G ? 0 : TR * i) + r % TR, a.N - 1) + (G ? i * a.N : 0)) * kb;
  const int xr = min(r % TR, a.M - 1);       // rows past the last are not stored

  // A lane's chunk h of piece p, zeros past the row's end (nothing is read there).
  auto byte_of = [&](int p, int h) __attribute__((always_inline)) {
    return (uint32_t)(p * PB + r / TR * 128 + h * 64 + q * 16);
  };
  auto in = [&](int p, int h) __attribute__((always_inline)) { return p < pieces && byte_of(p, h) < kb; };
  auto chunk = [&](const char* row, int p, int h) __attribute__((always_inline)) {
    return *(const u32x4*)(row + (in(p, h) ? byte_of(p, h) : 0u));
  };
  struct Piece {
    u32x4 w[RT][2];
  };
  auto bring = [&](int p) __attribute__((always_inline)) {
    Piece c;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) c.w[i][h] = chunk(wrow[i], p, h);
    return c;
  };
  Piece next[U];
#pragma unroll
  for (int t = 0; t < U; ++t) next[t] = bring(kw + t * KW);

  // the rows' quantisation: multiplier and scale of this lane's row
  float mul = 0.f, sx = 0.f;
  bool fine = true;
  if constexpr (XDT != kXOperand) {
    constexpr int N = Chunk<XDT>::N;
    for (int m = 0; m < a.M; ++m) {
      const u32x4* p = (const u32x4*)((const char*)a.a + (size_t)m * a.K * (16 / N));
      float am = 0.f;
      for (int c = tid; c < a.K / N; c += 64 * KW) {
        float f[N];
        Chunk<XDT>::unpack(p[c], f);
#pragma unroll
        for (int j = 0; j < N; ++j) am = amax_nan(am, fabsf(f[j]));
      }
#pragma unroll
      for (int o = 1; o < 64; o *= 2) am = amax_nan(am, __shfl_xor(am, o));
      if (lane == 0) amax[kw][m] = am;
    }
    __syncthreads();
    float am = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w) am = amax_nan(am, amax[w][xr]);
    int8_scale(am, &mul, &sx, &fine);
  }
  // 16 bytes of x's operand
  auto operand = [&](int p, int h) __attribute__((always_inline)) {
    u32x4 o = {0u, 0u, 0u, 0u};
    const uint32_t at = in(p, h) ? byte_of(p, h) : 0u;
    if constexpr (XDT == kXOperand) {
      o = *(const u32x4*)((const char*)a.a + (size_t)xr * kb + at);
    } else {
      constexpr int N = Chunk<XDT>::N;
      const u32x4* row = (const u32x4*)((const char*)a.a + ((size_t)xr * a.K + at) * (16 / N));
#pragma unroll
      for (int c = 0; c < 16 / N; ++c) {
        float f[N];
        Chunk<XDT>::unpack(row[c], f);
#pragma unroll
        for (int w = 0; w < N / 4; ++w) o[c * (N / 4) + w] = int8x4(f + 4 * w, mul, fine);
      }
    }
    return in(p, h) ? o : u32x4{0u, 0u, 0u, 0u};
  };

  Acc acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = Acc{};
  for (int p = kw; p < pieces; p += U * KW) {
    Piece now[U];
#pragma unroll
    for (int t = 0; t < U; ++t) now[t] = next[t];
    if (p + U * KW < pieces)
#pragma unroll
      for (int t = 0; t < U; ++t) next[t] = bring(p + (U + t) * KW);
#pragma unroll
    for (int t = 0; t < U; ++t)
      if (p + t * KW < pieces)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4 x = operand(p + t * KW, h);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const u32x4 w = in(p + t * KW, h) ? now[t].w[i][h] : u32x4{0u, 0u, 0u, 0u};
            acc[i] = Mma16<EL>::go(w, x, acc[i]);
          }
        }
  }
#pragma unroll
  for (int i = 0; i < RT; ++i)
    red[kw][i][lane] = __builtin_bit_cast(f32x4, acc[i]);
  __syncthreads();
  if (kw != 0) return;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int w = 1; w < KW; ++w) acc[i] += __builtin_bit_cast(Acc, red[w][i][lane]);
  if constexpr (HALF) {
    // rows 4 q .. of columns r < 8, and rows 8 + 4 q .. of columns 8 + r
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] += __shfl(acc[i][e], (lane + 40) & 63);
    if (q >= 2) return;
  }
  if (r >= a.M) return;
  typename EP::Pre pre;
  if constexpr (XDT == kXOperand) pre.get(a, r, n0);
  else pre.s = sx;
#pragma unroll
  for (int i = 0; i < OT; ++i) {
    const int n = n0 + TR * i + 4 * q;
    if (n >= a.N) continue;
    float v[4], u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = (float)acc[i][e];
      u[e] = (float)acc[RT - 1][e];
    }
    EP::put(a, r, n, v, u, pre);
  }
}

}  // namespace moe
