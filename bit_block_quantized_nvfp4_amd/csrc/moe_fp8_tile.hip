// e4m3 products of many rows: quantisation of the rows, then tiles of BN
// weight rows x BM token rows on the 128-wide f8 MFMA.
//
//   z[t][n] = sum_b s[t][b] S[n / 128][b] sum_{k in block b} q[t][k] W[n][k]
//
// One K step is one block of 128, so a step's MFMA starts from zero and its
// result is scaled into the f32 accumulators: 4 multiply-adds per MFMA of 32
// cycles, which run beside the matrix unit.  Weights are the MFMA's A operand:
// a lane then has one token per tile column, hence one scale, and four
// consecutive outputs.
//
// Both operands go from memory to LDS without registers (16 bytes a lane, the
// next step's while this one is computed).  A row of a step is 128 bytes, its
// 16-byte chunk c stands at place c ^ (row % 8), so that the reads of 16 rows
// at one chunk meet every bank once; the DMA writes lanes in order, hence the
// permutation is applied to the addresses that it reads.
#include <math.h>

#include "moe_ffn_common.hpp"
#include "moe_fp8.hpp"
#include "moe_internal.hpp"
#include "moe_prefill_items.hpp"

namespace moe {

// One thread per 8 values, 16 lanes to a block of 128.  ldq: bytes of a code
// row (K, or K rounded up to 128 with zeros behind).
template <int DT>
__global__ __launch_bounds__(256) void k_fp8_quant(const void* __restrict__ x, int T, int K,
                                                   int ldq, int lg, int cb,
                                                   uint8_t* __restrict__ codes,
                                                   float* __restrict__ scales) {
  constexpr int N = Chunk<DT>::N;
  const int nb = (K + kQB - 1) / kQB;
  int t, c;
  if (!row_chunk(lg, cb, T, nb * 16, &t, &c)) return;
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
  if ((c & 15) == 0) scales[(size_t)t * nb + c / 16] = am / 448.0f;
}

enum { kTileLinear = 0, kTileGateUp = 1, kTileDown = 2 };

struct TileArgs {
  const uint8_t* codes;    // weights [N][K] (of group 0)
  const float* scales;     // [ceil(N/128)][nb]
  const uint8_t* xq;       // token codes [rows][nb * 128]
  const float* xs;         // token scales [rows][nb]
  void* out;
  float* out_scales;       // gate_up: scales of h
  const int32_t* offsets;  // grouped modes
  const int32_t* sorted_slot;
  int R;                   // rows (linear)
  int N, K, T, topk, has_shared, G;
  int nt;                  // tiles along N
};

__device__ __forceinline__ void wait_dma() {
  __builtin_amdgcn_s_waitcnt(0 | (7 << 4) | (15 << 8));  // vmcnt(0) only
}

template <int MODE, int DT, int BN, int BM, int WN, int WM>
__global__ __launch_bounds__(64 * WN * WM) void k_fp8_tile(TileArgs a) {
  constexpr int NT = 64 * WN * WM;
  constexpr int TN = BN / WN, TM = BM / WM;    // a wave's part of the tile
  constexpr int FN = TN / 16, FM = TM / 16;
  constexpr int ROWS = BN + BM;
  constexpr int DMA = ROWS * 8 / NT;           // 16-byte chunks per thread and step
  constexpr bool EX = DT == MOE_DT_F32;
  static_assert(ROWS * 8 % NT == 0 && TN % 16 == 0 && TM % 16 == 0, "tile shape");
  __shared__ __align__(1024) uint8_t lds[2][ROWS * kQB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wv % WN, wm = wv / WN;        // waves of one SIMD share wn
  const int nb = (a.K + kQB - 1) / kQB;

  const uint8_t* codes = a.codes;
  const float* scales = a.scales;
  int m0, rows, n0;                            // first token row, rows left, first column
  if (MODE == kTileLinear) {
    const int mt = (a.R + BM - 1) / BM;
    // 8 XCDs take the blocks in turn: give each a run of token tiles of one
    // weight tile
    const int b = blockIdx.x;
    n0 = (b / mt) * BN;
    m0 = (b % mt) * BM;
    rows = a.R - m0;
  } else {
    __shared__ unsigned long long base[kPMaxG];
    __shared__ unsigned long long wsum[NT / 64];
    PfTile ti;
    if (!pf_find_tile<NT>(a.offsets, a.G, a.nt, base, wsum, &ti)) return;
    const int nr = MODE == kTileGateUp ? 2 * a.N : a.N;
    codes += (size_t)ti.g * nr * a.K;
    scales += (size_t)ti.g * (nr / kQB) * nb;
    m0 = ti.p0;
    rows = ti.rows;
    n0 = ti.nt * (MODE == kTileGateUp ? BN / 2 : BN);
  }
  if (rows > BM) rows = BM;

  // Weight row of LDS row lr.  gate_up: each wave's TN rows are TN / 2 gate
  // rows and the up rows of the same columns.
  auto wrow_of = [&](int lr) {
    if (MODE == kTileGateUp) {
      const int w = lr / TN, q = lr % TN;
      return n0 + w * (TN / 2) + q % (TN / 2) + (q < TN / 2 ? 0 : a.N);
    }
    return min(n0 + lr, a.N - 1);
  };
  const uint8_t* src[DMA];
  int kbase[DMA];                              // position of the chunk in the block
#pragma unroll
  for (int i = 0; i < DMA; ++i) {
    const int at = i * NT + tid;               // chunk: LDS row at / 8, place at % 8
    const int lr = at >> 3, c = (at & 7) ^ (lr & 7);
    kbase[i] = 16 * c;
    if (lr < BN) {
      src[i] = codes + (size_t)wrow_of(lr) * a.K;
    } else {
      const int r = min(lr - BN, rows - 1);
      int from = m0 + r;
      if (MODE == kTileGateUp) from = max(slot_token(a.sorted_slot[from], a.T, a.topk, a.has_shared), 0);
      src[i] = a.xq + (size_t)from * nb * kQB;
    }
  }
  auto dma = [&](int b, int buf) {
#pragma unroll
    for (int i = 0; i < DMA; ++i) {
      // past the end of a weight row its first chunk is read instead: the
      // tokens' codes there are zeros
      int k = b * kQB + kbase[i];
      if (i * NT < BN * 8 && k >= a.K && (i * NT + tid) < BN * 8) k = 0;
      dma16(src[i] + k, &lds[buf][(i * NT + wv * 64) * 16]);
    }
  };

  f32x4 acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // this lane's token of each tile column, for its scales
  const float* xs[FM];
  int live = 0;                                // columns of the wave with rows in them
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    const int r = wm * TM + 16 * j + (lane & 15);
    if (wm * TM + 16 * j < rows) live = j + 1;
    int from = m0 + min(r, rows - 1);
    if (MODE == kTileGateUp) from = max(slot_token(a.sorted_slot[from], a.T, a.topk, a.has_shared), 0);
    xs[j] = a.xs + (size_t)from * nb;
  }
  // weight scales of the wave's rows: constant over each 128 rows
  const float* ws[2];
  if (MODE == kTileGateUp) {
    ws[0] = scales + (size_t)(n0 / kQB) * nb;
    ws[1] = scales + (size_t)((n0 + a.N) / kQB) * nb;
  } else {
    ws[0] = ws[1] = scales + (size_t)(min(n0 + wn * TN, a.N - 1) / kQB) * nb;
  }

  // LDS address of this lane's two chunks of row 16 i + lane % 16
  const int fr = lane & 15, fq = lane >> 4;
  auto frag = [&](const uint8_t* p, int row16) {
    const uint8_t* r = p + (row16 + fr) * kQB;
    return join8(*(const u32x4*)(r + ((fq ^ (fr & 7)) << 4)),
                 *(const u32x4*)(r + (((fq + 4) ^ (fr & 7)) << 4)));
  };

  dma(0, 0);
  float sx[FM];
#pragma unroll
  for (int j = 0; j < FM; ++j) sx[j] = xs[j][0];
  wait_dma();
  __syncthreads();
  for (int b = 0; b < nb; ++b) {
    const int buf = b & 1;
    float sn[FM];
    if (b + 1 < nb) {
      dma(b + 1, buf ^ 1);
#pragma unroll
      for (int j = 0; j < FM; ++j) sn[j] = xs[j][b + 1];
    }
    const uint8_t* pw = &lds[buf][wn * TN * kQB];
    const uint8_t* pt = &lds[buf][(BN + wm * TM) * kQB];
    Frag<EX> tf[FM];
    if (live > 0) {
#pragma unroll
      for (int j = 0; j < FM; ++j) tf[j].set(frag(pt, 16 * j));
      const float w0 = ws[0][b], w1 = ws[1][b];
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        Frag<EX> wf;
        wf.set(frag(pw, 16 * i));
        const float sw = (MODE == kTileGateUp && i >= FN / 2) ? w1 : w0;
#pragma unroll
        for (int j = 0; j < FM; ++j) {
          if (MODE == kTileLinear || j < live) {
            const f32x4 p = mfma128(wf, tf[j]);
            const float s = sx[j] * sw;
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[i][j][q] = fmaf(s, p[q], acc[i][j][q]);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < FM; ++j) sx[j] = sn[j];
    wait_dma();
    __syncthreads();
  }

  if (MODE == kTileGateUp) {
    // h = silu(gate) up in f32, its absmax over the block's 128 columns (one
    // scale of h), then its codes
    constexpr int HN = FN / 2;
    static_assert(MODE != kTileGateUp || BN == 256, "a tile holds one scale of h");
    float* amax = (float*)&lds[0][0];          // [WN][BM]
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < HN; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float h = silu_f32(acc[i][j][q]) * acc[HN + i][j][q];
          acc[i][j][q] = h;
          am = fmaxf(am, fabsf(h));
        }
      am = fmaxf(am, __shfl_xor(am, 16));
      am = fmaxf(am, __shfl_xor(am, 32));
      if (fq == 0) amax[wn * BM + wm * TM + 16 * j + fr] = am;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int r = wm * TM + 16 * j + fr;
      float am = amax[r];
#pragma unroll
      for (int w = 1; w < WN; ++w) am = fmaxf(am, amax[w * BM + r]);
      am = q_floor(am);
      const float m = 448.0f / am;
      if (r < rows) {
        uint8_t* dst = (uint8_t*)a.out + (size_t)(m0 + r) * a.N + n0 + wn * (TN / 2);
#pragma unroll
        for (int i = 0; i < HN; ++i)
          *(uint32_t*)(dst + 16 * i + 4 * fq) = fp8x4(acc[i][j][0] * m, acc[i][j][1] * m,
                                                      acc[i][j][2] * m, acc[i][j][3] * m);
        if (wn == 0 && fq == 0)
          a.out_scales[(size_t)(m0 + r) * (a.N / kQB) + n0 / kQB] = am / 448.0f;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int r = wm * TM + 16 * j + fr;
      bool on = r < rows;
      if (MODE == kTileDown && on)
        on = slot_token(a.sorted_slot[m0 + r], a.T, a.topk, a.has_shared) >= 0;
      if (!on) continue;
#pragma unroll
      for (int i = 0; i < FN; ++i) {
        const int n = n0 + wn * TN + 16 * i + 4 * fq;
        if (n >= a.N) continue;
        const size_t at = (size_t)(m0 + r) * a.N + n;
        const f32x4 v = acc[i][j];
        if (DT == MOE_DT_F32)
          *(f32x4*)((float*)a.out + at) = v;
        else if (DT == MOE_DT_BF16)
          *(u32x2*)((uint16_t*)a.out + at) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        else
          *(u32x2*)((uint16_t*)a.out + at) = u32x2{pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3])};
      }
    }
  }
}

void register_fp8_tile_kernels(std::vector<const void*>& k) {
  auto add = [&](auto D) {
    constexpr int DT = decltype(D)::value;
    k.push_back((const void*)&k_fp8_quant<DT>);
    if constexpr (DT != MOE_DT_F32)
      k.push_back((const void*)&k_fp8_tile<kTileLinear, DT, 256, 256, 2, 4>);
    else
      k.push_back((const void*)&k_fp8_tile<kTileLinear, DT, 128, 128, 2, 2>);
    k.push_back((const void*)&k_fp8_tile<kTileLinear, DT, 128, 64, 4, 1>);
  };
  for (int dt = MOE_DT_BF16; dt <= MOE_DT_F32; ++dt) by_dtype(dt, add);
  k.push_back((const void*)&k_fp8_tile<kTileGateUp, MOE_DT_BF16, 256, 128, 4, 2>);
  k.push_back((const void*)&k_fp8_tile<kTileDown, MOE_DT_BF16, 256, 128, 4, 2>);
}

hipError_t launch_fp8_quant(const void* x, int T, int K, int dtype, int ldq, uint8_t* codes,
                            float* scales, hipStream_t s) {
  const RowGrid g = row_grid(T, (K + kQB - 1) / kQB * 16);
  by_dtype(dtype, [&](auto D) {
    MOE_LAUNCH("fp8_quant", s, k_fp8_quant<decltype(D)::value>, dim3(g.blocks), dim3(256), 0, s, x,
               T, K, ldq, g.lg, g.cb, codes, scales);
  });
  return hipGetLastError();
}

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
static int blocks_of(int K) { return (K + kQB - 1) / kQB; }

size_t fp8_linear_workspace_bytes(int T, int K) {
  if (T <= kFp8StreamMaxT) return 0;
  return up256((size_t)T * blocks_of(K) * kQB) + up256((size_t)T * blocks_of(K) * sizeof(float));
}

hipError_t launch_fp8_linear(const moe_fp8_matrix& M, const void* x, int T, int dtype, void* out,
                             void* ws, hipStream_t s) {
  if (T <= kFp8StreamMaxT) return launch_fp8_stream_linear(M, x, T, dtype, out, s);
  const int nb = blocks_of(M.K);
  uint8_t* xq = (uint8_t*)ws;
  float* xs = (float*)(xq + up256((size_t)T * nb * kQB));
  hipError_t e = launch_fp8_quant(x, T, M.K, dtype, nb * kQB, xq, xs, s);
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
  const long big = (long)((M.N + 255) / 256) * ((T + 255) / 256);
  by_dtype(dtype, [&](auto D) {
    constexpr int DT = decltype(D)::value;
    if (big >= 192) {
      if constexpr (DT != MOE_DT_F32) {
        MOE_LAUNCH("fp8_tile_256", s, (k_fp8_tile<kTileLinear, DT, 256, 256, 2, 4>),
                   dim3((unsigned)big), dim3(512), 0, s, a);
      } else {
        // f16 operands take twice the registers
        const unsigned n = (unsigned)((M.N + 127) / 128) * (unsigned)((T + 127) / 128);
        MOE_LAUNCH("fp8_tile_128", s, (k_fp8_tile<kTileLinear, DT, 128, 128, 2, 2>), dim3(n),
                   dim3(256), 0, s, a);
      }
    } else {
      const unsigned n = (unsigned)((M.N + 127) / 128) * (unsigned)((T + 63) / 64);
      MOE_LAUNCH("fp8_tile_128", s, (k_fp8_tile<kTileLinear, DT, 128, 64, 4, 1>), dim3(n),
                 dim3(256), 0, s, a);
    }
  });
  return hipGetLastError();
}

size_t fp8_expert_ffn_workspace_bytes(int T, int K, int H, int I, int has_shared) {
  const size_t S = (size_t)T * K + (has_shared ? T : 0);
  if (T <= kFp8StreamMaxT) return up256(S * I * sizeof(float));
  return up256((size_t)T * H) + up256((size_t)T * (H / kQB) * sizeof(float)) + up256(S * I) +
         up256(S * (I / kQB) * sizeof(float));
}

hipError_t launch_fp8_expert_ffn(const moe_fp8_weights& W, const uint16_t* x, int T, int K,
                                 const int32_t* offsets, const int32_t* sorted_slot,
                                 const int32_t* groups, uint16_t* y, void* ws, hipStream_t s) {
  if (T <= kFp8StreamMaxT)
    return launch_fp8_stream_experts(W, x, T, K, offsets, sorted_slot, groups, (float*)ws, y, s);
  const size_t S = (size_t)T * K + (W.has_shared ? T : 0);
  uint8_t* xq = (uint8_t*)ws;
  float* xs = (float*)(xq + up256((size_t)T * W.H));
  uint8_t* hq = (uint8_t*)xs + up256((size_t)T * (W.H / kQB) * sizeof(float));
  float* hs = (float*)(hq + up256(S * W.I));
  hipError_t e = launch_fp8_quant(x, T, W.H, MOE_DT_BF16, W.H, xq, xs, s);
  if (e != hipSuccess) return e;
  TileArgs a{};
  a.offsets = offsets;
  a.sorted_slot = sorted_slot;
  a.T = T;
  a.topk = K;
  a.has_shared = W.has_shared;
  a.G = W.E + W.has_shared;
  // row tiles: at most one partial tile per group, and the full ones
  const unsigned mt = (unsigned)(S / kPM + (size_t)a.G);
  a.codes = W.gu_codes;
  a.scales = W.gu_scales;
  a.xq = xq;
  a.xs = xs;
  a.out = hq;
  a.out_scales = hs;
  a.N = W.I;
  a.K = W.H;
  a.nt = W.I / 128;
  MOE_LAUNCH("fp8_tile_gate_up", s, (k_fp8_tile<kTileGateUp, MOE_DT_BF16, 256, 128, 4, 2>),
             dim3(mt * a.nt), dim3(512), 0, s, a);
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
  a.nt = (W.H + 255) / 256;
  MOE_LAUNCH("fp8_tile_down", s, (k_fp8_tile<kTileDown, MOE_DT_BF16, 256, 128, 4, 2>),
             dim3(mt * a.nt), dim3(512), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
