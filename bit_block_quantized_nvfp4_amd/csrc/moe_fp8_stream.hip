// e4m3 products of few rows (up to 16): the weights stream once from memory to
// registers, the rows are quantised on the way, in the same launch.
//
//   z[r][n] = sum_b s[r][b] S[n / 128][b] sum_{k in block b} q[r][k] W[n][k]
//
// Bound by the weight bytes.  A wave owns RT tiles of 16 weight rows and every
// KW-th block of 128 along K; the KW waves of a tile join through LDS in wave
// order.  16 rows are one MFMA operand whatever their number, so one row costs
// the same instructions as sixteen; the rows' own reads are masked off past
// the last.  Each wave quantises the blocks it needs by itself (32 values a
// lane): repeated per tile, but it saves a launch and its wait.
// Measured, calls in a row in a graph: one row of 2048 x 2048 4.1 us, of which a
// launch is most; 4096 x 4096 6.4 us (16.8 MB, 2.6 TB/s), 65536 x 512 8.3 us (34 MB,
// 4.1 TB/s), 4096 x 8192 10.6 us (34 MB, 3.2 TB/s).
// Experts, T = 8, about 75 of 512 groups (H = 2048, I = 512): gate_up 35 us (159
// MB, 4.5 TB/s), down 20 us (79 MB, 4.0 TB/s).
#include <math.h>

#include "moe_ffn_common.hpp"
#include "moe_fp8.hpp"
#include "moe_internal.hpp"

namespace moe {

enum { kStreamLinear = 0, kStreamGateUp = 1, kStreamDown = 2 };

struct StreamArgs {
  const uint8_t* codes;    // [N][K] (of group 0)
  const float* scales;     // [ceil(N/128)][ceil(K/128)]
  const void* x;           // rows of K values
  void* out;
  const int32_t* offsets;  // grouped modes
  const int32_t* sorted_slot;
  const int32_t* groups;
  int R;                   // rows (linear)
  int N, K, T, topk, has_shared;
  int tiles;               // blocks along N
};

// The 16 values of a row from position k on (zeros from K on), twice: at k and
// at k + 64, as loaded.  These are the chunks that a lane holds of the weights
// too: lane 16 q + r has chunks q and q + 4 of row r, so that a load of a wave
// takes whole halves of 16 lines (64 bytes each).
template <int DT>
__device__ __forceinline__ void load32(const void* __restrict__ row, int k, int K,
                                       u32x4 (&v)[32 / Chunk<DT>::N]) {
  constexpr int N = Chunk<DT>::N;
  const u32x4* p = (const u32x4*)row;
#pragma unroll
  for (int i = 0; i < 32 / N; ++i) {
    const int at = k + (i < 16 / N ? i * N : 64 + i * N - 16);
    if (at < K) v[i] = p[at / N];
  }
}

template <int DT, int MODE, int RT, int KW, int NW>
__global__ __launch_bounds__(64 * NW) void k_fp8_stream(StreamArgs a) {
  constexpr int RW = NW / KW;            // tile groups of the block
  constexpr int kPad = 1;
  __shared__ f32x4 red[NW][RT][64 + kPad];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int kw = wv % KW, rw = wv / KW;
  const int tile = blockIdx.x % a.tiles;

  const uint8_t* codes = a.codes;
  const float* scales = a.scales;
  const int nb = (a.K + kQB - 1) / kQB;
  int p0 = 0, rows = a.R;
  if (MODE != kStreamLinear) {
    const int gi = blockIdx.x / a.tiles;
    if (gi >= a.groups[0]) return;
    const int g = a.groups[1 + gi];
    p0 = a.offsets[g];
    rows = a.offsets[g + 1] - p0;
    const int nr = MODE == kStreamGateUp ? 2 * a.N : a.N;  // weight rows of a group
    codes += (size_t)g * nr * a.K;
    scales += (size_t)g * (nr / kQB) * nb;
  }
  // first weight row of each of the wave's tiles; tile i of gate_up is the
  // gate (i = 0) or the up (i = 1) row block of the same columns
  int n0[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
    n0[i] = MODE == kStreamGateUp ? (tile * RW + rw) * 16 + i * a.N
                                  : ((tile * RW + rw) * RT + i) * 16;
  const int nlim = MODE == kStreamGateUp ? 2 * a.N : a.N;
  const int q = lane >> 4;
  const uint8_t* wrow[RT];
  const float* srow[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    wrow[i] = codes + (size_t)min(n0[i] + (lane & 15), nlim - 1) * a.K;
    srow[i] = scales + (size_t)(min(n0[i], nlim - 1) / kQB) * nb;
  }
  // 16 rows at a time: a group has more than 16 only if a caller's ids name an
  // expert twice for one token
  for (int r0 = 0; r0 < rows; r0 += 16) {
    if (r0) __syncthreads();  // red[] is free again
    const int pos = p0 + r0 + (lane & 15);  // this lane's input row
    bool on = r0 + (lane & 15) < rows;
    const char* xrow = nullptr;
    if (on) {
      int from = pos;
      if (MODE != kStreamLinear) {
        const int tok = slot_token(a.sorted_slot[pos], a.T, a.topk, a.has_shared);
        on = tok >= 0;
        if (MODE == kStreamGateUp) from = tok;
      }
      if (on) xrow = (const char*)a.x + (size_t)from * a.K * (DT == MOE_DT_F32 ? 4 : 2);
    }
    f32x4 acc[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int b = kw; b < nb; b += KW) {
      const int k = b * kQB + 16 * q;
      Frag<16> w[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        // chunks past the row's end are read from its start instead: their
        // counterparts in the token rows are zeros
        w[i].set({*(const u32x4*)(wrow[i] + (k < a.K ? k : 0)),
                  *(const u32x4*)(wrow[i] + (k + 64 < a.K ? k + 64 : 0))});
      }
      constexpr int N = Chunk<DT>::N;
      u32x4 v[32 / N];
#pragma unroll
      for (int i = 0; i < 32 / N; ++i) v[i] = u32x4{0u, 0u, 0u, 0u};
      if (on) load32<DT>(xrow, k, a.K, v);
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < 32 / N; ++i) {
        float f[N];
        Chunk<DT>::unpack(v[i], f);
#pragma unroll
        for (int j = 0; j < N; ++j) am = fmaxf(am, fabsf(f[j]));
      }
      am = fmaxf(am, __shfl_xor(am, 16));
      am = fmaxf(am, __shfl_xor(am, 32));
      am = q_floor(am);
      const float m = 448.0f / am, sx = am / 448.0f;
      u32x4 xq[2];
#pragma unroll
      for (int i = 0; i < 32 / N; ++i) {
        float f[N];
        Chunk<DT>::unpack(v[i], f);
#pragma unroll
        for (int j = 0; j < N; j += 4)
          xq[(i * N + j) / 16][(i * N + j) / 4 % 4] =
              fp8x4(f[j] * m, f[j + 1] * m, f[j + 2] * m, f[j + 3] * m);
      }
      Frag<16> xf;
      xf.set(xq);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const f32x4 p = mfma128(w[i], xf);
        const float s = sx * srow[i][b];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(s, p[j], acc[i][j]);
      }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) red[wv][i][lane] = acc[i];
    __syncthreads();
    // wave rw * KW joins its tile group's KW partial sums, in wave order
    if (kw != 0) continue;
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int w2 = 1; w2 < KW; ++w2) acc[i] += red[wv + w2][i][lane];
    if (!on) continue;
    if (MODE == kStreamGateUp) {
      const int n = n0[0] + 4 * q;
      f32x4 h;
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = silu_f32(acc[0][j]) * acc[RT - 1][j];
      *(f32x4*)((float*)a.out + (size_t)pos * a.N + n) = h;
    } else {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int n = n0[i] + 4 * q;
        if (n >= a.N) continue;
        constexpr int ODT = MODE == kStreamDown ? MOE_DT_BF16 : DT;
        const size_t at = (size_t)pos * a.N + n;
        if (ODT == MOE_DT_F32) {
          *(f32x4*)((float*)a.out + at) = acc[i];
        } else if (ODT == MOE_DT_BF16) {
          *(u32x2*)((uint16_t*)a.out + at) =
              u32x2{pack_bf16x2(acc[i][0], acc[i][1]), pack_bf16x2(acc[i][2], acc[i][3])};
        } else {
          *(u32x2*)((uint16_t*)a.out + at) =
              u32x2{pack_f16x2(acc[i][0], acc[i][1]), pack_f16x2(acc[i][2], acc[i][3])};
        }
      }
    }
  }
}

// The linear mode's shapes: f with RT and KW (= NW).  A wave with one or two
// blocks along K waits the fewest times; where that leaves more waves than the
// chip holds, it takes two row tiles, which share its rows' quantisation, and
// more of K (in a row in a graph, us, RT x KW):
//   rows x N x K        1x16   1x8   2x8   1x4   2x4
//   1 x 4096 x 4096      6.4   7.2   8.9  10.0  12.1
//   16 x 512 x 8192     13.0  13.2  17.1  14.6  17.8
//   1 x 2048 x 2048      4.1   4.1   5.0   5.1   6.3
//   1 x 4096 x 1024      3.6   3.3   3.7   3.5   4.2
//   1 x 16384 x 1024     9.1   6.3   5.0   5.5   5.1
//   1 x 32768 x 512     12.2   7.9   5.9   6.2   4.9
//   1 x 2048 x 512       2.9   2.7   3.1   2.6   3.0
template <typename F>
static void by_linear_shape(int N, int K, F&& f) {
  const bool wide = N >= 8192;
  if (K >= 2048 && N <= 4096) f(IntC<1>{}, IntC<16>{});
  else if (K >= 1024) wide ? f(IntC<2>{}, IntC<8>{}) : f(IntC<1>{}, IntC<8>{});
  else wide ? f(IntC<2>{}, IntC<4>{}) : f(IntC<1>{}, IntC<4>{});
}

void register_fp8_stream_kernels(std::vector<const void*>& k) {
  for (int dt = MOE_DT_BF16; dt <= MOE_DT_F32; ++dt)
    by_dtype(dt, [&](auto D) {
      for (int N : {4096, 8192})
        for (int K : {512, 1024, 2048})
          by_linear_shape(N, K, [&](auto RT, auto KW) {
            constexpr int kw = decltype(KW)::value;
            k.push_back((const void*)&k_fp8_stream<decltype(D)::value, kStreamLinear,
                                                   decltype(RT)::value, kw, kw>);
          });
    });
  k.push_back((const void*)&k_fp8_stream<MOE_DT_BF16, kStreamGateUp, 2, 8, 8>);
  k.push_back((const void*)&k_fp8_stream<MOE_DT_BF16, kStreamGateUp, 2, 4, 4>);
  k.push_back((const void*)&k_fp8_stream<MOE_DT_F32, kStreamDown, 2, 2, 2>);
  k.push_back((const void*)&k_fp8_stream<MOE_DT_F32, kStreamDown, 4, 2, 2>);
  k.push_back((const void*)&k_fp8_stream<MOE_DT_F32, kStreamDown, 4, 1, 1>);
}

hipError_t launch_fp8_stream_linear(const moe_fp8_matrix& M, const void* x, int T, int dtype,
                                    void* out, hipStream_t s) {
  StreamArgs a{};
  a.codes = M.codes;
  a.scales = M.scales;
  a.x = x;
  a.out = out;
  a.R = T;
  a.N = M.N;
  a.K = M.K;
  by_dtype(dtype, [&](auto D) {
    by_linear_shape(M.N, M.K, [&](auto RT, auto KW) {
      constexpr int DT = decltype(D)::value, rt = decltype(RT)::value, kw = decltype(KW)::value;
      a.tiles = (M.N + 16 * rt - 1) / (16 * rt);
      MOE_LAUNCH("fp8_stream", s, (k_fp8_stream<DT, kStreamLinear, rt, kw, kw>), dim3(a.tiles),
                 dim3(64 * kw), 0, s, a);
    });
  });
  return hipGetLastError();
}

hipError_t launch_fp8_stream_experts(const moe_fp8_weights& W, const uint16_t* x, int T, int K,
                                     const int32_t* offsets, const int32_t* sorted_slot,
                                     const int32_t* groups, float* h, uint16_t* y,
                                     hipStream_t s) {
  const long most = (long)T * K < W.E ? (long)T * K : W.E;
  const int G = (int)most + W.has_shared;  // groups that can be active
  StreamArgs a{};
  a.codes = W.gu_codes;
  a.scales = W.gu_scales;
  a.x = x;
  a.out = h;
  a.offsets = offsets;
  a.sorted_slot = sorted_slot;
  a.groups = groups;
  a.N = W.I;
  a.K = W.H;
  a.T = T;
  a.topk = K;
  a.has_shared = W.has_shared;
  a.tiles = W.I / 16;
  // Blocks of 4 waves where there are enough of them, of 8 for fewer, each wave a
  // shorter stretch of K.  Down: four row tiles to a wave share its rows'
  // quantisation once there are groups enough, and one wave does all of a short
  // K.  The call in a row in a graph, H = 2048, I = 512, top 10 of 512 and a
  // shared one, us (gate_up waves, down row tiles x waves; * the one taken):
  //   T (groups)   8, 2x2  4, 2x2  8, 4x2  4, 4x2  4, 4x1
  //   1 (11)        15.0*   16.5    15.9    17.1    18.4
  //   2 (21)        21.5    21.1*   21.8    21.5    22.5
  //   4 (41)        33.6    32.6*   34.8    34.5    33.1
  //   6 (61)        48.0    44.2    48.2    44.1    43.5*
  //   8 (81)        53.7    49.7    54.9    50.8    47.7*
  //   12 (121)      77.4    70.6    77.5    70.5    66.2*
  if (G > 16)
    MOE_LAUNCH("fp8_stream_gate_up", s, (k_fp8_stream<MOE_DT_BF16, kStreamGateUp, 2, 4, 4>),
               dim3((unsigned)G * a.tiles), dim3(256), 0, s, a);
  else
    MOE_LAUNCH("fp8_stream_gate_up", s, (k_fp8_stream<MOE_DT_BF16, kStreamGateUp, 2, 8, 8>),
               dim3((unsigned)G * a.tiles), dim3(512), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.codes = W.dn_codes;
  a.scales = W.dn_scales;
  a.x = h;
  a.out = y;
  a.N = W.H;
  a.K = W.I;
  auto down = [&](auto RT, auto KW) {
    constexpr int rt = decltype(RT)::value, kw = decltype(KW)::value;
    a.tiles = W.H / (16 * rt);
    MOE_LAUNCH("fp8_stream_down", s, (k_fp8_stream<MOE_DT_F32, kStreamDown, rt, kw, kw>),
               dim3((unsigned)G * a.tiles), dim3(64 * kw), 0, s, a);
  };
  if (G <= 48) down(IntC<2>{}, IntC<2>{});
  else if (W.I > 512) down(IntC<4>{}, IntC<2>{});
  else down(IntC<4>{}, IntC<1>{});
  return hipGetLastError();
}

}  // namespace moe
