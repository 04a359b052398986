// Products in 8-bit integers with a scale per token and per channel:
//
//   a = max(absmax of row t, 2^-100), s[t] = a / 127, q[t][k] = rne(x[t][k] (127 / a))
//   z[t][n] = (sum_k q[t][k] W[n][k]) s[t] S[n]
//
// and, gated, silu of the first half of the columns times the second.  The sums are
// exact in 32-bit integers: |sum| <= 127 128 K < 2^31 for K <= 65536.
//
// bf16 rows: 8192 x 2048 x 8192 37.7 us of quantisation and 116.6 us (2.36 POP/s); gated, 8192 x
// 16384 x 2048, 14.6 and 275 us, where a tile's 16 steps are followed by as many values of silu and
// the columns' scales are read in every pass of the epilogue; f16 333 x 4168 x 2064 4.2 and 11.4 us,
// by latency; 1 row of 4096 x 4096 8.2 us in one launch.
#include "moe_int8.hpp"
#include "moe_stream.hpp"
#include "moe_tile.hpp"

namespace moe {

// A block of W waves quantises a row, whose chunks of 16 bytes, up to U a thread, stay in
// registers between its absmax and its codes; longer rows (U = 0) are read twice, from the
// L2 the second time.  Bound by memory, few rows by the launch (in a row in a graph, us): 333
// rows of 2064 f16 3.9, 8192 of 2048 bf16 13.5, of 8192 40.9, of 16384 90.8 (4.4 TB/s), 4 of 65536
// 9.0; 4 waves reading twice take 144.6 and 21.6 for the last two, a wave to a row 6.4 and
// 15.8 for the first two (the codes' arithmetic wants more waves).
template <int DT, int U, int W>
__global__ __launch_bounds__(64 * W) void k_int8_quant(const void* __restrict__ x, int K,
                                                       uint8_t* __restrict__ codes,
                                                       float* __restrict__ scales) {
  constexpr int N = Chunk<DT>::N, L = 64 * W;
  __shared__ float part[W];
  const int t = blockIdx.x, tid = threadIdx.x, chunks = K / N;
  const u32x4* p = (const u32x4*)((const char*)x + (size_t)t * K * (DT == MOE_DT_F32 ? 4 : 2));
  float am = 0.f;
  auto look = [&](u32x4 v) __attribute__((always_inline)) {
    float f[N];
    Chunk<DT>::unpack(v, f);
#pragma unroll
    for (int j = 0; j < N; ++j) am = amax_nan(am, fabsf(f[j]));
  };
  u32x4 held[U > 0 ? U : 1];
  if constexpr (U > 0) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      held[i] = u32x4{0u, 0u, 0u, 0u};
      if (tid + L * i < chunks) held[i] = p[tid + L * i];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) look(held[i]);
  } else {
    for (int c = tid; c < chunks; c += L) look(p[c]);
  }
#pragma unroll
  for (int o = 1; o < 64; o *= 2) am = amax_nan(am, __shfl_xor(am, o));
  if ((tid & 63) == 0) part[tid >> 6] = am;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) am = amax_nan(am, part[w]);
  float mul, scale;
  bool fine;
  int8_scale(am, &mul, &scale, &fine);
  uint32_t* q = (uint32_t*)(codes + (size_t)t * K);
  auto put = [&](u32x4 v, int c) __attribute__((always_inline)) {
    float f[N];
    Chunk<DT>::unpack(v, f);
#pragma unroll
    for (int w = 0; w < N / 4; ++w) q[c * (N / 4) + w] = int8x4(f + 4 * w, mul, fine);
  };
  if constexpr (U > 0) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (tid + L * i < chunks) put(held[i], tid + L * i);
  } else {
    for (int c = tid; c < chunks; c += L) put(p[c], c);
  }
  if (tid == 0) scales[t] = scale;
}

// f with the chunks that a thread holds and the waves of a block for rows of K values.
template <int DT, typename F>
static void by_row(int K, F&& f) {
  const int waves = (K / Chunk<DT>::N + 63) / 64;  // loads of a wave
  if (waves <= 4) f(IntC<1>{}, IntC<4>{});
  else if (waves <= 16) f(IntC<4>{}, IntC<4>{});
  else if (waves <= 64) f(IntC<4>{}, IntC<16>{});
  else f(IntC<0>{}, IntC<16>{});
}

hipError_t launch_int8_quant(const void* x, int T, int K, int dtype, int8_t* codes, float* scales,
                             hipStream_t s) {
  by_dtype(dtype, [&](auto D) {
    constexpr int DT = decltype(D)::value;
    by_row<DT>(K, [&](auto U, auto W) {
      constexpr int kWaves = decltype(W)::value;
      MOE_LAUNCH("int8_quant", s, (k_int8_quant<DT, decltype(U)::value, kWaves>), dim3((unsigned)T),
                 dim3(64 * kWaves), 0, s, x, K, (uint8_t*)codes, scales);
    });
  });
  return hipGetLastError();
}

// Up to 16 rows stream the weights.  Where the rows are few values they are quantised in
// the same launch, which every block repeats; else in one of their own, which costs a call
// outside a graph one more launch.  bf16, weights from memory, in a row in a graph, us, apart
// and joined:
//   N x K, plain     1 row        4 rows       8 rows       N x K, gated    1 row        4 rows
//   512 x 2048       5.8  5.4     6.1  7.5     6.3   9.8    512 x 2048      6.8  5.9     7.0  7.5
//   2048 x 2048      5.9  5.6     6.2  7.7     6.5  10.0    2048 x 2048     7.0  6.0     7.2  7.7
//   2048 x 4096      8.1  7.1     8.7  9.0                  8192 x 2048     9.4  8.7     9.7  10.8
//   8192 x 2048      9.2  9.3     9.7  11.6    10.1 14.0    16384 x 2048   11.1  10.9   11.4  12.8
//   8192 x 4096     11.7 13.3    12.4  15.9                 16384 x 4096   18.8  21.0   18.9  23.9
//   8192 x 8192     19.9 26.8                               8192 x 8192    18.1  20.0
// So joining wins in a graph for one row and up to about 4096 outputs (gated more), and loses
// from two rows on, though the rule goes by the rows' values alone.  The shapes: f with the
// kernel, outputs and threads of a block.
static bool int8_streams(int T) { return T <= kStreamRows; }
static bool int8_joins(int T, int K) { return T <= 4 && (long)T * K <= 8192; }
template <int XDT, class EP, typename F>
static void by_stream(int M, int N, int K, F&& f) {
  const bool half = takes_half(M, N, EP::kGated);
  if constexpr (EP::kGated) {
    if (half) f(&k_stream<kElI8, XDT, EP, 2, 8, 2, true>, 8, 512);
    else f(&k_stream<kElI8, XDT, EP, 2, 8, 2>, 16, 512);
  } else {
    if (half) f(&k_stream<kElI8, XDT, EP, 1, 16, 2, true>, 8, 1024);
    else if (K >= 8192) f(&k_stream<kElI8, XDT, EP, 1, 16, 4>, 16, 1024);
    else f(&k_stream<kElI8, XDT, EP, 1, 16, 2>, 16, 1024);
  }
}

void register_int8_kernels(std::vector<const void*>& k) {
  for (int dt = MOE_DT_BF16; dt <= MOE_DT_F32; ++dt)
    by_dtype(dt, [&](auto D) {
      constexpr int DT = decltype(D)::value;
      for (int K : {16, 4096, 16384, 65536})
        by_row<DT>(K, [&](auto U, auto W) {
          k.push_back((const void*)&k_int8_quant<DT, decltype(U)::value, decltype(W)::value>);
        });
      auto add_stream = [&](auto kernel, int, int) { k.push_back((const void*)kernel); };
      for (int M : {1, kStreamRows})
        for (int K : {16, 65536}) {
          by_stream<DT, PutInt8<DT>>(M, 8, K, add_stream);
          by_stream<kXOperand, PutInt8<DT>>(M, 8, K, add_stream);
          by_stream<DT, PutInt8Gated<DT>>(M, 8, K, add_stream);
          by_stream<kXOperand, PutInt8Gated<DT>>(M, 8, K, add_stream);
        }
      for (int i = 0; i < kTileShapes16; ++i)
        by_shape(i, [&](auto shape) {
          k.push_back((const void*)&k_tile<kElI8, false, false, PutInt8<DT>, decltype(shape)>);
          k.push_back((const void*)&k_tile<kElI8, false, false, PutInt8Gated<DT>, decltype(shape)>);
        });
    });
}

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

uint64_t int8_quant_threads(int T, int K, int dtype) {
  uint64_t n = 0;
  by_dtype(dtype, [&](auto D) {
    by_row<decltype(D)::value>(K, [&](auto, auto W) { n = (uint64_t)T * 64 * decltype(W)::value; });
  });
  return n;
}
uint64_t int8_linear_threads(int T, int N, int K, int dtype) {
  if (int8_streams(T)) return 0;  // at most 131072 / 8 blocks
  return std::max(tile_threads(T, N, steps_of(K, 1)), int8_quant_threads(T, K, dtype));
}

size_t int8_linear_workspace_bytes(int T, int N, int K) {
  if (int8_joins(T, K)) return 0;
  return up256((size_t)T * K) + up256((size_t)T * sizeof(float));
}

hipError_t launch_int8_linear(const moe_int8_matrix& W, const void* x, int T, int dtype, int gated,
                              void* out, void* ws, hipStream_t s) {
  TileArgs16 a{};
  a.a = x;
  a.b = W.codes;
  a.lda = a.ldb = (uint32_t)W.K;
  a.M = T;
  a.N = gated ? W.N / 2 : W.N;
  a.K = W.K;
  a.out = out;
  a.sn = W.scales;
  if (!int8_joins(T, W.K)) {
    int8_t* q = (int8_t*)ws;
    float* sx = (float*)((char*)ws + up256((size_t)T * W.K));
    hipError_t e = launch_int8_quant(x, T, W.K, dtype, q, sx, s);
    if (e != hipSuccess) return e;
    a.a = q;
    a.sm = sx;
  }
  by_dtype(dtype, [&](auto D) {
    constexpr int DT = decltype(D)::value;
    auto stream = [&](auto kernel, int outs, int threads) {
      MOE_LAUNCH("int8_stream", s, kernel, dim3((unsigned)((a.N + outs - 1) / outs)), dim3(threads), 0, s, a);
    };
    auto go = [&](auto ep) {
      typedef decltype(ep) EP;
      if (int8_joins(T, W.K)) by_stream<DT, EP>(T, a.N, W.K, stream);
      else if (int8_streams(T)) by_stream<kXOperand, EP>(T, a.N, W.K, stream);
      else {
        const int best = tile_shape(T, W.N, steps_of(W.K, 1));
        by_shape(best, [&](auto shape) {
          a.nt = (W.N + shape.BN - 1) / shape.BN;
          MOE_LAUNCH("int8_tile", s, (k_tile<kElI8, false, false, EP, decltype(shape)>),
                     dim3((unsigned)tiles_of(best, T, W.N)), dim3(shape.kThreads), 0, s, a);
        });
      }
    };
    if (gated) go(PutInt8Gated<DT>{});
    else go(PutInt8<DT>{});
  });
  return hipGetLastError();
}

}  // namespace moe
