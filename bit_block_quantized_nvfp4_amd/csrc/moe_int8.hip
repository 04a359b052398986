// Products in 8-bit integers with a scale per token and per channel:
//
//   a = max(absmax of row t, 2^-100), s[t] = a / 127, q[t][k] = rne(x[t][k] (127 / a))
//   z[t][n] = (sum_k q[t][k] W[n][k]) s[t] S[n]
//
// and, gated, silu of the first half of the columns times the second.  The sums are
// exact in 32-bit integers: |sum| <= 127 128 K < 2^31 for K <= 65536.
#include "moe_int8.hpp"
#include "moe_stream.hpp"
#include "moe_tile.hpp"

namespace moe {

// A block quantises a row: 16 bytes a thread at a time, twice over the row (its absmax,
// then the codes, from the L2).
template <int DT>
__global__ __launch_bounds__(256) void k_int8_quant(const void* __restrict__ x, int K,
                                                    uint8_t* __restrict__ codes,
                                                    float* __restrict__ scales) {
  constexpr int N = Chunk<DT>::N;
  __shared__ float part[4];
  const int t = blockIdx.x, tid = threadIdx.x;
  const u32x4* p = (const u32x4*)((const char*)x + (size_t)t * K * (DT == MOE_DT_F32 ? 4 : 2));
  float am = 0.f;
  for (int c = tid; c < K / N; c += 256) {
    float f[N];
    Chunk<DT>::unpack(p[c], f);
#pragma unroll
    for (int j = 0; j < N; ++j) am = amax_nan(am, fabsf(f[j]));
  }
#pragma unroll
  for (int o = 1; o < 64; o *= 2) am = amax_nan(am, __shfl_xor(am, o));
  if ((tid & 63) == 0) part[tid >> 6] = am;
  __syncthreads();
  am = amax_nan(amax_nan(part[0], part[1]), amax_nan(part[2], part[3]));
  float mul, scale;
  bool fine;
  int8_scale(am, &mul, &scale, &fine);
  uint32_t* q = (uint32_t*)(codes + (size_t)t * K);
  for (int c = tid; c < K / N; c += 256) {
    float f[N];
    Chunk<DT>::unpack(p[c], f);
#pragma unroll
    for (int w = 0; w < N / 4; ++w) q[c * (N / 4) + w] = int8x4(f + 4 * w, mul, fine);
  }
  if (tid == 0) scales[t] = scale;
}

hipError_t launch_int8_quant(const void* x, int T, int K, int dtype, int8_t* codes, float* scales,
                             hipStream_t s) {
  by_dtype(dtype, [&](auto D) {
    MOE_LAUNCH("int8_quant", s, (k_int8_quant<decltype(D)::value>), dim3((unsigned)T), dim3(256), 0, s, x, K,
               (uint8_t*)codes, scales);
  });
  return hipGetLastError();
}

// Up to 16 rows stream the weights.  Where the rows are few values they are quantised in
// the same launch, which every block repeats; else in one of their own.  The shapes: f
// with the kernel, outputs and threads of a block.
static bool int8_streams(int T) { return T <= kStreamRows; }
static bool int8_joins(int T, int K) { return int8_streams(T) && (long)T * K <= 16384; }
template <int XDT, class EP, typename F>
static void by_stream(int K, F&& f) {
  if constexpr (EP::kGated) {
    f(&k_stream<kElI8, XDT, EP, 2, 8, 2>, 16, 512);
  } else {
    if (K >= 8192) f(&k_stream<kElI8, XDT, EP, 1, 16, 4>, 16, 1024);
    else f(&k_stream<kElI8, XDT, EP, 1, 16, 2>, 16, 1024);
  }
}

void register_int8_kernels(std::vector<const void*>& k) {
  for (int dt = MOE_DT_BF16; dt <= MOE_DT_F32; ++dt)
    by_dtype(dt, [&](auto D) {
      constexpr int DT = decltype(D)::value;
      k.push_back((const void*)&k_int8_quant<DT>);
      auto add_stream = [&](auto kernel, int, int) { k.push_back((const void*)kernel); };
      for (int K : {16, 65536}) {
        by_stream<DT, PutInt8<DT>>(K, add_stream);
        by_stream<kXOperand, PutInt8<DT>>(K, add_stream);
      }
      by_stream<DT, PutInt8Gated<DT>>(16, add_stream);
      by_stream<kXOperand, PutInt8Gated<DT>>(16, add_stream);
      for (int i = 0; i < kTileShapes16; ++i)
        by_shape(i, [&](auto shape) {
          k.push_back((const void*)&k_tile<kElI8, false, false, PutInt8<DT>, decltype(shape)>);
          k.push_back((const void*)&k_tile<kElI8, false, false, PutInt8Gated<DT>, decltype(shape)>);
        });
    });
}

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

uint64_t int8_linear_threads(int T, int N) {
  return std::max(tile_threads(T, N), (uint64_t)T * 256);
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
      if (int8_joins(T, W.K)) by_stream<DT, EP>(W.K, stream);
      else if (int8_streams(T)) by_stream<kXOperand, EP>(W.K, stream);
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
