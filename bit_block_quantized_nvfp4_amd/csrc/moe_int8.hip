// Products in 8-bit integers with a scale per token and per channel:
//
//   a = max(absmax of row t, 2^-100), s[t] = a / 127, q[t][k] = rne(x[t][k] (127 / a))
//   z[t][n] = (sum_k q[t][k] W[n][k]) s[t] S[n]
//
// and, gated, silu of the first half of the columns times the second.  The sums are
// exact in 32-bit integers: |sum| <= 127 128 K < 2^31 for K <= 65536.
#include "moe_tile.hpp"

namespace moe {

// z from the sum and its two scales, each product rounded to f32: not joined with the
// rounding to f16 that follows (one instruction does both), so that every type has the
// same z.
__device__ __forceinline__ float scaled(float sum, float s, float w) {
#pragma clang fp contract(off)
  float z = sum * s;
  z = z * w;
  asm("" : "+v"(z));
  return z;
}

template <int DT>
struct PutInt8 {
  static constexpr bool kGated = false;
  typedef NoPre Pre;
  static __device__ __forceinline__ void put(const TileArgs16& a, int m, int n, float (&v)[8],
                                             const float (&)[8], const Pre&) {
    const float s = a.sm[m];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = scaled(v[e], s, a.sn[n + e]);
    put8<DT>(a.out, (size_t)m * a.N + n, v);
  }
};

template <int DT>
struct PutInt8Gated {
  static constexpr bool kGated = true;
  typedef NoPre Pre;
  static __device__ __forceinline__ void put(const TileArgs16& a, int m, int n, float (&v)[8],
                                             const float (&u)[8], const Pre&) {
    const float s = a.sm[m];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = silu_f32(scaled(v[e], s, a.sn[n + e])) * scaled(u[e], s, a.sn[a.N + n + e]);
    put8<DT>(a.out, (size_t)m * a.N + n, v);
  }
};

// Largest magnitude so far: a NaN stays.
__device__ __forceinline__ float amax_nan(float a, float b) { return b > a || b != b ? b : a; }

// A block quantises a row: 16 values a thread at a time, twice over the row (its
// absmax, then the codes, from the L2).  A NaN or an infinity makes the scale NaN
// and the codes zeros, so the row's outputs are NaN, and no other row's.
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
  const bool fine = am <= 3.402823466e38f;
  am = am < 0x1p-100f ? 0x1p-100f : am;
  const float m = 127.0f / am;
  uint32_t* q = (uint32_t*)(codes + (size_t)t * K);
  for (int c = tid; c < K / N; c += 256) {
    float f[N];
    Chunk<DT>::unpack(p[c], f);
#pragma unroll
    for (int w = 0; w < N / 4; ++w) {
      uint32_t o = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        o |= ((uint32_t)(fine ? (int)rintf(f[4 * w + j] * m) : 0) & 0xFFu) << (8 * j);
      q[c * (N / 4) + w] = o;
    }
  }
  if (tid == 0) scales[t] = fine ? am / 127.0f : __uint_as_float(0x7FC00000u);
}

hipError_t launch_int8_quant(const void* x, int T, int K, int dtype, int8_t* codes, float* scales,
                             hipStream_t s) {
  by_dtype(dtype, [&](auto D) {
    MOE_LAUNCH("int8_quant", s, (k_int8_quant<decltype(D)::value>), dim3((unsigned)T), dim3(256), 0, s, x, K,
               (uint8_t*)codes, scales);
  });
  return hipGetLastError();
}

// Tile shapes, largest first: f with the kernel, BN, BM and threads.
constexpr int kInt8Shapes = 3;
template <class EP, typename F>
static void by_tile(int shape, F&& f) {
  if (shape == 0) f(&k_tile<kElI8, false, false, EP, 256, 256, 2, 2, 128, 2, 3>, 256, 256, 256);
  if (shape == 1) f(&k_tile<kElI8, false, false, EP, 128, 128, 2, 2, 128, 2, 2>, 128, 128, 256);
  if (shape == 2) f(&k_tile<kElI8, false, false, EP, 64, 64, 1, 2, 128, 4, 4>, 64, 64, 128);
}

// The shape whose rounds of 256 blocks take the least time together.
static int tile_shape(int M, int N) {
  constexpr int size[kInt8Shapes] = {256, 128, 64};
  constexpr int cost[kInt8Shapes] = {100, 30, 10};
  int best = 0;
  long least = 0;
  for (int s = 0; s < kInt8Shapes; ++s) {
    const long tiles = (long)((N + size[s] - 1) / size[s]) * ((M + size[s] - 1) / size[s]);
    const long t = (tiles + 255) / 256 * cost[s];
    if (least == 0 || t < least) least = t, best = s;
  }
  return best;
}

void register_int8_kernels(std::vector<const void*>& k) {
  auto add = [&](auto kernel, int, int, int) { k.push_back((const void*)kernel); };
  for (int dt = MOE_DT_BF16; dt <= MOE_DT_F32; ++dt)
    by_dtype(dt, [&](auto D) {
      constexpr int DT = decltype(D)::value;
      k.push_back((const void*)&k_int8_quant<DT>);
      for (int s = 0; s < kInt8Shapes; ++s) {
        by_tile<PutInt8<DT>>(s, add);
        by_tile<PutInt8Gated<DT>>(s, add);
      }
    });
}

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

uint64_t int8_linear_threads(int T, int N) {
  return std::max<uint64_t>((uint64_t)((T + 63) / 64) * ((N + 63) / 64) * 128, (uint64_t)T * 256);
}

size_t int8_linear_workspace_bytes(int T, int N, int K) {
  return up256((size_t)T * K) + up256((size_t)T * sizeof(float));
}

hipError_t launch_int8_linear(const moe_int8_matrix& W, const void* x, int T, int dtype, int gated,
                              void* out, void* ws, hipStream_t s) {
  int8_t* q = (int8_t*)ws;
  float* sx = (float*)((char*)ws + up256((size_t)T * W.K));
  hipError_t e = launch_int8_quant(x, T, W.K, dtype, q, sx, s);
  if (e != hipSuccess) return e;
  TileArgs16 a{};
  a.a = q;
  a.b = W.codes;
  a.lda = a.ldb = (uint32_t)W.K;
  a.M = T;
  a.N = gated ? W.N / 2 : W.N;
  a.K = W.K;
  a.out = out;
  a.sm = sx;
  a.sn = W.scales;
  by_dtype(dtype, [&](auto D) {
    constexpr int DT = decltype(D)::value;
    auto go = [&](auto kernel, int bn, int bm, int threads) {
      a.nt = (W.N + bn - 1) / bn;
      MOE_LAUNCH("int8_tile", s, kernel, dim3((unsigned)a.nt * (unsigned)((T + bm - 1) / bm)), dim3(threads), 0, s, a);
    };
    if (gated) by_tile<PutInt8Gated<DT>>(tile_shape(T, W.N), go);
    else by_tile<PutInt8<DT>>(tile_shape(T, W.N), go);
  });
  return hipGetLastError();
}

}  // namespace moe
