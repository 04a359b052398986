// The dense gated feed-forward block in 16 bits and its gradients:
//
//   g = x Wg^T, u = x Wu^T, h = silu(g) u, y = h Wd^T
//   dh = dy Wd, dg = dh u s (1 + g (1 - s)), du = dh g s   with s = sigmoid(g)
//   dx = [dg du] Wgu, dWgu = [dg du]^T x, dWd = dy^T h
//
// Seven products in two (forward) and four launches of the tiles of moe_tile.hpp.
// The activation and its gradient are epilogues: both projections of an output
// come from one block, which holds gate and up rows side by side, and dh never
// leaves the block that computes it.  h, dg and du are operands of the next
// product and rounded to the rows' type for that, as every operand of a 16-bit
// product is; all sums and the activation are in f32.
#include "moe_tile.hpp"

namespace moe {

template <int DT>
struct PutLinear {
  static constexpr bool kGated = false;
  typedef NoPre Pre;
  static __device__ __forceinline__ void put(const TileArgs16& a, int m, int n, const float (&v)[8],
                                             const float (&)[8], const Pre&) {
    put8<DT>(a.out, (size_t)m * a.N + n, v);
  }
};

// h, and (KEEP) the projections, [M][2N]
template <int DT, bool KEEP>
struct PutGated {
  static constexpr bool kGated = true;
  typedef NoPre Pre;
  static __device__ __forceinline__ void put(const TileArgs16& a, int m, int n, const float (&v)[8],
                                             const float (&u)[8], const Pre&) {
    float h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = silu_f32(v[e]) * u[e];
    put8<DT>(a.out, (size_t)m * a.N + n, h);
    if (KEEP) {
      put8<DT>(a.out2, (size_t)m * 2 * a.N + n, v);
      put8<DT>(a.out2, (size_t)m * 2 * a.N + a.N + n, u);
    }
  }
};

// From dh and the projections aux [M][2N]: their gradients [M][2N], and h again
template <int DT>
struct PutGatedGrad {
  static constexpr bool kGated = false;
  struct Pre {
    u32x4 g, u;
    __device__ __forceinline__ void get(const TileArgs16& a, int m, int n) {
      const uint16_t* p = (const uint16_t*)a.aux + (size_t)m * 2 * a.N + n;
      g = *(const u32x4*)p;
      u = *(const u32x4*)(p + a.N);
    }
  };
  static __device__ __forceinline__ void put(const TileArgs16& a, int m, int n, const float (&v)[8],
                                             const float (&)[8], const Pre& pre) {
    const size_t at = (size_t)m * 2 * a.N + n;
    float g[8], u[8], h[8], dg[8], du[8];
    Chunk<DT>::unpack(pre.g, g);
    Chunk<DT>::unpack(pre.u, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // e = exp(-g), s = 1 / (1 + e), 1 - s = e s: no difference that would lose its
      // bits (with e infinite s is 0, and so is what 1 - s is multiplied with)
      const float e = __builtin_amdgcn_exp2f(g[i] * -1.4426950408889634f);
      const float s = __builtin_amdgcn_rcpf(1.0f + e);
      const float gs = g[i] * s;
      h[i] = gs * u[i];
      du[i] = v[i] * gs;
      dg[i] = v[i] * u[i] * fmaf(gs, fminf(e, 0x1p100f) * s, s);
    }
    put8<DT>(a.out, at, dg);
    put8<DT>(a.out, at + a.N, du);
    put8<DT>(a.out2, (size_t)m * a.N + n, h);
  }
};

// Tile shapes, largest first: f with the kernel, BN, BM and threads.
constexpr int kDenseShapes = 3;
template <int DT, bool BROWS, bool AROWS, class EP, typename F>
static void by_tile(int shape, F&& f) {
  if (shape == 0) f(&k_tile<DT, BROWS, AROWS, EP, 256, 256, 2, 2, 128, 2, 3>, 256, 256, 256);
  if (shape == 1) f(&k_tile<DT, BROWS, AROWS, EP, 128, 128, 2, 2, 128, 2, 2>, 128, 128, 256);
  if (shape == 2) f(&k_tile<DT, BROWS, AROWS, EP, 64, 64, 1, 2, 128, 4, 4>, 64, 64, 128);
}

// The shape whose rounds of 256 blocks take the least time together.
static int tile_shape(int M, int N) {
  constexpr int size[kDenseShapes] = {256, 128, 64};
  constexpr int cost[kDenseShapes] = {100, 30, 10};
  int best = 0;
  long least = 0;
  for (int s = 0; s < kDenseShapes; ++s) {
    const long tiles = (long)((N + size[s] - 1) / size[s]) * ((M + size[s] - 1) / size[s]);
    const long t = (tiles + 255) / 256 * cost[s];
    if (least == 0 || t < least) least = t, best = s;
  }
  return best;
}

template <int DT, bool BROWS, bool AROWS, class EP>
static hipError_t product(const char* name, TileArgs16 a, hipStream_t s) {
  const int cols = EP::kGated ? 2 * a.N : a.N;
  by_tile<DT, BROWS, AROWS, EP>(tile_shape(a.M, cols), [&](auto kernel, int bn, int bm, int threads) {
    a.nt = (cols + bn - 1) / bn;
    MOE_LAUNCH(name, s, kernel, dim3((unsigned)a.nt * (unsigned)((a.M + bm - 1) / bm)), dim3(threads), 0, s, a);
  });
  return hipGetLastError();
}

template <typename F>
static void by_half(int dt, F&& f) {
  if (dt == MOE_DT_BF16) f(IntC<MOE_DT_BF16>{});
  else f(IntC<MOE_DT_F16>{});
}

void register_dense_kernels(std::vector<const void*>& k) {
  auto add = [&](auto kernel, int, int, int) { k.push_back((const void*)kernel); };
  for (int dt : {MOE_DT_BF16, MOE_DT_F16})
    by_half(dt, [&](auto D) {
      constexpr int DT = decltype(D)::value;
      for (int s = 0; s < kDenseShapes; ++s) {
        by_tile<DT, false, false, PutGated<DT, false>>(s, add);
        by_tile<DT, false, false, PutGated<DT, true>>(s, add);
        by_tile<DT, false, false, PutLinear<DT>>(s, add);
        by_tile<DT, true, false, PutGatedGrad<DT>>(s, add);
        by_tile<DT, true, false, PutLinear<DT>>(s, add);
        by_tile<DT, true, true, PutLinear<DT>>(s, add);
      }
    });
}

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Blocks of 64 x 64 at most, or fewer, larger ones, of at most eight threads a row
// and column of 64.
uint64_t dense_threads(int T, int H, int I) {
  const uint64_t rows = std::max({T, H, 2 * I}), cols = std::max(H, 2 * I);
  return (rows + 63) / 64 * ((cols + 63) / 64) * 128;
}

size_t dense_ffn_workspace_bytes(int T, int H, int I) { return up256((size_t)T * I * 2); }
size_t dense_ffn_grad_workspace_bytes(int T, int H, int I) {
  return up256((size_t)T * 2 * I * 2) + up256((size_t)T * I * 2);
}

hipError_t launch_dense_ffn(const moe_dense_weights& W, const void* x, int T, void* y, void* gu,
                            void* ws, hipStream_t s) {
  hipError_t e = hipSuccess;
  by_half(W.dtype, [&](auto D) {
    constexpr int DT = decltype(D)::value;
    TileArgs16 a{};
    a.a = x;
    a.b = W.gu;
    a.lda = a.ldb = (uint32_t)W.H * 2;
    a.M = T;
    a.N = W.I;
    a.K = W.H;
    a.out = ws;
    a.out2 = gu;
    e = gu ? product<DT, false, false, PutGated<DT, true>>("dense_gate_up", a, s)
           : product<DT, false, false, PutGated<DT, false>>("dense_gate_up", a, s);
    if (e != hipSuccess) return;
    a.a = ws;
    a.b = W.dn;
    a.lda = a.ldb = (uint32_t)W.I * 2;
    a.N = W.H;
    a.K = W.I;
    a.out = y;
    e = product<DT, false, false, PutLinear<DT>>("dense_down", a, s);
  });
  return e;
}

hipError_t launch_dense_ffn_grad(const moe_dense_weights& W, const void* dy, const void* x,
                                 const void* gu, int T, void* dx, void* dw_gu, void* dw_dn,
                                 void* ws, hipStream_t s) {
  void* dgu = ws;
  void* h = (char*)ws + up256((size_t)T * 2 * W.I * 2);
  const uint32_t hb = (uint32_t)W.H * 2, ib = (uint32_t)W.I * 2;
  hipError_t e = hipSuccess;
  by_half(W.dtype, [&](auto D) {
    constexpr int DT = decltype(D)::value;
    TileArgs16 a{};
    a.a = dy;  // dh = dy Wd, then the activation's gradient
    a.lda = hb;
    a.b = W.dn;
    a.ldb = ib;
    a.M = T;
    a.N = W.I;
    a.K = W.H;
    a.aux = gu;
    a.out = dgu;
    a.out2 = h;
    e = product<DT, true, false, PutGatedGrad<DT>>("dense_down_grad", a, s);
    if (e != hipSuccess) return;
    a = TileArgs16{};
    a.a = dgu;  // dx = dgu Wgu
    a.lda = 2 * ib;
    a.b = W.gu;
    a.ldb = hb;
    a.M = T;
    a.N = W.H;
    a.K = 2 * W.I;
    a.out = dx;
    e = product<DT, true, false, PutLinear<DT>>("dense_dx", a, s);
    if (e != hipSuccess) return;
    a = TileArgs16{};
    a.a = dgu;  // dWgu = dgu^T x
    a.lda = 2 * ib;
    a.b = x;
    a.ldb = hb;
    a.M = 2 * W.I;
    a.N = W.H;
    a.K = T;
    a.out = dw_gu;
    e = product<DT, true, true, PutLinear<DT>>("dense_dw_gu", a, s);
    if (e != hipSuccess) return;
    a.a = dy;  // dWd = dy^T h
    a.lda = hb;
    a.b = h;
    a.ldb = ib;
    a.M = W.H;
    a.N = W.I;
    a.out = dw_dn;
    e = product<DT, true, true, PutLinear<DT>>("dense_dw_dn", a, s);
  });
  return e;
}

}  // namespace moe
