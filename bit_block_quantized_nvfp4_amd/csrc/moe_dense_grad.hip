// The gradients of the dense gated feed-forward block (moe_dense.hip):
//
//   dh = dy Wd, dg = dh u s (1 + g (1 - s)), du = dh g s   with s = sigmoid(g)
//   dx = [dg du] Wgu, dWgu = [dg du]^T x, dWd = dy^T h
//
// in two launches of the tiles of moe_tile.hpp.  dh never leaves the block that computes
// it: the activation's gradient is that product's epilogue, which reads the kept
// projections and makes h again.  h, dg and du are operands of the next products and
// rounded to the rows' type for that; all sums and the activation's gradient are in f32.
//
// 8192 rows, H = 2048, I = 8192, bf16: dh 379 us, of which its epilogue takes about 150 to move
// 670 MB, the other three 999 us (1.38 PFLOP/s); 133 rows, 1032, 520, f16: 8.9 and 10.5 us, by
// latency.
#include "moe_dense.hpp"

namespace moe {

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
      // bits.  Finite up to g = -88.7; beyond, s is 0 and e held finite, so that e s is 0
      // and no NaN, and so are all three factors (below 2^-119 there)
      const float e = __builtin_amdgcn_exp2f(g[i] * -1.4426950408889634f);
      const float s = __builtin_amdgcn_rcpf(1.0f + e);
      const float gs = g[i] * s;
      h[i] = gs * u[i];
      du[i] = v[i] * gs;
      dg[i] = v[i] * u[i] * fmaf(gs, fminf(e, 0x1.fffffep127f) * s, s);
    }
    put_row<DT>(a.out, at, dg);
    put_row<DT>(a.out, at + a.N, du);
    put_row<DT>(a.out2, (size_t)m * a.N + n, h);
  }
};

// The three products that follow from dgu and h, in one launch: dx (A's rows run along K,
// B's across), then the weights' gradients (both across).  Small ones would not fill the
// chip one after the other (T = 133, H = 1032, I = 520: 10 us together, 18 apart).
struct GradArgs {
  TileArgs16 dx, dgu, ddn;
  int dx_blocks, dgu_blocks, ddn_blocks;
};
template <int DT, class TS>
__global__ __launch_bounds__(TS::kThreads) void k_dense_grads(GradArgs g) {
  __shared__ __align__(1024) uint8_t lds[TS::kLds];
  const int b = blockIdx.x;
  if (b < g.dx_blocks) {
    tile_block<DT, true, false, PutLinear<DT>, TS>(g.dx, b, g.dx_blocks, (lds_u8*)lds);
  } else {
    const bool first = b < g.dx_blocks + g.dgu_blocks;
    const TileArgs16 a = first ? g.dgu : g.ddn;
    tile_block<DT, true, true, PutLinear<DT>, TS>(a, b - g.dx_blocks - (first ? 0 : g.dgu_blocks),
                                                  first ? g.dgu_blocks : g.ddn_blocks, (lds_u8*)lds);
  }
}
// Their shape: the longest product's tiles, alone on their compute units if those that are as
// long leave room for that, or the rounds of all tiles, each as long as its own steps.
static int grads_shape(const GradArgs& g) {
  int best = 0;
  long least = 0;
  for (int s = 0; s < kTileShapes16; ++s) {
    const TileCost c = tile_cost(s);
    long tiles = 0, work = 0, t = 0;
    for (const TileArgs16* a : {&g.dx, &g.dgu, &g.ddn}) {
      const long n = tiles_of(s, a->M, a->N), steps = steps_of(a->K, 2);
      long as_long = 0;
      for (const TileArgs16* b : {&g.dx, &g.dgu, &g.ddn})
        if (b->K >= a->K) as_long += tiles_of(s, b->M, b->N);
      tiles += n;
      work += n * (c.fixed + steps * c.step);
      t = std::max(t, as_long <= 256 ? c.fixed1 + steps * c.step1 : c.fixed + steps * c.step);
    }
    if (tiles > c.places) t = std::max(t, work / c.places);
    if (least == 0 || t < least) least = t, best = s;
  }
  return best;
}

void register_dense_grad_kernels(std::vector<const void*>& k) {
  for (int dt : {MOE_DT_BF16, MOE_DT_F16})
    by_half(dt, [&](auto D) {
      constexpr int DT = decltype(D)::value;
      for (int i = 0; i < kTileShapes16; ++i)
        by_shape(i, [&](auto shape) {
          typedef decltype(shape) TS;
          k.push_back((const void*)&k_tile<DT, true, false, PutGatedGrad<DT>, TS>);
          k.push_back((const void*)&k_dense_grads<DT, TS>);
        });
    });
}

// The sizes of the three products.
static GradArgs grads_of(int T, int H, int I) {
  GradArgs g{};
  g.dx.M = T, g.dx.N = H, g.dx.K = 2 * I;
  g.dgu.M = 2 * I, g.dgu.N = H, g.dgu.K = T;
  g.ddn.M = H, g.ddn.N = I, g.ddn.K = T;
  return g;
}

uint64_t dense_ffn_grad_threads(int T, int H, int I) {
  const GradArgs g = grads_of(T, H, I);
  const int best = grads_shape(g);
  uint64_t t = tile_threads(T, I, steps_of(H, 2));
  by_shape(best, [&](auto shape) {
    uint64_t tiles = 0;
    for (const TileArgs16* a : {&g.dx, &g.dgu, &g.ddn}) tiles += (uint64_t)tiles_of(best, a->M, a->N);
    t = std::max(t, tiles * shape.kThreads);
  });
  return t;
}

size_t dense_ffn_grad_workspace_bytes(int T, int H, int I) {
  return up256((size_t)T * 2 * I * 2) + up256((size_t)T * I * 2);
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
    e = product<DT, true, PutGatedGrad<DT>>("dense_down_grad", a, s);
    if (e != hipSuccess) return;
    GradArgs g = grads_of(T, W.H, W.I);
    g.dx.a = dgu;  // dx = dgu Wgu
    g.dx.lda = 2 * ib;
    g.dx.b = W.gu;
    g.dx.ldb = hb;
    g.dx.out = dx;
    g.dgu.a = dgu;  // dWgu = dgu^T x
    g.dgu.lda = 2 * ib;
    g.dgu.b = x;
    g.dgu.ldb = hb;
    g.dgu.out = dw_gu;
    g.ddn.a = dy;  // dWd = dy^T h
    g.ddn.lda = hb;
    g.ddn.b = h;
    g.ddn.ldb = ib;
    g.ddn.out = dw_dn;
    const int best = grads_shape(g);
    by_shape(best, [&](auto shape) {
      for (TileArgs16* p : {&g.dx, &g.dgu, &g.ddn}) p->nt = (p->N + shape.BN - 1) / shape.BN;
      g.dx_blocks = (int)tiles_of(best, g.dx.M, g.dx.N);
      g.dgu_blocks = (int)tiles_of(best, g.dgu.M, g.dgu.N);
      g.ddn_blocks = (int)tiles_of(best, g.ddn.M, g.ddn.N);
      MOE_LAUNCH("dense_grads", s, (k_dense_grads<DT, decltype(shape)>),
                 dim3((unsigned)g.dx_blocks + (unsigned)g.dgu_blocks + (unsigned)g.ddn_blocks), dim3(shape.kThreads), 0,
                 s, g);
    });
    e = hipGetLastError();
  });
  return e;
}

}  // namespace moe
