// The dense gated feed-forward block in 16 bits:
//
//   g = x Wg^T, u = x Wu^T, h = silu(g) u, y = h Wd^T
//
// in two launches of the tiles of moe_tile.hpp (up to 16 rows: of moe_stream.hpp).  The
// activation is an epilogue: both projections of an output come from one block, which
// holds gate and up rows side by side.  h is the next product's operand and rounded to the
// rows' type for that, as every operand of a 16-bit product is; all sums and the
// activation are in f32.
//
// 8192 rows, H = 2048, I = 8192, bf16: 471 us (with the projections kept, whose 403 MB the
// epilogue writes) and 205 us, one after the other; 333 rows, 2056, 1032, f16: 13.3 and 7.8 us, by
// latency; 1 row, 2048, 8192: 13.4 and 8.5 us, the weights from memory at 5.0 and 3.9 TB/s.
#include "moe_dense.hpp"
#include "moe_stream.hpp"

namespace moe {

// h, and (KEEP) the projections, [M][2N]
template <int DT, bool KEEP>
struct PutGated {
  static constexpr bool kGated = true;
  typedef NoPre Pre;
  template <int C>
  static __device__ __forceinline__ void put(const TileArgs16& a, int m, int n, const float (&v)[C],
                                             const float (&u)[C], const Pre&) {
    float h[C];
#pragma unroll
    for (int e = 0; e < C; ++e) h[e] = silu_f32(v[e]) * u[e];
    put_row<DT>(a.out, (size_t)m * a.N + n, h);
    if (KEEP) {
      put_row<DT>(a.out2, (size_t)m * 2 * a.N + n, v);
      put_row<DT>(a.out2, (size_t)m * 2 * a.N + a.N + n, u);
    }
  }
};

// Up to 16 rows stream the weights.  The shapes: f with the kernel, outputs and threads of
// a block (1 row of 2048 x 8192, us: 8 waves along K 15.8, 16 waves 13.7; four pieces ahead
// instead of two 12.8, but for 2048 x 512 4.1 instead of 3.3).
template <int DT, class EP, typename F>
static void by_stream(int M, int N, int K, F&& f) {
  const bool half = takes_half(M, N, EP::kGated);
  if constexpr (EP::kGated) {
    if (half) f(&k_stream<DT, kXOperand, EP, 2, 8, 2, true>, 8, 512);
    else f(&k_stream<DT, kXOperand, EP, 2, 8, 2>, 16, 512);
  } else {
    if (half) f(&k_stream<DT, kXOperand, EP, 1, 8, 2, true>, 8, 512);
    else if (K >= 4096) f(&k_stream<DT, kXOperand, EP, 1, 16, 4>, 16, 1024);
    else f(&k_stream<DT, kXOperand, EP, 1, 16, 2>, 16, 1024);
  }
}

template <int DT, class EP>
static hipError_t few_rows(const char* name, const TileArgs16& a, hipStream_t s) {
  by_stream<DT, EP>(a.M, a.N, a.K, [&](auto kernel, int outs, int threads) {
    MOE_LAUNCH(name, s, kernel, dim3((unsigned)((a.N + outs - 1) / outs)), dim3(threads), 0, s, a);
  });
  return hipGetLastError();
}

// One of the forward pass's products, whose operands both have k fastest.
template <int DT, class EP>
static hipError_t forward(const char* name, const TileArgs16& a, hipStream_t s) {
  if (a.M <= kStreamRows) return few_rows<DT, EP>(name, a, s);
  return product<DT, false, EP>(name, a, s);
}

void register_dense_kernels(std::vector<const void*>& k) {
  auto add_stream = [&](auto kernel, int, int) { k.push_back((const void*)kernel); };
  for (int dt : {MOE_DT_BF16, MOE_DT_F16})
    by_half(dt, [&](auto D) {
      constexpr int DT = decltype(D)::value;
      for (int M : {1, kStreamRows})
        for (int K : {8, 65536}) {
          by_stream<DT, PutGated<DT, false>>(M, 8, K, add_stream);
          by_stream<DT, PutGated<DT, true>>(M, 8, K, add_stream);
          by_stream<DT, PutLinear<DT>>(M, 8, K, add_stream);
        }
      for (int i = 0; i < kTileShapes16; ++i)
        by_shape(i, [&](auto shape) {
          typedef decltype(shape) TS;
          k.push_back((const void*)&k_tile<DT, false, false, PutGated<DT, false>, TS>);
          k.push_back((const void*)&k_tile<DT, false, false, PutGated<DT, true>, TS>);
          k.push_back((const void*)&k_tile<DT, false, false, PutLinear<DT>, TS>);
        });
    });
}

uint64_t dense_ffn_threads(int T, int H, int I) {
  if (T <= kStreamRows) return 0;  // at most 65536 / 8 blocks
  return std::max(tile_threads(T, 2 * I, steps_of(H, 2)), tile_threads(T, H, steps_of(I, 2)));
}

size_t dense_ffn_workspace_bytes(int T, int H, int I) { return up256((size_t)T * I * 2); }
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
    e = gu ? forward<DT, PutGated<DT, true>>("dense_gate_up", a, s)
           : forward<DT, PutGated<DT, false>>("dense_gate_up", a, s);
    if (e != hipSuccess) return;
    a.a = ws;
    a.b = W.dn;
    a.lda = a.ldb = (uint32_t)W.I * 2;
    a.N = W.H;
    a.K = W.I;
    a.out = y;
    e = forward<DT, PutLinear<DT>>("dense_down", a, s);
  });
  return e;
}

}  // namespace moe
