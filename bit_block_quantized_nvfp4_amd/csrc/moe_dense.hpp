// What the dense block's two directions share: the plain epilogue and the launch of one
// product.
#pragma once

#include "moe_tile.hpp"

namespace moe {

template <int DT>
struct PutLinear {
  static constexpr bool kGated = false;
  typedef NoPre Pre;
  template <int C>
  static __device__ __forceinline__ void put(const TileArgs16& a, int m, int n, const float (&v)[C],
                                             const float (&)[C], const Pre&) {
    put_row<DT>(a.out, (size_t)m * a.N + n, v);
  }
};

template <int DT, bool BROWS, class EP>
static hipError_t product(const char* name, TileArgs16 a, hipStream_t s) {
  const int cols = EP::kGated ? 2 * a.N : a.N, best = tile_shape(a.M, cols, steps_of(a.K, 2));
  by_shape(best, [&](auto shape) {
    a.nt = (cols + shape.BN - 1) / shape.BN;
    MOE_LAUNCH(name, s, (k_tile<DT, BROWS, false, EP, decltype(shape)>), dim3((unsigned)tiles_of(best, a.M, cols)),
               dim3(shape.kThreads), 0, s, a);
  });
  return hipGetLastError();
}

template <typename F>
static void by_half(int dt, F&& f) {
  if (dt == MOE_DT_BF16) f(IntC<MOE_DT_BF16>{});
  else f(IntC<MOE_DT_F16>{});
}

inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace moe
