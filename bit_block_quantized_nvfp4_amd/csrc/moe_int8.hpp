// Helpers of the 8-bit integer products: the quantisation of a row and the epilogues.
//
// A row x has one scale: a = max(absmax, 2^-100), s = a / 127, codes rne(x (127 / a)),
// each operation rounded to f32.  The largest magnitude becomes 127 exactly or a last
// place beside it, which rounds to 127.  The floor keeps 127 / a finite for rows of
// zeros and of the smallest numbers, which become codes of 0.  A NaN or an infinity makes
// the scale NaN and the codes 0: the row's outputs are NaN, and no other row's.
#pragma once

#include "moe_tile.hpp"

namespace moe {

// Largest magnitude so far: a NaN stays.
__device__ __forceinline__ float amax_nan(float a, float b) { return b > a || b != b ? b : a; }
__device__ __forceinline__ void int8_scale(float amax, float* mul, float* scale, bool* fine) {
  *fine = amax <= 3.402823466e38f;
  const float a = amax < 0x1p-100f ? 0x1p-100f : amax;
  *mul = 127.0f / a;
  *scale = *fine ? a / 127.0f : __uint_as_float(0x7FC00000u);
}
// Four codes.
__device__ __forceinline__ uint32_t int8x4(const float* f, float mul, bool fine) {
  uint32_t o = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) o |= ((uint32_t)(fine ? (int)rintf(f[j] * mul) : 0) & 0xFFu) << (8 * j);
  return o;
}

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

// The scale of an output's row.
struct RowScale {
  float s;
  __device__ __forceinline__ void get(const TileArgs16& a, int m, int) { s = a.sm[m]; }
};

template <int DT>
struct PutInt8 {
  static constexpr bool kGated = false;
  typedef RowScale Pre;
  template <int C>
  static __device__ __forceinline__ void put(const TileArgs16& a, int m, int n, float (&v)[C],
                                             const float (&)[C], const Pre& row) {
#pragma unroll
    for (int e = 0; e < C; ++e) v[e] = scaled(v[e], row.s, a.sn[n + e]);
    put_row<DT>(a.out, (size_t)m * a.N + n, v);
  }
};

template <int DT>
struct PutInt8Gated {
  static constexpr bool kGated = true;
  typedef RowScale Pre;
  template <int C>
  static __device__ __forceinline__ void put(const TileArgs16& a, int m, int n, float (&v)[C],
                                             const float (&u)[C], const Pre& row) {
#pragma unroll
    for (int e = 0; e < C; ++e)
      v[e] = silu_f32(scaled(v[e], row.s, a.sn[n + e])) * scaled(u[e], row.s, a.sn[a.N + n + e]);
    put_row<DT>(a.out, (size_t)m * a.N + n, v);
  }
};

}  // namespace moe
