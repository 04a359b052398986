// 16-byte chunks of the element types the training and norm operators take
// (moe_dtype of the public header): a chunk holds 8 values of bf16 or f16, or
// 4 of f32.  Arithmetic is in f32; store() rounds once, to nearest even.
#pragma once

#include <math.h>

#include "../../include/moe_nvfp4.h"
#include "moe_device.hpp"

namespace moe {

template <int DT>
struct Chunk;

template <>
struct Chunk<MOE_DT_BF16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(u32x4 v, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = bf16_bits_to_f32(v[j] & 0xFFFFu);
      f[2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[8]) {
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
    return v;
  }
};

template <>
struct Chunk<MOE_DT_F16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(u32x4 v, float (&f)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(v[j] & 0xFFFFu));
      f[2 * j + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(v[j] >> 16));
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[8]) {
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f[2 * j]) |
             ((uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f[2 * j + 1]) << 16);
    return v;
  }
};

template <>
struct Chunk<MOE_DT_F32> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(u32x4 v, float (&f)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = __uint_as_float(v[j]);
  }
  static __device__ __forceinline__ u32x4 pack(const float (&f)[4]) {
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __float_as_uint(f[j]);
    return v;
  }
};

// c = sigmoid(g) and 1 - c, each to a few units of its last place: 1 - c taken from
// c would lose its bits for a positive g (all of them from 17.4 on).
__device__ __forceinline__ float sigmoid_f32(float g) { return 1.0f / (1.0f + expf(-g)); }
__device__ __forceinline__ float sigmoid_rest_f32(float g) { return 1.0f / (1.0f + expf(g)); }

// Host side: bytes of one element of a moe_dtype, and the call of a generic
// lambda with the type as a compile-time constant.
inline int dtype_bytes(int dt) { return dt == MOE_DT_F32 ? 4 : 2; }
template <int V>
using IntC = std::integral_constant<int, V>;
template <typename F>
inline void by_dtype(int dt, F&& f) {
  if (dt == MOE_DT_BF16) f(IntC<MOE_DT_BF16>{});
  else if (dt == MOE_DT_F16) f(IntC<MOE_DT_F16>{});
  else f(IntC<MOE_DT_F32>{});
}

// How a grid covers T rows of cpr 16-byte chunks: 2^lg threads to a row, 2^(8-lg)
// rows to a block, cb blocks side by side along the row.  Nothing is divided
// per thread, and from 64 chunks on a wave has one token only, whose
// positions and weights are then scalar loads.
struct RowGrid {
  int lg, cb;
  unsigned blocks;
};

// This thread's token and chunk; false outside.
__device__ __forceinline__ bool row_chunk(unsigned block, int lg, int cb, int T, int cpr, int* t, int* c) {
  const int rb = (int)(block / (unsigned)cb), seg = (int)(block % (unsigned)cb);
  int sub = (int)threadIdx.x >> lg;
  if (lg >= 6) sub = __builtin_amdgcn_readfirstlane(sub);
  *t = (rb << (8 - lg)) + sub;
  *c = (seg << 8) + ((int)threadIdx.x & ((1 << lg) - 1));
  return *t < T && *c < cpr;
}

inline unsigned blocks(long n, int per) { return (unsigned)((n + per - 1) / per); }

inline RowGrid row_grid(int T, int cpr) {
  RowGrid g;
  g.lg = 0;
  while (g.lg < 8 && (1 << g.lg) < cpr) ++g.lg;
  g.cb = (cpr + 255) / 256;
  g.blocks = blocks(T, 256 >> g.lg) * (unsigned)g.cb;
  return g;
}
inline uint64_t row_grid_threads(int T, int cpr) {
  const RowGrid g = row_grid(1, cpr);
  return (uint64_t)blocks(T, 256 >> g.lg) * (uint64_t)g.cb * 256;
}

}  // namespace moe
