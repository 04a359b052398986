// Helpers of the e4m3 products with a scale per block of 128: the
// quantisation of a row's block, the MFMA, and its operand layout.
//
// A row x of K values is cut into blocks of 128.  With a = max(absmax, 2^-100)
// of a block (NaN apart), its codes are q = e4m3(x * (448 / a)) and its scale
// is s = a / 448 (each operation rounded to f32; the largest magnitude becomes
// 448 exactly or a last place above it, which rounds to 448, so nothing
// saturates).  The floor 2^-100 keeps 448 / a finite for blocks of zeros and
// of the smallest numbers, which become codes of 0.  A NaN is the code NaN; an
// infinity makes a infinite and its own code NaN, so either makes the row's
// outputs NaN and touches no other row.
#pragma once

#include "moe_ffn_common.hpp"
#include "moe_vec.hpp"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kQB = 128;  // values per scale

__device__ __forceinline__ float q_floor(float amax) { return fmaxf(amax, 0x1p-100f); }

// Four f32 -> four e4m3 codes, nearest even.
__device__ __forceinline__ uint32_t fp8x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

__device__ __forceinline__ i32x8 join8(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w,
               (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// Operands of the product of 16 weight rows and 16 token rows over one block
// of 128: lane l holds 32 codes of row l % 16, both operands of the same 32
// positions of the block (which 32 is the caller's choice for l / 16, the sum
// runs over all of them); the result's lane l has rows 4 (l / 16) .. + 3 of
// token l % 16.
//
// EXACT = false: the 128-wide f8 MFMA.  Measured on gfx950: it adds each run of
// 8 codes after aligning their products to the run's largest exponent E and
// cutting them below 2^(E - 13), and adds the runs in f32.  Only products less
// than 2^-6 of their run's largest lose bits; over normally distributed rows
// the result is off by 5e-6 of its norm, which the rounding of the output to
// bf16 (2e-3) or f16 (2e-4) covers.
// EXACT = true, for rows of f32: the codes as f16 (exact) on the f16 MFMA, whose
// sums of such products came out exact: half the rate.
template <bool EXACT>
struct Frag;
template <>
struct Frag<false> {
  i32x8 v;
  __device__ __forceinline__ void set(i32x8 c) { v = c; }
};
template <>
struct Frag<true> {
  f16x8 v[4];
  __device__ __forceinline__ void set(i32x8 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const u32x2 a = fp8x4_to_f16((uint32_t)c[2 * i]), b = fp8x4_to_f16((uint32_t)c[2 * i + 1]);
      v[i] = __builtin_bit_cast(f16x8, u32x4{a.x, a.y, b.x, b.y});
    }
  }
};

__device__ __forceinline__ f32x4 mfma128(const Frag<false>& w, const Frag<false>& t) {
  // the unscaled form: no block scales of the instruction's own
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, t.v, f32x4{0.f, 0.f, 0.f, 0.f}, 0,
                                                          0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma128(const Frag<true>& w, const Frag<true>& t) {
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.v[i], t.v[i], acc, 0, 0, 0);
  return acc;
}

}  // namespace moe
