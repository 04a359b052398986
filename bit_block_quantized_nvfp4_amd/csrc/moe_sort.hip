// Token rows into expert order and back, and the gradients of the sort, the
// weighted combine and the routing weights.
//
//   dispatch:        xs[slot_pos[s]] = x[token(s)]
//   dispatch_grad:   dx[t] = sum over t's slots of dxs[slot_pos[s]]
//   combine (typed): out[t] = sum_k w[t][k] y[slot_pos[tK+k]] + c_t y[slot_pos[TK+t]]
//   combine_grad:    dy[p] = w dout[t],  dw = <dout[t], y[p]>,
//                    dgate[t] = c_t (1 - c_t) <dout[t], y[p_shared]>
//   topk_grad:       dlogits[t][ids[t][k]] = w_k (dw_k - sum_j w_j dw_j)
//
// All are bound by memory: every row of x, xs, y, dy is moved once.  Sums are
// f32, in slot order (then the shared expert), with one rounding at the end;
// no sum crosses blocks, so no result depends on timing.  H = 2048, K = 10 + 1
// of 512, where a 1 GB device copy runs at 5.1 TB/s: dispatch of 4096 rows of
// f16 33 us (201 MB, 6.1 TB/s), combine 37 us (5.4 TB/s); of 8192 rows of bf16
// dispatch_grad 67 us (403 MB, 6.0 TB/s), combine_grad 147 us (772 MB, 5.3
// TB/s), topk_grad 6.4 us (17 MB).
#include <math.h>

#include "moe_internal.hpp"
#include "moe_vec.hpp"

namespace moe {

// Limit of the positions a slot may have: routed slots sort below T*K, the
// shared slots after the routed ones, below T*K + T (which fits an int).
__device__ __forceinline__ bool slot_ok(int p, int lim) { return p >= 0 && p < lim; }

// One thread per 16-byte chunk of one token's row (cpr chunks a row, whatever
// the element type): read once, written to every slot of the token.
__global__ __launch_bounds__(256) void k_dispatch(const u32x4* __restrict__ x,
                                                  const int32_t* __restrict__ slot_pos, int T,
                                                  int K, int cpr, int lg, int cb, int has_shared,
                                                  u32x4* __restrict__ xs) {
  int t, c;
  if (!row_chunk(blockIdx.x, lg, cb, T, cpr, &t, &c)) return;
  const int TK = T * K;
  const u32x4 v = x[(size_t)t * cpr + c];
  const int32_t* sp = slot_pos + (size_t)t * K;
  for (int k = 0; k < K; ++k) {
    const int p = sp[k];
    if (slot_ok(p, TK)) xs[(size_t)p * cpr + c] = v;
  }
  if (has_shared) {
    const int p = slot_pos[(size_t)TK + t];
    if (slot_ok(p, TK + T)) xs[(size_t)p * cpr + c] = v;
  }
}

// Sum of a token's slot rows, one thread per 16-byte chunk.  w == nullptr:
// plain sum (the gradient of dispatch).
template <int DT>
__global__ __launch_bounds__(256) void k_slot_sum(const u32x4* __restrict__ y,
                                                  const float* __restrict__ w,
                                                  const int32_t* __restrict__ slot_pos,
                                                  const float* __restrict__ gate, int T, int K,
                                                  int cpr, int lg, int cb, int has_shared,
                                                  u32x4* __restrict__ out) {
  constexpr int N = Chunk<DT>::N;
  int t, c;
  if (!row_chunk(blockIdx.x, lg, cb, T, cpr, &t, &c)) return;
  const int TK = T * K;
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  const int ps = has_shared ? slot_pos[(size_t)TK + t] : -1;
  // batches of 12 slots: positions and weights, then the rows (row 0 for a slot
  // that is skipped: a load without a branch), then the sums in slot order
  for (int k0 = 0; k0 < K; k0 += 12) {
    int p[12];
    float wt[12];
#pragma unroll
    for (int j = 0; j < 12; ++j) {
      const int k = k0 + j;
      p[j] = (k < K) ? slot_pos[(size_t)t * K + k] : -1;
      wt[j] = (w && k < K) ? w[(size_t)t * K + k] : 1.f;
    }
    u32x4 v[12];
#pragma unroll
    for (int j = 0; j < 12; ++j)
      if (k0 + j < K)
        v[j] = __builtin_nontemporal_load(y + (size_t)(slot_ok(p[j], TK) ? p[j] : 0) * cpr + c);
#pragma unroll
    for (int j = 0; j < 12; ++j) {
      if (slot_ok(p[j], TK)) {
        float f[N];
        Chunk<DT>::unpack(v[j], f);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(wt[j], f[i], acc[i]);
      }
    }
  }
  if (slot_ok(ps, TK + T)) {
    const float sg = gate ? sigmoid_f32(gate[t]) : 1.0f;
    float f[N];
    Chunk<DT>::unpack(y[(size_t)ps * cpr + c], f);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = fmaf(sg, f[i], acc[i]);
  }
  out[(size_t)t * cpr + c] = Chunk<DT>::pack(acc);
}

// One wave per slot row: dy = weight * dout, and the dot product <dout, y>
// reduced over the wave in a fixed order.
template <int DT, bool PAST>
__global__ __launch_bounds__(256) void k_combine_grad(
    const u32x4* __restrict__ dout, const u32x4* __restrict__ y, const float* __restrict__ w,
    const int32_t* __restrict__ slot_pos, const float* __restrict__ gate, int T, int K, int cpr,
    int has_shared, u32x4* __restrict__ dy, float* __restrict__ dw,
    float* __restrict__ dgate) {
  constexpr int N = Chunk<DT>::N;
  const int lane = threadIdx.x & 63;
  const int SP = K + has_shared;  // slots per token
  const unsigned row =
      blockIdx.x * 4u + (unsigned)__builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int t = (int)(row / (unsigned)SP), k = (int)(row % (unsigned)SP);
  if (t >= T) return;
  const int TK = T * K;
  const bool shared = k == K;
  const int p = shared ? slot_pos[(size_t)TK + t] : slot_pos[(size_t)t * K + k];
  const bool on = slot_ok(p, shared ? TK + T : TK);
  float wt = 1.f, rest = 0.f;
  if (!shared) wt = w[(size_t)t * K + k];
  else if (gate) {
    wt = sigmoid_f32(gate[t]);
    rest = sigmoid_rest_f32(gate[t]);
  }
  float dot = 0.f;
  if (on) {
    const u32x4* dr = dout + (size_t)t * cpr;
    const u32x4* yr = y + (size_t)p * cpr;
    u32x4* dyr = dy + (size_t)p * cpr;
    for (int c0 = 0; c0 < cpr; c0 += 256) {
      u32x4 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + 64 * i + lane;
        if (c < cpr) {
          a[i] = dr[c];
          b[i] = __builtin_nontemporal_load(yr + c);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + 64 * i + lane;
        if (c < cpr) {
          float fa[N], fb[N];
          Chunk<DT>::unpack(a[i], fa);
          Chunk<DT>::unpack(b[i], fb);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            dot = fmaf(fa[j], fb[j], dot);
            fa[j] *= wt;
          }
          if (PAST) __builtin_nontemporal_store(Chunk<DT>::pack(fa), dyr + c);
          else dyr[c] = Chunk<DT>::pack(fa);
        }
      }
    }
  }
  dot = wave_sum_dpp(dot);
  if (lane == 0) {
    if (!shared) dw[(size_t)t * K + k] = dot;
    else if (gate) dgate[t] = wt * rest * dot;
  }
}

// One wave per token.  Lanes k < K hold the slots' gradients; a lane adds up
// those of the slots that name its expert too (a caller may name one twice), in
// slot order, and puts the sum into the row of zeros that the wave keeps in LDS
// and then stores as 16 bytes a lane (VEC: E a multiple of 4) or 4.
template <bool VEC>
__global__ __launch_bounds__(256) void k_topk_grad(const int32_t* __restrict__ ids,
                                                   const float* __restrict__ w,
                                                   const float* __restrict__ dw, int T, int E,
                                                   int K, float* __restrict__ dlogits) {
  __shared__ f32x4 rows[4][256];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const long t = (long)blockIdx.x * 4 + wv;
  if (t >= T) return;
  int id = -1;
  float wk = 0.f, g = 0.f;
  if (lane < K) {
    id = ids[t * K + lane];
    wk = w[t * K + lane];
    g = dw[t * K + lane];
  }
  const int nv = (E + 3) / 4;
  for (int e = lane; e < nv; e += 64) rows[wv][e] = f32x4{0.f, 0.f, 0.f, 0.f};
  const float mean = wave_sum_dpp(wk * g);
  g = wk * (g - mean);
  float sum = 0.f;
  for (int k = 0; k < K; ++k) {
    const int ik = __builtin_amdgcn_readlane(id, k);
    const float gk = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), k));
    if (ik == id) sum += gk;
  }
  // a wave's LDS operations keep their order
  __builtin_amdgcn_wave_barrier();
  if (id >= 0 && id < E) ((float*)rows[wv])[id] = sum;
  __builtin_amdgcn_wave_barrier();
  float* row = dlogits + t * E;
  if (VEC)
    for (int e = lane; e < nv; e += 64) ((f32x4*)row)[e] = rows[wv][e];
  else
    for (int e = lane; e < E; e += 64) row[e] = ((const float*)rows[wv])[e];
}

void register_sort_kernels(std::vector<const void*>& k) {
  k.push_back((const void*)&k_dispatch);
  k.push_back((const void*)&k_topk_grad<true>);
  k.push_back((const void*)&k_topk_grad<false>);
  for (int dt = MOE_DT_BF16; dt <= MOE_DT_F32; ++dt)
    by_dtype(dt, [&](auto D) {
      k.push_back((const void*)&k_slot_sum<decltype(D)::value>);
      k.push_back((const void*)&k_combine_grad<decltype(D)::value, false>);
      k.push_back((const void*)&k_combine_grad<decltype(D)::value, true>);
    });
}

uint64_t slot_rows_threads(int T, int H, int dtype) {
  return row_grid_threads(T, H * dtype_bytes(dtype) / 16);
}

hipError_t launch_dispatch(const void* x, const int32_t* slot_pos, int T, int K, int H,
                           int has_shared, int dtype, void* xs, hipStream_t s) {
  const int cpr = H * dtype_bytes(dtype) / 16;
  const RowGrid g = row_grid(T, cpr);
  MOE_LAUNCH("dispatch", s, k_dispatch, dim3(g.blocks), dim3(256), 0, s, (const u32x4*)x,
             slot_pos, T, K, cpr, g.lg, g.cb, has_shared, (u32x4*)xs);
  return hipGetLastError();
}

hipError_t launch_slot_sum(const void* y, const float* w, const int32_t* slot_pos,
                           const float* gate, int T, int K, int H, int has_shared, int dtype,
                           void* out, hipStream_t s) {
  const int cpr = H * dtype_bytes(dtype) / 16;
  const RowGrid g = row_grid(T, cpr);
  by_dtype(dtype, [&](auto D) {
    MOE_LAUNCH(w ? "combine" : "dispatch_grad", s, k_slot_sum<decltype(D)::value>,
               dim3(g.blocks), dim3(256), 0, s, (const u32x4*)y, w, slot_pos, gate, T, K, cpr,
               g.lg, g.cb, has_shared, (u32x4*)out);
  });
  return hipGetLastError();
}

hipError_t launch_combine_grad(const void* dout, const void* y, const float* w,
                               const int32_t* slot_pos, const float* gate, int T, int K, int H,
                               int has_shared, int dtype, void* dy, float* dw, float* dgate,
                               hipStream_t s) {
  const int cpr = H * dtype_bytes(dtype) / 16;
  // Rows of dy that the 256 MB last-level cache cannot hold anyway are stored
  // past it (T = 8192, K = 10 + 1, H = 2048 bf16, 369 MB: 148 us and 67 us for
  // the dispatch_grad that follows, instead of 155 us and 84 us); fewer stay
  // there for whoever reads them next.
  const bool past = (size_t)T * (K + has_shared) * cpr * 16 > (size_t)256 << 20;
  by_dtype(dtype, [&](auto D) {
    constexpr int DT = decltype(D)::value;
    MOE_LAUNCH("combine_grad", s, (past ? k_combine_grad<DT, true> : k_combine_grad<DT, false>),
               dim3(blocks((long)T * (K + has_shared), 4)), dim3(256), 0, s, (const u32x4*)dout,
               (const u32x4*)y, w, slot_pos, gate, T, K, cpr, has_shared, (u32x4*)dy, dw, dgate);
  });
  return hipGetLastError();
}

hipError_t launch_topk_grad(const int32_t* ids, const float* w, const float* dw, int T, int E,
                            int K, float* dlogits, hipStream_t s) {
  // rows of 16 bytes need E a multiple of 4 and an aligned start
  const bool vec = E % 4 == 0 && ((uintptr_t)dlogits & 15) == 0;
  MOE_LAUNCH("topk_grad", s, vec ? k_topk_grad<true> : k_topk_grad<false>, dim3(blocks(T, 4)),
             dim3(256), 0, s, ids, w, dw, T, E, K, dlogits);
  return hipGetLastError();
}

}  // namespace moe
