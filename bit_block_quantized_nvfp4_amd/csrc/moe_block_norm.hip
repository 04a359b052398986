// The norms before and after a block, fused with the block's gate and the
// residual scale, and the gradients.  Per row t, with c = 1, sigmoid(g_t) or
// sigmoid(g_th), rms statistics in f32:
//
//   u  = y rstd(y) w_post          (u = y without w_post)
//   r' = a r + b c u               rounded to the rows' type: what is stored
//   n  = r' rstd(r') w_pre         of the stored r'
//
// and backward, with xh = r' rstd(r'), yh = y rstd(y), mean over the H columns:
//
//   D  = dr' + rstd(r') (dn w_pre - xh mean(dn w_pre xh))
//   dr = a D,  du = b c D
//   dg = b c (1 - c) D u           (summed over the row for a token's gate)
//   dy = rstd(y) (du w_post - yh mean(du w_post yh))
//   dw_pre = sum_t dn xh,  dw_post = sum_t du yh
//
// Bound by memory: each row of each tensor is read (non-temporal: 135 us, as
// ordinary loads 144 us at T = 32768, H = 2048 with an element gate) and written
// once, a row's values stay in registers between the statistics and their use.
// H = 2048, bf16: T = 32768 with an element gate 122 us (671 MB, 5.5 TB/s; a 1
// GB device copy runs at 5.1); backward T = 8191 with a token gate 44 us + 4 us
// for the weight gradients (201 MB of rows and 8 MB of partials, 4.8 TB/s).
#include <math.h>

#include "moe_internal.hpp"
#include "moe_vec.hpp"

namespace moe {

// Sum over the threads of a row: one wave, or the W waves of the block (the
// waves' sums join in wave order).  slot: LDS of this reduction alone.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = wave_sum_dpp(v);
  if (W == 1) return v;
  if ((threadIdx.x & 63) == 0) slot[(threadIdx.x >> 6) % W] = v;
  __syncthreads();
  float r = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) r += slot[i];
  return r;
}

// N f32 weights at column c * N.
template <int N>
__device__ __forceinline__ void load_w(const float* __restrict__ w, int c, float (&f)[N]) {
  const f32x4* p = (const f32x4*)w + (size_t)c * (N / 4);
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    const f32x4 v = p[q];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[4 * q + j] = v[j];
  }
}

struct NormFwd {
  const u32x4* res;
  const u32x4* y;       // NULL: r' = res, not written
  const void* gate;     // NULL, f32 [T], or rows of the element type
  const float* w_post;  // NULL: no norm after
  const float* w_pre;   // NULL: no norm before the next block
  u32x4* r_out;
  u32x4* n_out;
  float* rstd_post;
  float* rstd_pre;
  float res_scale, out_scale, eps;
  int T, H, cpr, gate_kind;
};

// W == 1: a wave per row, four rows to a block; else the block's W waves share
// one row.
template <int DT, int NC, int W>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void k_block_norm(NormFwd a) {
  constexpr int N = Chunk<DT>::N;
  constexpr int TPR = 64 * W;
  __shared__ float red[2][W];
  const int lane = W == 1 ? (threadIdx.x & 63) : threadIdx.x;
  const int t = W == 1 ? blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6)
                       : blockIdx.x;
  if (t >= a.T) return;
  const size_t base = (size_t)t * a.cpr;
  float v[NC][N];
  u32x4 rr[NC], yy[NC], gg[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = lane + TPR * i;
    rr[i] = yy[i] = gg[i] = u32x4{0u, 0u, 0u, 0u};
    if (c < a.cpr) {
      if (a.y) yy[i] = __builtin_nontemporal_load(a.y + base + c);
      rr[i] = __builtin_nontemporal_load(a.res + base + c);
      if (a.gate_kind == MOE_GATE_ELEMENT)
        gg[i] = __builtin_nontemporal_load((const u32x4*)a.gate + base + c);
    }
  }
  const float inv_h = 1.0f / (float)a.H;
  if (a.y) {
    float rstd = 1.f;
    if (a.w_post) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        Chunk<DT>::unpack(yy[i], v[i]);
#pragma unroll
        for (int j = 0; j < N; ++j) ss = fmaf(v[i][j], v[i][j], ss);
      }
      rstd = 1.0f / sqrtf(row_sum<W>(ss, red[0]) * inv_h + a.eps);
      if (a.rstd_post && lane == 0) a.rstd_post[t] = rstd;
    }
    float scale = a.out_scale;
    if (a.gate_kind == MOE_GATE_TOKEN) scale *= sigmoid_f32(((const float*)a.gate)[t]);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lane + TPR * i;
      if (c < a.cpr) {
        float r[N], g[N], wp[N];
        Chunk<DT>::unpack(yy[i], v[i]);
        Chunk<DT>::unpack(rr[i], r);
        if (a.w_post) {
          load_w<N>(a.w_post, c, wp);
#pragma unroll
          for (int j = 0; j < N; ++j) v[i][j] = v[i][j] * rstd * wp[j];
        }
        if (a.gate_kind == MOE_GATE_ELEMENT) {
          Chunk<DT>::unpack(gg[i], g);
#pragma unroll
          for (int j = 0; j < N; ++j) v[i][j] *= sigmoid_f32(g[j]);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) v[i][j] = fmaf(scale, v[i][j], a.res_scale * r[j]);
        rr[i] = Chunk<DT>::pack(v[i]);
        a.r_out[base + c] = rr[i];
      }
    }
  }
  if (!a.w_pre) return;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    Chunk<DT>::unpack(rr[i], v[i]);  // as stored
#pragma unroll
    for (int j = 0; j < N; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  }
  const float rstd = 1.0f / sqrtf(row_sum<W>(ss, red[1]) * inv_h + a.eps);
  if (a.rstd_pre && lane == 0) a.rstd_pre[t] = rstd;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = lane + TPR * i;
    if (c < a.cpr) {
      float wp[N];
      load_w<N>(a.w_pre, c, wp);
#pragma unroll
      for (int j = 0; j < N; ++j) v[i][j] = v[i][j] * rstd * wp[j];
      a.n_out[base + c] = Chunk<DT>::pack(v[i]);
    }
  }
}

struct NormBwd {
  const u32x4* dr;      // NULL: zero
  const u32x4* dn;      // NULL iff no w_pre
  const u32x4* r_out;
  const u32x4* y;       // NULL: r' = res
  const void* gate;
  const float* w_post;
  const float* w_pre;
  const float* rstd_post;
  const float* rstd_pre;
  u32x4* dres;
  u32x4* dy;
  void* dgate;
  float* part;          // [gridDim.x][2][H] partial sums of dw_post, dw_pre
  float res_scale, out_scale;
  int T, H, cpr, gate_kind;
};

// A block has R rows in flight, W waves to a row.  Each such group takes every
// P R-th row and keeps its share of the weight gradients in registers; at the
// end the groups join theirs and the block writes one partial row of each.
template <int DT, int NC, int W, int R>
__global__ __launch_bounds__(64 * W * R) void k_block_norm_grad(NormBwd a) {
  constexpr int N = Chunk<DT>::N;
  constexpr int TPR = 64 * W;
  __shared__ float red[2][R][W];
  __shared__ f32x4 join[R > 1 ? (R - 1) * TPR * NC * (N / 4) : 1];
  const int lane = (int)threadIdx.x % TPR;
  const int grp = R == 1 ? 0 : __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR);
  const float inv_h = 1.0f / (float)a.H;
  float gw_post[NC][N], gw_pre[NC][N];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) gw_post[i][j] = gw_pre[i][j] = 0.f;

  // the block's groups stay together for the barriers: past the last row a
  // group computes with zeros
  for (long t0 = (long)blockIdx.x * R; t0 < a.T; t0 += (long)gridDim.x * R) {
    const bool on = R == 1 || t0 + grp < a.T;
    const long t = on ? t0 + grp : 0;
    const size_t base = (size_t)t * a.cpr;
    const int cols = on ? a.cpr : 0;
    float D[NC][N];
    u32x4 vr[NC], vn[NC], vx[NC], vy[NC], vg[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lane + TPR * i;
      vr[i] = vn[i] = vx[i] = vy[i] = vg[i] = u32x4{0u, 0u, 0u, 0u};
      if (c < cols) {
        if (a.dr) vr[i] = __builtin_nontemporal_load(a.dr + base + c);
        if (a.w_pre) {
          vn[i] = __builtin_nontemporal_load(a.dn + base + c);
          vx[i] = __builtin_nontemporal_load(a.r_out + base + c);
        }
        if (a.y) vy[i] = __builtin_nontemporal_load(a.y + base + c);
        if (a.gate_kind == MOE_GATE_ELEMENT) vg[i] = ((const u32x4*)a.gate)[base + c];
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) Chunk<DT>::unpack(vr[i], D[i]);
    if (a.w_pre) {
      const float rstd = on ? a.rstd_pre[t] : 0.f;
      float g[NC][N], xh[NC][N], s = 0.f;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = lane + TPR * i;
        float wp[N];
        Chunk<DT>::unpack(vn[i], g[i]);
        Chunk<DT>::unpack(vx[i], xh[i]);
        if (c < cols) {
          load_w<N>(a.w_pre, c, wp);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            xh[i][j] *= rstd;
            gw_pre[i][j] = fmaf(g[i][j], xh[i][j], gw_pre[i][j]);
            g[i][j] *= wp[j];
            s = fmaf(g[i][j], xh[i][j], s);
          }
        }
      }
      const float m = row_sum<W>(s, red[0][grp]) * inv_h;
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) D[i][j] = fmaf(rstd, g[i][j] - xh[i][j] * m, D[i][j]);
    }
    // without y the rows passed through: dr = D
    const float rs = a.y ? a.res_scale : 1.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lane + TPR * i;
      if (c < cols) {
        float o[N];
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = rs * D[i][j];
        a.dres[base + c] = Chunk<DT>::pack(o);
      }
    }
    if (!a.y) {
      if (W > 1) __syncthreads();  // red[] is free again
      continue;
    }
    const float rstd = !on ? 0.f : a.w_post ? a.rstd_post[t] : 1.f;
    float sg = 1.f, sg_rest = 0.f;
    if (a.gate_kind == MOE_GATE_TOKEN) {
      const float g = ((const float*)a.gate)[t];
      sg = sigmoid_f32(g);
      sg_rest = sigmoid_rest_f32(g);
    }
    // D becomes b D, then du w_post = b c D w_post; s sums that times yh,
    // which is <b c D, u>, also the token gate's gradient up to (1 - c)
    float s = 0.f;
    float yh[NC][N];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lane + TPR * i;
      Chunk<DT>::unpack(vy[i], yh[i]);
      float wp[N], gt[N];
#pragma unroll
      for (int j = 0; j < N; ++j) wp[j] = 1.f;
      if (c < cols) {
        if (a.w_post) load_w<N>(a.w_post, c, wp);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          yh[i][j] *= rstd;
          D[i][j] *= a.out_scale;
        }
        if (a.gate_kind == MOE_GATE_ELEMENT) {
          Chunk<DT>::unpack(vg[i], gt);
          float o[N];
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float c1 = sigmoid_f32(gt[j]);
            D[i][j] *= c1;
            o[j] = D[i][j] * yh[i][j] * wp[j] * sigmoid_rest_f32(gt[j]);
          }
          ((u32x4*)a.dgate)[base + c] = Chunk<DT>::pack(o);
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j) D[i][j] *= sg;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
          gw_post[i][j] = fmaf(D[i][j], yh[i][j], gw_post[i][j]);
          D[i][j] *= wp[j];
          s = fmaf(D[i][j], yh[i][j], s);
        }
      }
    }
    float m = 0.f;
    if (a.w_post || a.gate_kind == MOE_GATE_TOKEN) {
      s = row_sum<W>(s, red[1][grp]);
      if (a.gate_kind == MOE_GATE_TOKEN && lane == 0 && on) ((float*)a.dgate)[t] = sg_rest * s;
      if (a.w_post) m = s * inv_h;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lane + TPR * i;
      if (c < cols) {
        float o[N];
#pragma unroll
        for (int j = 0; j < N; ++j) o[j] = rstd * (D[i][j] - yh[i][j] * m);
        a.dy[base + c] = Chunk<DT>::pack(o);
      }
    }
    if (W > 1) __syncthreads();  // red[] is free again
  }

  // the block's partial sums: its groups join in order
  auto put = [&](float (&gw)[NC][N], int which) {
    constexpr int Q = N / 4;
    if (R > 1) {
      __syncthreads();
      if (grp > 0) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int q = 0; q < Q; ++q)
            join[((grp - 1) * NC * Q + i * Q + q) * TPR + lane] =
                f32x4{gw[i][4 * q], gw[i][4 * q + 1], gw[i][4 * q + 2], gw[i][4 * q + 3]};
      }
      __syncthreads();
      if (grp > 0) return;
      for (int g = 0; g < R - 1; ++g)
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            const f32x4 v = join[(g * NC * Q + i * Q + q) * TPR + lane];
#pragma unroll
            for (int j = 0; j < 4; ++j) gw[i][4 * q + j] += v[j];
          }
    }
    f32x4* dst = (f32x4*)(a.part + ((size_t)blockIdx.x * 2 + which) * a.H);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lane + TPR * i;
      if (c < a.cpr) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
          dst[c * Q + q] =
              f32x4{gw[i][4 * q], gw[i][4 * q + 1], gw[i][4 * q + 2], gw[i][4 * q + 3]};
      }
    }
  };
  if (a.w_post) put(gw_post, 0);
  if (a.w_pre) put(gw_pre, 1);
}

// dw[which][h] = sum over the P partial rows: a block has 32 columns, 8 lanes of
// 4 side by side, and 32 strided shares of the rows; the shares join in order.
__global__ __launch_bounds__(256) void k_norm_dw(const float* __restrict__ part, int P, int H,
                                                 int first, float* __restrict__ dw_post,
                                                 float* __restrict__ dw_pre) {
  __shared__ f32x4 sh[32][8];
  const int which = first + (int)blockIdx.y;
  const int q = threadIdx.x & 7, share = threadIdx.x >> 3;
  const int col = blockIdx.x * 32 + 4 * q;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (col < H) {
    const f32x4* src = (const f32x4*)(part + (size_t)which * H + col);
    const size_t ld = (size_t)2 * H / 4;  // H is a multiple of 8
#pragma unroll 8
    for (int p = share; p < P; p += 32) s += src[p * ld];
  }
  sh[share][q] = s;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  const int c = threadIdx.x;
  float r = 0.f;
  for (int i = 0; i < 32; ++i) r += ((const float*)sh[i])[c];
  const int h = blockIdx.x * 32 + c;
  if (h < H) (which ? dw_pre : dw_post)[h] = r;
}

// Waves to a row: one wave holds up to 256 chunks, four up to 1024 (the widest
// rows of 16 bits), eight up to 2048 (f32).  From 65 chunks on four waves share a row where rows are few, since
// the latency of a row counts then, and backward, whose registers leave one
// wave a row too few rows in flight (T = 8191, H = 2048: 47 us, one wave 52 us;
// forward at T = 32768 one wave 124 us, four 140 us).
static int norm_waves(int T, int cpr, bool grad) {
  if (cpr > 1024) return 8;
  if (cpr > 256) return 4;
  return (cpr > 64 && (grad || T <= 512)) ? 4 : 1;
}

// f with the chunks per thread and the waves to a row.
template <int DT, bool GRAD, typename F>
static void by_shape(int T, int cpr, F&& f) {
  const int W = norm_waves(T, cpr, GRAD);
  if constexpr (DT == MOE_DT_F32) {
    if (W == 8) return f(IntC<4>{}, IntC<8>{});
  }
  if (W == 4 && cpr <= 256) f(IntC<1>{}, IntC<4>{});
  else if (W == 4) f(IntC<4>{}, IntC<4>{});
  else if (GRAD || cpr <= 64) f(IntC<1>{}, IntC<1>{});
  else if constexpr (!GRAD) f(IntC<4>{}, IntC<1>{});
}

// Rows in flight of a backward block of W waves a row: two where the registers
// allow (T = 8191, H = 2048: 47 us + 6 us for half the partial rows; one row and
// twice the blocks 47 + 8 us, half the blocks 57 + 6 us; four rows 50 + 6 us;
// by events).
constexpr int grad_rows(int NC, int W) { return W == 1 ? 4 : NC == 1 ? 2 : 1; }

void register_block_norm_kernels(std::vector<const void*>& k) {
  auto add = [&](auto D) {
    constexpr int DT = decltype(D)::value;
    auto one = [&](auto NC, auto W) {
      k.push_back((const void*)&k_block_norm<DT, decltype(NC)::value, decltype(W)::value>);
      if constexpr (decltype(NC)::value == 1 || decltype(W)::value > 1)
        k.push_back((const void*)&k_block_norm_grad<DT, decltype(NC)::value, decltype(W)::value,
                                                    grad_rows(decltype(NC)::value, decltype(W)::value)>);
    };
    one(IntC<1>{}, IntC<1>{});
    one(IntC<4>{}, IntC<1>{});
    one(IntC<1>{}, IntC<4>{});
    one(IntC<4>{}, IntC<4>{});
    if constexpr (DT == MOE_DT_F32) one(IntC<4>{}, IntC<8>{});
  };
  for (int dt = MOE_DT_BF16; dt <= MOE_DT_F32; ++dt) by_dtype(dt, add);
  k.push_back((const void*)&k_norm_dw);
}

uint64_t block_norm_threads(int T, int H, int dtype) {
  const int W = norm_waves(T, H * dtype_bytes(dtype) / 16, false);
  return W == 1 ? wave_rows_threads(T) : (uint64_t)T * 64 * W;
}

hipError_t launch_block_norm(const void* res, const void* y, const void* gate, int gate_kind,
                             const float* w_post, const float* w_pre, float res_scale,
                             float out_scale, float eps, int T, int H, int dtype, void* r_out,
                             void* n_out, float* rstd_post, float* rstd_pre, hipStream_t s) {
  const int cpr = H * dtype_bytes(dtype) / 16;
  const NormFwd a{(const u32x4*)res, (const u32x4*)y, gate,      w_post,    w_pre,
                  (u32x4*)r_out,     (u32x4*)n_out,   rstd_post, rstd_pre,  res_scale,
                  out_scale,         eps,             T,         H,         cpr,
                  gate_kind};
  by_dtype(dtype, [&](auto D) {
    constexpr int DT = decltype(D)::value;
    by_shape<DT, false>(T, cpr, [&](auto NC, auto W) {
      constexpr int w = decltype(W)::value;
      MOE_LAUNCH("block_norm", s, (k_block_norm<DT, decltype(NC)::value, w>),
                 dim3(w == 1 ? (T + 3) / 4 : T), dim3(w == 1 ? 256 : 64 * w), 0, s, a);
    });
  });
  return hipGetLastError();
}

// Blocks of the backward kernel, each with a partial row of the weight
// gradients: enough to fill the chip, and 8 rows to a block at least once that
// is so, which keeps the partials small beside the rows.  A function of the
// sizes alone, so results do not depend on the device's state.
static int norm_parts(int T, int H, int dtype) {
  const int cpr = H * dtype_bytes(dtype) / 16;
  const int W = norm_waves(T, cpr, true), rows = grad_rows(cpr <= 64 * W ? 1 : 4, W);
  const int P = (T + rows - 1) / rows;
  const int top = rows == 2 ? 512 : 1024;
  const int most = T / 8 < 256 ? 256 : T / 8 < top ? T / 8 : top;
  return P < most ? P : most;
}

size_t block_norm_workspace_bytes(int T, int H, int dtype) {
  return (size_t)norm_parts(T, H, dtype) * 2 * H * sizeof(float);
}

hipError_t launch_block_norm_grad(const void* dr, const void* dn, const void* r_out, const void* y,
                                  const void* gate, int gate_kind, const float* w_post,
                                  const float* w_pre, const float* rstd_post,
                                  const float* rstd_pre, float res_scale, float out_scale, int T,
                                  int H, int dtype, void* dres, void* dy, void* dgate,
                                  float* dw_post, float* dw_pre, void* ws, hipStream_t s) {
  const int cpr = H * dtype_bytes(dtype) / 16;
  const int P = norm_parts(T, H, dtype);
  const NormBwd a{(const u32x4*)dr, (const u32x4*)dn, (const u32x4*)r_out, (const u32x4*)y,
                  gate,             w_post,           w_pre,               rstd_post,
                  rstd_pre,         (u32x4*)dres,     (u32x4*)dy,          dgate,
                  (float*)ws,       res_scale,        out_scale,           T,
                  H,                cpr,              gate_kind};
  by_dtype(dtype, [&](auto D) {
    constexpr int DT = decltype(D)::value;
    by_shape<DT, true>(T, cpr, [&](auto NC, auto W) {
      constexpr int w = decltype(W)::value;
      constexpr int r = grad_rows(decltype(NC)::value, w);
      MOE_LAUNCH("block_norm_grad", s, (k_block_norm_grad<DT, decltype(NC)::value, w, r>), dim3(P),
                 dim3(64 * w * r), 0, s, a);
    });
  });
  hipError_t e = hipGetLastError();
  const int n = (w_post ? 1 : 0) + (w_pre ? 1 : 0);
  if (e != hipSuccess || n == 0) return e;
  MOE_LAUNCH("block_norm_dw", s, k_norm_dw, dim3((H + 31) / 32, n), dim3(256), 0, s,
             (const float*)ws, P, H, w_post ? 0 : 1, dw_post, dw_pre);
  return hipGetLastError();
}

}  // namespace moe
