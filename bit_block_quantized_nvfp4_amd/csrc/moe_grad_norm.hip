// The norm of many gradients together, and the gradients scaled down to a limit:
//
//   norm = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (norm + 1e-6)),  g' = c g
//
// Bound by memory: the gradients are read once for the norm, once for the scaling,
// and written once.  One launch covers up to kTensors tensors of any sizes and
// types: their table travels with the launch (nothing of it stands in device
// memory, so a captured graph keeps its own), each tensor is cut into pieces of
// kPiece values, and the blocks take the pieces in turn.
//
// The squares and their sums are held in 64 bits: f32 squares would pass its range
// from values of 1.8e19 on, and the conversion is free beside the loads.
#include "moe_internal.hpp"
#include "moe_vec.hpp"

namespace moe {

constexpr int kTensors = 112;     // a table of 3.6 KB: kernel arguments end at 4 KB
constexpr int kPiece = 16384;     // values
constexpr int kNormBlocks = 2048; // of a launch at most, eight on a compute unit

struct GradEntry {
  const void* in;
  void* out;
  int64_t n;
  uint32_t first;  // its first piece
  int32_t dtype;
};
struct GradTable {
  uint32_t pieces;
  int32_t count;
  GradEntry e[kTensors];
};
static_assert(sizeof(GradTable) <= 3800, "kernel arguments");

// The tensor of a piece: the last one that begins at or before it (each lane looks at
// two; entries behind the last one begin past every piece).
__device__ __forceinline__ int entry_of(const GradTable& t, uint32_t piece) {
  const int lane = threadIdx.x & 63;
  const bool a = lane < t.count && t.e[lane].first <= piece;
  const bool b = lane + 64 < t.count && t.e[min(lane + 64, kTensors - 1)].first <= piece;
  return __popcll(__ballot(a)) + __popcll(__ballot(b)) - 1;
}

template <int DT>
__device__ __forceinline__ float value_at(const void* p, int64_t i) {
  if constexpr (DT == MOE_DT_F32) return ((const float*)p)[i];
  else if constexpr (DT == MOE_DT_F16) return (float)((const _Float16*)p)[i];
  else return bf16_bits_to_f32(((const uint16_t*)p)[i]);
}
template <int DT>
__device__ __forceinline__ void put_value(void* p, int64_t i, float v) {
  if constexpr (DT == MOE_DT_F32) ((float*)p)[i] = v;
  else if constexpr (DT == MOE_DT_F16) ((_Float16*)p)[i] = (_Float16)v;
  else ((uint16_t*)p)[i] = f32_to_bf16_bits(v);
}

// A piece in 16-byte chunks: `head` values before the first aligned address, nv chunks,
// then the rest.
template <int DT>
struct Span {
  static constexpr int N = Chunk<DT>::N, ES = 16 / N;
  int64_t lo;
  int cnt, head, nv;
  __device__ __forceinline__ Span(const GradEntry& e, uint32_t piece) {
    lo = (int64_t)(piece - e.first) * kPiece;
    cnt = (int)(e.n - lo < kPiece ? e.n - lo : (int64_t)kPiece);
    const int past = (int)((uintptr_t)e.in & 15) / ES;  // kPiece values are whole chunks
    head = min(cnt, (N - past) % N);
    nv = (cnt - head) / N;
  }
};

template <int DT>
__device__ __forceinline__ double squares(const GradEntry& e, uint32_t piece, int tid, int threads) {
  constexpr int N = Chunk<DT>::N;
  const Span<DT> s(e, piece);
  double sum = 0.0;
  const u32x4* p = (const u32x4*)((const char*)e.in + (s.lo + s.head) * Span<DT>::ES);
  for (int c = tid; c < s.nv; c += threads) {
    float f[N];
    Chunk<DT>::unpack(p[c], f);
#pragma unroll
    for (int j = 0; j < N; ++j) sum = fma((double)f[j], (double)f[j], sum);
  }
  const int rest = s.cnt - s.nv * N;  // the head's, then the tail's
  for (int i = tid; i < rest; i += threads) {
    const double v = value_at<DT>(e.in, s.lo + (i < s.head ? i : s.nv * N + i));
    sum = fma(v, v, sum);
  }
  return sum;
}

template <int W>
__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
  for (int o = 32; o > 0; o /= 2) v += __shfl_xor(v, o);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int i = 1; i < W; ++i) v += part[i];
  return v;
}

template <typename F>
__device__ __forceinline__ void by_type(int dt, F&& f) {
  if (dt == MOE_DT_BF16) f(IntC<MOE_DT_BF16>{});
  else if (dt == MOE_DT_F16) f(IntC<MOE_DT_F16>{});
  else f(IntC<MOE_DT_F32>{});
}

__global__ __launch_bounds__(256) void k_grad_squares(GradTable t, double* __restrict__ partial) {
  __shared__ double part[4];
  double sum = 0.0;
  for (uint32_t piece = blockIdx.x; piece < t.pieces; piece += gridDim.x) {
    const GradEntry& e = t.e[__builtin_amdgcn_readfirstlane(entry_of(t, piece))];
    by_type(e.dtype, [&](auto D) { sum += squares<decltype(D)::value>(e, piece, threadIdx.x, 256); });
  }
  sum = block_sum<4>(sum, part);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

__global__ __launch_bounds__(1024) void k_grad_norm(const double* __restrict__ partial, int n,
                                                    float* __restrict__ norm) {
  __shared__ double part[16];
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) sum += partial[i];
  sum = block_sum<16>(sum, part);
  if (threadIdx.x == 0) norm[0] = (float)sqrt(sum);
}

template <int DT>
__device__ __forceinline__ void scale_piece(const GradEntry& e, uint32_t piece, float c, int tid) {
  constexpr int N = Chunk<DT>::N, ES = Span<DT>::ES;
  Span<DT> s(e, piece);
  // both sides aligned alike, or value by value
  if (((uintptr_t)e.in ^ (uintptr_t)e.out) & 15) s.head = s.cnt, s.nv = 0;
  const u32x4* p = (const u32x4*)((const char*)e.in + (s.lo + s.head) * ES);
  u32x4* q = (u32x4*)((char*)e.out + (s.lo + s.head) * ES);
  for (int i = tid; i < s.nv; i += 256) {
    float f[N];
    Chunk<DT>::unpack(p[i], f);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] *= c;
    q[i] = Chunk<DT>::pack(f);
  }
  const int rest = s.cnt - s.nv * N;
  for (int i = tid; i < rest; i += 256) {
    const int64_t at = s.lo + (i < s.head ? i : s.nv * N + i);
    put_value<DT>(e.out, at, value_at<DT>(e.in, at) * c);
  }
}

__global__ __launch_bounds__(256) void k_grad_scale(GradTable t, const float* __restrict__ norm,
                                                    float max_norm) {
  // a NaN norm gives NaN, an infinite one zeros (and NaN for infinite values)
  float c = max_norm / (norm[0] + 1e-6f);
  c = c > 1.0f ? 1.0f : c;
  for (uint32_t piece = blockIdx.x; piece < t.pieces; piece += gridDim.x) {
    const GradEntry& e = t.e[__builtin_amdgcn_readfirstlane(entry_of(t, piece))];
    if (c == 1.0f && e.in == e.out) continue;  // in place, and nothing to change
    by_type(e.dtype, [&](auto D) { scale_piece<decltype(D)::value>(e, piece, c, threadIdx.x); });
  }
}

void register_grad_norm_kernels(std::vector<const void*>& k) {
  k.push_back((const void*)&k_grad_squares);
  k.push_back((const void*)&k_grad_norm);
  k.push_back((const void*)&k_grad_scale);
}

// The tensors with values in them, kTensors to a launch: f(table, blocks).
template <typename F>
static hipError_t by_tables(const moe_grad_tensor* g, int count, F&& f) {
  GradTable t;
  t.pieces = 0;
  t.count = 0;
  for (int i = 0; i <= count; ++i) {
    if (t.count == kTensors || (i == count && t.count > 0)) {
      f(t, t.pieces < (uint32_t)kNormBlocks ? t.pieces : (uint32_t)kNormBlocks);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      t.pieces = 0;
      t.count = 0;
    }
    if (i == count || g[i].n == 0) continue;
    t.e[t.count++] = GradEntry{g[i].grad, g[i].out, g[i].n, t.pieces, g[i].dtype};
    t.pieces += (uint32_t)((g[i].n + kPiece - 1) / kPiece);
  }
  return hipSuccess;
}

size_t grad_norm_workspace_bytes(int count) {
  return (size_t)((count + kTensors - 1) / kTensors) * kNormBlocks * sizeof(double);
}

hipError_t launch_grad_norm(const moe_grad_tensor* g, int count, float* norm, double* ws,
                            hipStream_t s) {
  int n = 0;
  const hipError_t e = by_tables(g, count, [&](const GradTable& t, uint32_t blocks) {
    MOE_LAUNCH("grad_squares", s, k_grad_squares, dim3(blocks), dim3(256), 0, s, t, ws + n);
    n += (int)blocks;
  });
  if (e != hipSuccess) return e;
  MOE_LAUNCH("grad_norm", s, k_grad_norm, dim3(1), dim3(1024), 0, s, ws, n, norm);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const moe_grad_tensor* g, int count, const float* norm, float max_norm,
                            hipStream_t s) {
  return by_tables(g, count, [&](const GradTable& t, uint32_t blocks) {
    MOE_LAUNCH("grad_scale", s, k_grad_scale, dim3(blocks), dim3(256), 0, s, t, norm, max_norm);
  });
}

}  // namespace moe
