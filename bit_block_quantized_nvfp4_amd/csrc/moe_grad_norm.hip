// The norm of many gradients together, and the gradients scaled down to a limit:
//
//   norm = sqrt(sum over all tensors of g^2),  c = min(1, max_norm / (norm + 1e-6)),  g' = c g
//
// Bound by memory: the gradients are read once for the norm, once for the scaling,
// and written once.  One launch covers up to kTensors tensors of any sizes and
// types: their table travels with the launch (nothing of it stands in device
// memory, so a captured graph keeps its own), each tensor is cut into pieces,
// and the blocks take the pieces in turn.  The scaling takes them from the last to the
// first: what the norm read last is still in the last-level cache.  120 MB take 19.6 us for the
// squares (6.1 TB/s), 4.6 to join them and 36.8 for the scaling (6.5 TB/s); a few small
// tensors 4.3 and 3.4 us, the length of two launches.
//
// The squares and their sums are held in 64 bits: f32 squares would pass its range
// from values of 1.8e19 on, and the conversion is free beside the loads.
#include <algorithm>

#include "moe_internal.hpp"
#include "moe_vec.hpp"

namespace moe {

constexpr int kTensors = 112;     // a table of 3.6 KB: kernel arguments end at 4 KB
constexpr int kNormBlocks = 2048; // of a launch at most, eight on a compute unit
constexpr int kOneBlock = 16;     // pieces that one block takes, a wave each, with the root too
constexpr int kOneChunks = 1024;  // 16-byte chunks of such a piece
constexpr int kLeastChunks = 256, kMostChunks = 8192;  // of the others

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
  int32_t chunks;  // 16-byte chunks of a piece
  GradEntry e[kTensors];
};
static_assert(sizeof(GradTable) <= 3800, "kernel arguments");

// The tensor of a piece: the last one that begins at or before it (each lane looks at
// two).
__device__ __forceinline__ int entry_of(const GradTable& t, uint32_t piece) {
  const int lane = threadIdx.x & 63;
  const bool a = lane < t.count && t.e[lane].first <= piece;
  const bool b = lane + 64 < t.count && t.e[min(lane + 64, kTensors - 1)].first <= piece;
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(a)) + __popcll(__ballot(b)) - 1);
}

// f(entry, piece) for this block's pieces.  BACK: from the last to the first.
template <bool BACK, typename F>
__device__ __forceinline__ void by_pieces(const GradTable& t, F&& f) {
  for (uint32_t i = blockIdx.x; i < t.pieces; i += gridDim.x) {
    const uint32_t piece = BACK ? t.pieces - 1 - i : i;
    f(t.e[entry_of(t, piece)], piece);
  }
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

// A piece of a tensor in 16-byte chunks: `head` values before the first aligned address, nv
// chunks, then the rest.
template <int DT>
struct Span {
  static constexpr int N = Chunk<DT>::N, ES = 16 / N;
  int64_t lo;
  int cnt, head, nv;
  __device__ __forceinline__ Span(const GradEntry& e, uint32_t piece, int chunks) {
    const int64_t most = (int64_t)chunks * N;
    lo = (int64_t)(piece - e.first) * most;
    cnt = (int)(e.n - lo < most ? e.n - lo : most);
    const int past = (int)((uintptr_t)e.in & 15) / ES;  // a piece is whole chunks: the same for each
    head = min(cnt, (N - past) % N);
    nv = (cnt - head) / N;
  }
  // Value i of those outside the chunks: the head's, then the tail's.
  __device__ __forceinline__ int64_t other(int i) const { return lo + (i < head ? i : nv * N + i); }
};

// f(chunk, place) for the nv chunks at p, by THREADS threads, four at a time under way.
template <int THREADS, int U, typename F>
__device__ __forceinline__ void by_chunks(const u32x4* __restrict__ p, int nv, int tid, F&& f) {
  int c = tid;
  for (; c + (U - 1) * THREADS < nv; c += U * THREADS) {
    u32x4 v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) v[k] = p[c + k * THREADS];
#pragma unroll
    for (int k = 0; k < U; ++k) f(v[k], c + k * THREADS);
  }
  for (; c < nv; c += THREADS) f(p[c], c);
}

// The sum of a piece's squares: the part of thread tid of THREADS.
template <int DT, int THREADS, int U>
__device__ __forceinline__ double squares(const GradEntry& e, uint32_t piece, int chunks, int tid) {
  constexpr int N = Chunk<DT>::N;
  const Span<DT> s(e, piece, chunks);
  double sum = 0.0;
  by_chunks<THREADS, U>((const u32x4*)((const char*)e.in + (s.lo + s.head) * Span<DT>::ES), s.nv, tid,
                        [&](u32x4 v, int) {
                          float f[N];
                          Chunk<DT>::unpack(v, f);
#pragma unroll
                          for (int j = 0; j < N; ++j) sum = fma((double)f[j], (double)f[j], sum);
                        });
  if (tid < s.cnt - s.nv * N) {  // at most two chunks' worth
    const double w = value_at<DT>(e.in, s.other(tid));
    sum = fma(w, w, sum);
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

__global__ __launch_bounds__(256, 8) void k_grad_squares(GradTable t, double* __restrict__ partial) {
  __shared__ double part[4];
  double sum = 0.0;
  by_pieces<false>(t, [&](const GradEntry& e, uint32_t piece) {
    by_type(e.dtype, [&](auto D) { sum += squares<decltype(D)::value, 256, 4>(e, piece, t.chunks, threadIdx.x); });
  });
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

// Up to kOneBlock pieces in one launch.
__global__ __launch_bounds__(1024) void k_grad_norm_small(GradTable t, float* __restrict__ norm) {
  static_assert(kOneBlock == 16, "a piece to a wave");
  __shared__ double part[16];
  double sum = 0.0;
  const uint32_t piece = (uint32_t)__builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (piece < t.pieces) {
    const GradEntry& e = t.e[entry_of(t, piece)];
    by_type(e.dtype, [&](auto D) { sum = squares<decltype(D)::value, 64, 8>(e, piece, t.chunks, threadIdx.x & 63); });
  }
  sum = block_sum<16>(sum, part);
  if (threadIdx.x == 0) norm[0] = (float)sqrt(sum);
}

template <int DT, bool FAR>
__device__ __forceinline__ void scale_piece(const GradEntry& e, uint32_t piece, int chunks, float c, int tid) {
  constexpr int N = Chunk<DT>::N, ES = Span<DT>::ES;
  Span<DT> s(e, piece, chunks);
  // both sides aligned alike, or value by value
  if (((uintptr_t)e.in ^ (uintptr_t)e.out) & 15) s.head = s.cnt, s.nv = 0;
  u32x4* q = (u32x4*)((char*)e.out + (s.lo + s.head) * ES);
  by_chunks<256, 4>((const u32x4*)((const char*)e.in + (s.lo + s.head) * ES), s.nv, tid, [&](u32x4 v, int at) {
    float f[N];
    Chunk<DT>::unpack(v, f);
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] *= c;
    if (FAR) __builtin_nontemporal_store(Chunk<DT>::pack(f), q + at);
    else q[at] = Chunk<DT>::pack(f);
  });
  for (int i = tid; i < s.cnt - s.nv * N; i += 256) put_value<DT>(e.out, s.other(i), value_at<DT>(e.in, s.other(i)) * c);
}

// FAR: the outputs go past the last-level cache.
template <bool FAR>
__global__ __launch_bounds__(256, 8) void k_grad_scale(GradTable t, const float* __restrict__ norm,
                                                    float max_norm) {
  // a NaN norm gives NaN, an infinite one zeros (and NaN for infinite values)
  float c = max_norm / (norm[0] + 1e-6f);
  c = c > 1.0f ? 1.0f : c;
  by_pieces<true>(t, [&](const GradEntry& e, uint32_t piece) {
    if (c == 1.0f && e.in == e.out) return;  // in place, and nothing to change
    by_type(e.dtype, [&](auto D) { scale_piece<decltype(D)::value, FAR>(e, piece, t.chunks, c, threadIdx.x); });
  });
}

void register_grad_norm_kernels(std::vector<const void*>& k) {
  k.push_back((const void*)&k_grad_squares);
  k.push_back((const void*)&k_grad_norm);
  k.push_back((const void*)&k_grad_norm_small);
  k.push_back((const void*)&k_grad_scale<false>);
  k.push_back((const void*)&k_grad_scale<true>);
}

// 16-byte chunks of a tensor's values.
static int64_t chunks_of(const moe_grad_tensor& g) { return (g.n * dtype_bytes(g.dtype) + 15) / 16; }

// The table of the tensors [from, to) that hold values, at most kTensors, in pieces of
// `chunks`; 0: as many as give each of the chip's blocks the same number of pieces (the
// last round of blocks is then as full as the others).
static GradTable table_of(const moe_grad_tensor* g, int from, int to, int chunks) {
  GradTable t;
  if (chunks == 0) {
    int64_t all = 0;
    for (int i = from; i < to; ++i) all += chunks_of(g[i]);
    const int64_t rounds = (all + (int64_t)kNormBlocks * kMostChunks - 1) / ((int64_t)kNormBlocks * kMostChunks);
    const int64_t each = all / (std::max<int64_t>(rounds, 1) * kNormBlocks) + 1;
    chunks = (int)((each + kLeastChunks - 1) / kLeastChunks * kLeastChunks);
  }
  t.pieces = 0;
  t.count = 0;
  t.chunks = chunks;
  for (int i = from; i < to; ++i) {
    if (g[i].n == 0) continue;
    t.e[t.count++] = GradEntry{g[i].grad, g[i].out, g[i].n, t.pieces, g[i].dtype};
    t.pieces += (uint32_t)((chunks_of(g[i]) + chunks - 1) / chunks);
  }
  return t;
}
static unsigned blocks_of(const GradTable& t) { return (unsigned)std::min<uint32_t>(t.pieces, kNormBlocks); }

size_t grad_norm_workspace_bytes(int count) {
  return (size_t)((count + kTensors - 1) / kTensors) * kNormBlocks * sizeof(double);
}

hipError_t launch_grad_norm(const moe_grad_tensor* g, int count, float* norm, double* ws,
                            hipStream_t s) {
  if (count <= kTensors) {
    const GradTable t = table_of(g, 0, count, kOneChunks);
    if (t.pieces <= (uint32_t)kOneBlock) {
      MOE_LAUNCH("grad_norm", s, k_grad_norm_small, dim3(1), dim3(1024), 0, s, t, norm);
      return hipGetLastError();
    }
  }
  int n = 0;
  for (int i = 0; i < count; i += kTensors) {
    const GradTable t = table_of(g, i, std::min(i + kTensors, count), 0);
    if (t.pieces == 0) continue;
    MOE_LAUNCH("grad_squares", s, k_grad_squares, dim3(blocks_of(t)), dim3(256), 0, s, t, ws + n);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    n += (int)blocks_of(t);
  }
  MOE_LAUNCH("grad_norm", s, k_grad_norm, dim3(1), dim3(1024), 0, s, ws, n, norm);
  return hipGetLastError();
}

// Outputs go past the last-level cache where they and the gradients would fill most of its
// 256 MB: the gradients that the norm read last then stay for the scaling (norm and
// scaling of 120 MB beside the gradients 78 us with ordinary stores, 61 so; of 2.4 GB 1355 and 1313
// us).
constexpr int64_t kFarBytes = (int64_t)192 << 20;

hipError_t launch_grad_clip(const moe_grad_tensor* g, int count, const float* norm, float max_norm,
                            hipStream_t s) {
  int64_t bytes = 0;
  for (int i = 0; i < count; ++i) bytes += 16 * chunks_of(g[i]) * (g[i].out == g[i].grad ? 1 : 2);
  const auto kernel = bytes > kFarBytes ? &k_grad_scale<true> : &k_grad_scale<false>;
  for (int i = (count - 1) / kTensors * kTensors; i >= 0; i -= kTensors) {
    const GradTable t = table_of(g, i, std::min(i + kTensors, count), 0);
    if (t.pieces == 0) continue;
    MOE_LAUNCH("grad_scale", s, kernel, dim3(blocks_of(t)), dim3(256), 0, s, t, norm, max_norm);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
