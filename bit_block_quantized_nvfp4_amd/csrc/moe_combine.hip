// Combine (A10): out[t] = bf16( sum_k w[t][k] * y[slot_pos[t*K+k]] + c_t y[slot_pos[T*K+t]] ),
// c_t = 1, or sigmoid(gate[t]) for the gated shared expert (combine_chunk in
// moe_combine.hpp).  Each thread owns 8 consecutive columns of one token
// (16-byte loads/stores); the order of the sum is fixed per element and
// independent of how the grid is cut.
#include "moe_combine.hpp"
#include "moe_internal.hpp"

namespace moe {

__global__ __launch_bounds__(256) void k_combine(const uint16_t* __restrict__ y,
                                                 const float* __restrict__ w,
                                                 const int32_t* __restrict__ slot_pos,
                                                 const float* __restrict__ gate, int T, int K,
                                                 int H, int has_shared,
                                                 uint16_t* __restrict__ out) {
  const int cpr = H / 8;  // 8-column chunks per row
  const long gid = (long)blockIdx.x * 256 + threadIdx.x;
  if (gid >= (long)T * cpr) return;
  const int t = (int)(gid / cpr), c = (int)(gid % cpr);
  combine_chunk(y, w, slot_pos, gate, T, K, H, has_shared, out, t, 8 * c);
}

void register_combine_kernels(std::vector<const void*>& k) { k.push_back((const void*)&k_combine); }

uint64_t combine_threads(int T, int H) {
  const uint64_t here = ((uint64_t)T * (H / 8) + 255) / 256 * 256, there = slot_rows_threads(T, H, MOE_DT_BF16);
  return here > there ? here : there;
}

hipError_t launch_combine(const uint16_t* y, const float* w, const int32_t* slot_pos,
                          const float* gate, int T, int K, int H, int has_shared, uint16_t* out,
                          hipStream_t s) {
  // Rows that the 256 MB last-level cache does not hold go to the typed operators'
  // kernel, which gives the same bits and reads past the caches, unless more than
  // a quarter of its threads would stand idle behind the row's end (it gives a row
  // 2^n threads, or a multiple of 256).  In a row in a graph, us, here and there:
  //                      184 MB         300 MB         600 MB
  //   H = 2048, K = 10   32.4   37.3    68.6   58.9   133.5  114.9
  //   H = 2048, K = 2    47.2   48.6   107.5   76.7   210.9  172.1
  //   H = 768, K = 10    32.7   38.9    69.0   61.8   134.5  120.4  (3/4 in use)
  //   H = 768, K = 2     50.7   61.1   110.4   98.5   218.1  208.5
  //   H = 2560, K = 10   32.7   43.1    67.6   69.3   133.2  136.5  (5/8 in use)
  //   H = 2560, K = 2    48.1   70.8   108.8  113.8   214.3  241.2
  const size_t bytes = (size_t)T * (K + has_shared) * H * sizeof(uint16_t);
  const uint64_t there = slot_rows_threads(T, H, MOE_DT_BF16), used = (uint64_t)T * (H / 8);
  if (bytes > (size_t)256 << 20 && 4 * used >= 3 * there)
    return launch_slot_sum(y, w, slot_pos, gate, T, K, H, has_shared, MOE_DT_BF16, out, s);
  const long n = (long)T * (H / 8);
  MOE_LAUNCH("combine", s, k_combine, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, y, w,
             slot_pos, gate, T, K, H, has_shared, out);
  return hipGetLastError();
}

}  // namespace moe
