// C entry points of libmoe_nvfp4: argument checks, the gfx950 gate, one-time
// kernel resolution, dispatch to the launchers, error text, and the optional
// per-kernel event timing.
#include <float.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <string>
#include <vector>

#include "moe_internal.hpp"

namespace {

thread_local std::string g_err;

int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_err = buf;
  return code;
}

int ok() {
  g_err.clear();
  return MOE_OK;
}

int hip_fail(hipError_t e, const char* what) {
  return fail(MOE_EHIP, "%s: %s", what, hipGetErrorString(e));
}

constexpr int kMaxDevices = 64;
std::mutex g_init_mu;
int g_init_state[kMaxDevices];  // 0 = not yet, 1 = ready, < 0 = status of the failure
std::string g_init_msg[kMaxDevices];
int g_cus[kMaxDevices];

// Workspace of moe_expert_ffn_noalloc: one copy per device, held until the
// process ends.  In host code `scratch` is only a stand-in for the symbol; its
// device address on each GPU is g_scratch[dev], taken once at init.
static __device__ __align__(256) uint8_t scratch[MOE_NOALLOC_WS_BYTES];
void* g_scratch[kMaxDevices];

int ensure_init() {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(MOE_EUNSUPPORTED, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_init_mu);
  if (g_init_state[dev] == 1) return MOE_OK;
  if (g_init_state[dev] < 0) {
    g_err = g_init_msg[dev];
    return g_init_state[dev];
  }
  hipDeviceProp_t prop;
  e = hipGetDeviceProperties(&prop, dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDeviceProperties");
  if (strncmp(prop.gcnArchName, "gfx950", 6) != 0) {
    int rc = fail(MOE_EUNSUPPORTED,
                  "moe_nvfp4 is built for gfx950 (MI355X) only; device %d is %s", dev,
                  prop.gcnArchName);
    g_init_state[dev] = rc;
    g_init_msg[dev] = g_err;
    return rc;
  }
  g_cus[dev] = prop.multiProcessorCount > 0 ? prop.multiProcessorCount : 256;
  {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess || p == nullptr) {
      int rc = e != hipSuccess ? hip_fail(e, "hipGetSymbolAddress(scratch) at init")
                               : fail(MOE_EHIP, "hipGetSymbolAddress(scratch) returned null");
      g_init_state[dev] = rc;
      g_init_msg[dev] = g_err;
      return rc;
    }
    g_scratch[dev] = p;
  }
  std::vector<const void*> ks;
  moe::register_route_kernels(ks);
  moe::register_router_kernels(ks);
  moe::register_permute_kernels(ks);
  moe::register_combine_kernels(ks);
  moe::register_ffn_kernels(ks);
  moe::register_sort_kernels(ks);
  moe::register_block_norm_kernels(ks);
  moe::register_fp8_stream_kernels(ks);
  moe::register_fp8_tile_kernels(ks);
  moe::register_dense_kernels(ks);
  moe::register_dense_grad_kernels(ks);
  moe::register_int8_kernels(ks);
  moe::register_grad_norm_kernels(ks);
  for (const void* k : ks) {
    hipFuncAttributes attr;
    e = hipFuncGetAttributes(&attr, k);
    if (e != hipSuccess) {
      int rc = hip_fail(e, "kernel lookup at init");
      g_init_state[dev] = rc;
      g_init_msg[dev] = g_err;
      return rc;
    }
  }
  g_init_state[dev] = 1;
  return MOE_OK;
}

// ---- timing ----
struct TimingRec {
  const char* name;
  hipEvent_t a, b;
};
std::atomic<bool> g_timing_on{false};
std::mutex g_tmu;
std::vector<TimingRec> g_pool;
size_t g_used = 0;
long g_dropped = 0;
constexpr size_t kMaxRecords = 65536;

bool sizes_ok_common(int T, int E, int K) {
  return T >= 1 && E >= 1 && E <= 1024 && K >= 1 && K <= 32 && K <= E &&
         (long long)T * K <= (1LL << 30) && (long long)T * E <= (1LL << 40);
}

// Slots and positions are int32: T*K routed ones, then T shared ones.
bool slots_ok(int T, int K, int has_shared) {
  return (long long)T * (K + has_shared) <= INT32_MAX;
}

// HIP launches fewer than 2^32 threads.
bool grid_ok(uint64_t threads) { return threads < (1ull << 32); }

bool dtype_ok(int dt) { return dt >= MOE_DT_BF16 && dt <= MOE_DT_F32; }

template <typename... P>
bool aligned16(const P*... p) {
  return ((((uintptr_t)p) & 15) | ...) == 0;
}

// Sizes of the sort entry points.
int sort_sizes(const char* who, int T, int K, int H, int has_shared, int dtype) {
  if (!dtype_ok(dtype)) return fail(MOE_EUNSUPPORTED, "%s: unknown dtype %d", who, dtype);
  if (T < 1 || K < 1 || K > 32 || H < 8 || H > 65536 || H % 8 != 0 ||
      (has_shared != 0 && has_shared != 1) || (long long)T * K > (1LL << 30))
    return fail(MOE_EINVAL, "%s: need T >= 1, 1 <= K <= 32, T*K <= 2^30, H a multiple of 8 in [8, 65536], has_shared in {0,1} (T=%d K=%d H=%d)", who, T, K, H);
  if (!slots_ok(T, K, has_shared))
    return fail(MOE_EINVAL, "%s: T*(K + has_shared) must be below 2^31 (T=%d K=%d)", who, T, K);
  return MOE_OK;
}

int too_many_rows(const char* who, int T) {
  return fail(MOE_EINVAL, "%s: T=%d takes a launch of 2^32 threads or more", who, T);
}

int launched(hipError_t e, const char* what) { return e == hipSuccess ? ok() : hip_fail(e, what); }

}  // namespace

namespace moe {

int num_cus() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices || g_cus[dev] <= 0) return 256;
  return g_cus[dev];
}

int timing_begin(const char* name, hipStream_t s) {
  if (!g_timing_on.load(std::memory_order_relaxed)) return -1;
  std::lock_guard<std::mutex> lk(g_tmu);
  if (g_used >= kMaxRecords) {
    ++g_dropped;
    return -1;
  }
  if (g_used == g_pool.size()) {
    TimingRec r{name, nullptr, nullptr};
    if (hipEventCreate(&r.a) != hipSuccess) return -1;
    if (hipEventCreate(&r.b) != hipSuccess) {
      (void)hipEventDestroy(r.a);
      return -1;
    }
    g_pool.push_back(r);
  }
  TimingRec& r = g_pool[g_used];
  r.name = name;
  if (hipEventRecord(r.a, s) != hipSuccess) return -1;
  return (int)g_used++;
}

void timing_end(int slot, hipStream_t s) {
  if (slot < 0) return;
  std::lock_guard<std::mutex> lk(g_tmu);
  (void)hipEventRecord(g_pool[(size_t)slot].b, s);
}

}  // namespace moe

extern "C" {

int moe_init(void) {
  const int rc = ensure_init();
  return rc == MOE_OK ? ok() : rc;
}

const char* moe_last_error(void) { return g_err.c_str(); }

size_t moe_workspace_bytes(int op, int T, int E, int K, int H, int I, int has_shared,
                           int act_mode) {
  if (!sizes_ok_common(T, E, K) || (has_shared != 0 && has_shared != 1)) return 0;
  if (op == MOE_OP_PERMUTE) return moe::permute_workspace_bytes(T, E, K);
  if (op == MOE_OP_LAYER) {
    if (H <= 0 || I <= 0 || act_mode < MOE_ACT_BF16 || act_mode > MOE_ACT_FP8_SHARED) return 0;
    return moe::layer_workspace_bytes(T, E, K, H, I, has_shared, act_mode);
  }
  if (op == MOE_OP_EXPERT_FFN || op == MOE_OP_EXPERT_FFN_COMBINE) {
    if (H <= 0 || I <= 0 || act_mode < MOE_ACT_BF16 || act_mode > MOE_ACT_FP8_SHARED) return 0;
    return op == MOE_OP_EXPERT_FFN ? moe::ffn_workspace_bytes(T, K, H, I, has_shared, act_mode)
                                   : moe::ffn_combine_workspace_bytes(T, K, H, I, has_shared, act_mode);
  }
  return 0;
}

int moe_route_topk(const float* logits, int T, int E, int K, int32_t* ids, float* w,
                   void* stream) {
  if (!logits || !ids || !w) return fail(MOE_EINVAL, "moe_route_topk: null pointer");
  if (!sizes_ok_common(T, E, K))
    return fail(MOE_EINVAL, "moe_route_topk: need T >= 1, 1 <= K <= min(E, 32), E <= 1024 (T=%d E=%d K=%d)", T, E, K);
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  hipError_t e = moe::launch_route_topk(logits, T, E, K, ids, w, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "moe_route_topk launch");
}

int moe_permute(const int32_t* ids, int T, int E, int K, int has_shared, int32_t* counts,
                int32_t* offsets, int32_t* sorted_slot, int32_t* slot_pos, int32_t* groups,
                void* ws, size_t ws_bytes, void* stream) {
  if (!ids || !counts || !offsets || !sorted_slot || !slot_pos || !groups)
    return fail(MOE_EINVAL, "moe_permute: null pointer");
  if (!sizes_ok_common(T, E, K) || (has_shared != 0 && has_shared != 1))
    return fail(MOE_EINVAL, "moe_permute: need T >= 1, 1 <= K <= min(E, 32), E <= 1024, has_shared in {0,1}");
  if (!slots_ok(T, K, has_shared))
    return fail(MOE_EINVAL, "moe_permute: T*(K + has_shared) must be below 2^31 (T=%d K=%d)", T, K);
  const size_t need = moe::permute_workspace_bytes(T, E, K);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(MOE_EWORKSPACE, "moe_permute: workspace of %zu bytes needed, %zu given", need, ws_bytes);
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  hipError_t e = moe::launch_permute(ids, T, E, K, has_shared, counts, offsets, sorted_slot,
                                     slot_pos, groups, ws, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "moe_permute launch");
}

int moe_expert_ffn(const moe_nvfp4_weights* W, const uint16_t* x, int T, int K,
                   const int32_t* offsets, const int32_t* sorted_slot, const int32_t* groups,
                   int act_mode, uint16_t* y_slots, void* ws, size_t ws_bytes, void* stream) {
  if (!W || !x || !offsets || !sorted_slot || !groups || !y_slots)
    return fail(MOE_EINVAL, "moe_expert_ffn: null pointer");
  if (!W->gu_codes || !W->gu_scales || !W->dn_codes || !W->dn_scales || !W->scale2)
    return fail(MOE_EINVAL, "moe_expert_ffn: null weight pointer");
  if (act_mode < MOE_ACT_BF16 || act_mode > MOE_ACT_FP8_SHARED)
    return fail(MOE_EUNSUPPORTED, "moe_expert_ffn: unknown act_mode %d", act_mode);
  if (!sizes_ok_common(T, W->E, K) || (W->has_shared != 0 && W->has_shared != 1))
    return fail(MOE_EINVAL, "moe_expert_ffn: need T >= 1, 1 <= K <= min(E, 32), E <= 1024, has_shared in {0,1}");
  if (W->H < 256 || W->H > 4096 || W->H % 256 != 0 || W->I < 128 || W->I > 1024 || W->I % 128 != 0)
    return fail(MOE_EINVAL, "moe_expert_ffn: need H a multiple of 256 in [256, 4096] and I a multiple of 128 in [128, 1024] (H=%d I=%d)", W->H, W->I);
  const size_t need = moe::ffn_workspace_bytes(T, K, W->H, W->I, W->has_shared, act_mode);
  if (!ws || ws_bytes < need)
    return fail(MOE_EWORKSPACE, "moe_expert_ffn: workspace of %zu bytes needed, %zu given", need, ws_bytes);
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  hipError_t e = moe::launch_expert_ffn(*W, x, T, K, offsets, sorted_slot, groups, act_mode,
                                        y_slots, ws, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "moe_expert_ffn launch");
}

int moe_expert_ffn_noalloc(const moe_nvfp4_weights* W, const uint16_t* x, int T, int K,
                           const int32_t* offsets, const int32_t* sorted_slot,
                           const int32_t* groups, int act_mode, uint16_t* y_slots,
                           void* stream) {
  if (!W || !x || !offsets || !sorted_slot || !groups || !y_slots)
    return fail(MOE_EINVAL, "moe_expert_ffn_noalloc: null pointer");
  if (!W->gu_codes || !W->gu_scales || !W->dn_codes || !W->dn_scales || !W->scale2)
    return fail(MOE_EINVAL, "moe_expert_ffn_noalloc: null weight pointer");
  if (act_mode < MOE_ACT_BF16 || act_mode > MOE_ACT_FP8_SHARED)
    return fail(MOE_EUNSUPPORTED, "moe_expert_ffn_noalloc: unknown act_mode %d", act_mode);
  if (!sizes_ok_common(T, W->E, K) || (W->has_shared != 0 && W->has_shared != 1))
    return fail(MOE_EINVAL, "moe_expert_ffn_noalloc: need T >= 1, 1 <= K <= min(E, 32), E <= 1024, has_shared in {0,1}");
  if (W->H < 256 || W->H > 4096 || W->H % 256 != 0 || W->I < 128 || W->I > 1024 || W->I % 128 != 0)
    return fail(MOE_EINVAL, "moe_expert_ffn_noalloc: need H a multiple of 256 in [256, 4096] and I a multiple of 128 in [128, 1024] (H=%d I=%d)", W->H, W->I);
  const size_t need = moe::ffn_workspace_bytes(T, K, W->H, W->I, W->has_shared, act_mode);
  if (need > (size_t)MOE_NOALLOC_WS_BYTES)
    return fail(MOE_EWORKSPACE,
                "moe_expert_ffn_noalloc: these sizes need %zu bytes of workspace, more than the "
                "library's fixed %zu (use moe_expert_ffn with a caller workspace)",
                need, (size_t)MOE_NOALLOC_WS_BYTES);
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e, "hipGetDevice");
  e = moe::launch_expert_ffn(*W, x, T, K, offsets, sorted_slot, groups, act_mode, y_slots,
                             g_scratch[dev], (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "moe_expert_ffn_noalloc launch");
}

int moe_route_permute(const float* logits, int T, int E, int K, int has_shared, int32_t* ids,
                      float* w, int32_t* counts, int32_t* offsets, int32_t* sorted_slot,
                      int32_t* slot_pos, int32_t* groups, void* ws, size_t ws_bytes,
                      void* stream) {
  if (!logits || !ids || !w || !counts || !offsets || !sorted_slot || !slot_pos || !groups)
    return fail(MOE_EINVAL, "moe_route_permute: null pointer");
  if (!sizes_ok_common(T, E, K) || (has_shared != 0 && has_shared != 1))
    return fail(MOE_EINVAL, "moe_route_permute: need T >= 1, 1 <= K <= min(E, 32), E <= 1024, has_shared in {0,1}");
  if (!slots_ok(T, K, has_shared))
    return fail(MOE_EINVAL, "moe_route_permute: T*(K + has_shared) must be below 2^31 (T=%d K=%d)", T, K);
  const size_t need = moe::permute_workspace_bytes(T, E, K);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(MOE_EWORKSPACE, "moe_route_permute: workspace of %zu bytes needed, %zu given", need, ws_bytes);
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  hipError_t e = moe::launch_route_permute(logits, T, E, K, has_shared, ids, w, counts, offsets,
                                           sorted_slot, slot_pos, groups, ws, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "moe_route_permute launch");
}

int moe_expert_ffn_combine(const moe_nvfp4_weights* W, const uint16_t* x, int T, int K,
                           const int32_t* offsets, const int32_t* sorted_slot,
                           const int32_t* groups, int act_mode, const float* w,
                           const int32_t* slot_pos, const float* gate, uint16_t* y_slots,
                           uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
  if (!W || !x || !offsets || !sorted_slot || !groups || !w || !slot_pos || !y_slots || !out)
    return fail(MOE_EINVAL, "moe_expert_ffn_combine: null pointer");
  if (!W->gu_codes || !W->gu_scales || !W->dn_codes || !W->dn_scales || !W->scale2)
    return fail(MOE_EINVAL, "moe_expert_ffn_combine: null weight pointer");
  if (act_mode < MOE_ACT_BF16 || act_mode > MOE_ACT_FP8_SHARED)
    return fail(MOE_EUNSUPPORTED, "moe_expert_ffn_combine: unknown act_mode %d", act_mode);
  if (!sizes_ok_common(T, W->E, K) || (W->has_shared != 0 && W->has_shared != 1))
    return fail(MOE_EINVAL, "moe_expert_ffn_combine: need T >= 1, 1 <= K <= min(E, 32), E <= 1024, has_shared in {0,1}");
  if (W->H < 256 || W->H > 4096 || W->H % 256 != 0 || W->I < 128 || W->I > 1024 || W->I % 128 != 0)
    return fail(MOE_EINVAL, "moe_expert_ffn_combine: need H a multiple of 256 in [256, 4096] and I a multiple of 128 in [128, 1024] (H=%d I=%d)", W->H, W->I);
  if (gate && !W->has_shared)
    return fail(MOE_EINVAL, "moe_expert_ffn_combine: a shared-expert gate needs has_shared");
  const size_t need = moe::ffn_combine_workspace_bytes(T, K, W->H, W->I, W->has_shared, act_mode);
  if (!ws || ws_bytes < need)
    return fail(MOE_EWORKSPACE, "moe_expert_ffn_combine: workspace of %zu bytes needed, %zu given", need, ws_bytes);
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  hipError_t e = moe::launch_expert_ffn_combine(*W, x, T, K, offsets, sorted_slot, groups, act_mode,
                                                w, slot_pos, gate, y_slots, out, ws,
                                                (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "moe_expert_ffn_combine launch");
}

int moe_layer(const moe_nvfp4_weights* W, const float* logits, const uint16_t* x, int T, int K,
              int act_mode, const float* gate, int32_t* ids, float* w, int32_t* counts,
              int32_t* offsets, int32_t* sorted_slot, int32_t* slot_pos, int32_t* groups,
              uint16_t* y_slots, uint16_t* out, void* ws, size_t ws_bytes, void* stream) {
  if (!W || !logits || !x || !ids || !w || !counts || !offsets || !sorted_slot || !slot_pos ||
      !groups || !y_slots || !out)
    return fail(MOE_EINVAL, "moe_layer: null pointer");
  if (!W->gu_codes || !W->gu_scales || !W->dn_codes || !W->dn_scales || !W->scale2)
    return fail(MOE_EINVAL, "moe_layer: null weight pointer");
  if (act_mode < MOE_ACT_BF16 || act_mode > MOE_ACT_FP8_SHARED)
    return fail(MOE_EUNSUPPORTED, "moe_layer: unknown act_mode %d", act_mode);
  if (!sizes_ok_common(T, W->E, K) || (W->has_shared != 0 && W->has_shared != 1))
    return fail(MOE_EINVAL, "moe_layer: need T >= 1, 1 <= K <= min(E, 32), E <= 1024, has_shared in {0,1}");
  if (W->H < 256 || W->H > 4096 || W->H % 256 != 0 || W->I < 128 || W->I > 1024 || W->I % 128 != 0)
    return fail(MOE_EINVAL, "moe_layer: need H a multiple of 256 in [256, 4096] and I a multiple of 128 in [128, 1024] (H=%d I=%d)", W->H, W->I);
  if (gate && !W->has_shared)
    return fail(MOE_EINVAL, "moe_layer: a shared-expert gate needs has_shared");
  const size_t need = moe::layer_workspace_bytes(T, W->E, K, W->H, W->I, W->has_shared, act_mode);
  if (!ws || ws_bytes < need)
    return fail(MOE_EWORKSPACE, "moe_layer: workspace of %zu bytes needed, %zu given", need, ws_bytes);
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  const moe::RpOut ro{ids, w, counts, offsets, sorted_slot, slot_pos, groups};
  hipError_t e = moe::launch_layer(*W, logits, x, T, K, act_mode, gate, ro, y_slots, out, ws,
                                   (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "moe_layer launch");
}

int moe_combine(const uint16_t* y_slots, const float* w, const int32_t* slot_pos, int T, int K,
                int H, int has_shared, uint16_t* out, void* stream) {
  if (!y_slots || !w || !slot_pos || !out) return fail(MOE_EINVAL, "moe_combine: null pointer");
  if (T < 1 || K < 1 || K > 32 || H < 8 || H % 8 != 0 || (has_shared != 0 && has_shared != 1) ||
      (long long)T * K > (1LL << 30))
    return fail(MOE_EINVAL, "moe_combine: need T >= 1, 1 <= K <= 32, H a positive multiple of 8, has_shared in {0,1}");
  if (!slots_ok(T, K, has_shared))
    return fail(MOE_EINVAL, "moe_combine: T*(K + has_shared) must be below 2^31 (T=%d K=%d)", T, K);
  if (!grid_ok(moe::combine_threads(T, H))) return too_many_rows("moe_combine", T);
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  hipError_t e = moe::launch_combine(y_slots, w, slot_pos, nullptr, T, K, H, has_shared, out,
                                     (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "moe_combine launch");
}

int moe_combine_gated(const uint16_t* y_slots, const float* w, const int32_t* slot_pos,
                      const float* gate, int T, int K, int H, uint16_t* out, void* stream) {
  if (!y_slots || !w || !slot_pos || !gate || !out)
    return fail(MOE_EINVAL, "moe_combine_gated: null pointer");
  if (T < 1 || K < 1 || K > 32 || H < 8 || H % 8 != 0 || (long long)T * K > (1LL << 30))
    return fail(MOE_EINVAL, "moe_combine_gated: need T >= 1, 1 <= K <= 32, H a positive multiple of 8");
  if (!slots_ok(T, K, 1))
    return fail(MOE_EINVAL, "moe_combine_gated: T*(K + 1) must be below 2^31 (T=%d K=%d)", T, K);
  if (!grid_ok(moe::combine_threads(T, H))) return too_many_rows("moe_combine_gated", T);
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  hipError_t e = moe::launch_combine(y_slots, w, slot_pos, gate, T, K, H, 1, out, (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "moe_combine_gated launch");
}

int moe_router_topk(const moe_nvfp4_router* R, const uint16_t* x, int T, int K, int32_t* ids,
                    float* w, float* logits, float* gate, void* stream) {
  if (!R || !x || !ids || !w || !logits) return fail(MOE_EINVAL, "moe_router_topk: null pointer");
  if (!R->codes || !R->scales) return fail(MOE_EINVAL, "moe_router_topk: null weight pointer");
  if (R->has_gate != 0 && R->has_gate != 1)
    return fail(MOE_EINVAL, "moe_router_topk: has_gate must be 0 or 1");
  if (R->has_gate && !gate)
    return fail(MOE_EINVAL, "moe_router_topk: the matrix has a gate row but gate is NULL");
  if (!sizes_ok_common(T, R->E, K))
    return fail(MOE_EINVAL, "moe_router_topk: need T >= 1, 1 <= K <= min(E, 32), E <= 1024 (T=%d E=%d K=%d)", T, R->E, K);
  if (R->H < 256 || R->H > 8192 || R->H % 256 != 0 || (long long)T * R->H >= (1LL << 30))
    return fail(MOE_EINVAL, "moe_router_topk: need H a multiple of 256 in [256, 8192] and T*H < 2^30 (T=%d H=%d)", T, R->H);
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  hipError_t e = moe::launch_router_topk(*R, x, T, K, ids, w, logits, R->has_gate ? gate : nullptr,
                                         (hipStream_t)stream);
  return e == hipSuccess ? ok() : hip_fail(e, "moe_router_topk launch");
}

int moe_dispatch(const void* x, const int32_t* slot_pos, int T, int K, int H, int has_shared,
                 int dtype, void* xs, void* stream) {
  if (!x || !slot_pos || !xs) return fail(MOE_EINVAL, "moe_dispatch: null pointer");
  int rc = sort_sizes("moe_dispatch", T, K, H, has_shared, dtype);
  if (rc != MOE_OK) return rc;
  if (!grid_ok(moe::slot_rows_threads(T, H, dtype))) return too_many_rows("moe_dispatch", T);
  if (!aligned16((const char*)x, (const char*)xs))
    return fail(MOE_EINVAL, "moe_dispatch: rows must be aligned to 16 bytes");
  rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_dispatch(x, slot_pos, T, K, H, has_shared, dtype, xs, (hipStream_t)stream),
                  "moe_dispatch launch");
}

int moe_dispatch_grad(const void* dxs, const int32_t* slot_pos, int T, int K, int H,
                      int has_shared, int dtype, void* dx, void* stream) {
  if (!dxs || !slot_pos || !dx) return fail(MOE_EINVAL, "moe_dispatch_grad: null pointer");
  int rc = sort_sizes("moe_dispatch_grad", T, K, H, has_shared, dtype);
  if (rc != MOE_OK) return rc;
  if (!grid_ok(moe::slot_rows_threads(T, H, dtype))) return too_many_rows("moe_dispatch_grad", T);
  if (!aligned16((const char*)dxs, (const char*)dx))
    return fail(MOE_EINVAL, "moe_dispatch_grad: rows must be aligned to 16 bytes");
  rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_slot_sum(dxs, nullptr, slot_pos, nullptr, T, K, H, has_shared, dtype,
                                       dx, (hipStream_t)stream),
                  "moe_dispatch_grad launch");
}

int moe_combine_typed(const void* y_slots, const float* w, const int32_t* slot_pos,
                      const float* gate, int T, int K, int H, int has_shared, int dtype, void* out,
                      void* stream) {
  if (!y_slots || !w || !slot_pos || !out) return fail(MOE_EINVAL, "moe_combine_typed: null pointer");
  int rc = sort_sizes("moe_combine_typed", T, K, H, has_shared, dtype);
  if (rc != MOE_OK) return rc;
  if (!grid_ok(dtype == MOE_DT_BF16 ? moe::combine_threads(T, H) : moe::slot_rows_threads(T, H, dtype)))
    return too_many_rows("moe_combine_typed", T);
  if (gate && !has_shared)
    return fail(MOE_EINVAL, "moe_combine_typed: a shared-expert gate needs has_shared");
  if (!aligned16((const char*)y_slots, (const char*)out))
    return fail(MOE_EINVAL, "moe_combine_typed: rows must be aligned to 16 bytes");
  rc = ensure_init();
  if (rc != MOE_OK) return rc;
  hipStream_t s = (hipStream_t)stream;
  return launched(dtype == MOE_DT_BF16
                      ? moe::launch_combine((const uint16_t*)y_slots, w, slot_pos, gate, T, K, H,
                                            has_shared, (uint16_t*)out, s)
                      : moe::launch_slot_sum(y_slots, w, slot_pos, gate, T, K, H, has_shared,
                                             dtype, out, s),
                  "moe_combine_typed launch");
}

int moe_combine_grad(const void* dout, const void* y_slots, const float* w,
                     const int32_t* slot_pos, const float* gate, int T, int K, int H,
                     int has_shared, int dtype, void* dy_slots, float* dw, float* dgate,
                     void* stream) {
  if (!dout || !y_slots || !w || !slot_pos || !dy_slots || !dw)
    return fail(MOE_EINVAL, "moe_combine_grad: null pointer");
  int rc = sort_sizes("moe_combine_grad", T, K, H, has_shared, dtype);
  if (rc != MOE_OK) return rc;
  if (!grid_ok(moe::wave_rows_threads((long long)T * (K + has_shared))))
    return too_many_rows("moe_combine_grad", T);
  if (gate && !has_shared)
    return fail(MOE_EINVAL, "moe_combine_grad: a shared-expert gate needs has_shared");
  if ((gate != nullptr) != (dgate != nullptr))
    return fail(MOE_EINVAL, "moe_combine_grad: gate and dgate are given together");
  if (!aligned16((const char*)dout, (const char*)y_slots, (const char*)dy_slots))
    return fail(MOE_EINVAL, "moe_combine_grad: rows must be aligned to 16 bytes");
  rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_combine_grad(dout, y_slots, w, slot_pos, gate, T, K, H, has_shared,
                                           dtype, dy_slots, dw, dgate, (hipStream_t)stream),
                  "moe_combine_grad launch");
}

int moe_route_topk_grad(const int32_t* ids, const float* w, const float* dw, int T, int E, int K,
                        float* dlogits, void* stream) {
  if (!ids || !w || !dw || !dlogits) return fail(MOE_EINVAL, "moe_route_topk_grad: null pointer");
  if (!sizes_ok_common(T, E, K))
    return fail(MOE_EINVAL, "moe_route_topk_grad: need T >= 1, 1 <= K <= min(E, 32), E <= 1024 (T=%d E=%d K=%d)", T, E, K);
  if (!grid_ok(moe::wave_rows_threads(T))) return too_many_rows("moe_route_topk_grad", T);
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_topk_grad(ids, w, dw, T, E, K, dlogits, (hipStream_t)stream),
                  "moe_route_topk_grad launch");
}

static int norm_sizes(const char* who, int T, int H, int dtype, int gate_kind) {
  if (!dtype_ok(dtype)) return fail(MOE_EUNSUPPORTED, "%s: unknown dtype %d", who, dtype);
  if (gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_ELEMENT)
    return fail(MOE_EUNSUPPORTED, "%s: unknown gate_kind %d", who, gate_kind);
  if (T < 1 || T > (1 << 30) || H < 8 || H > 8192 || H % 8 != 0)
    return fail(MOE_EINVAL, "%s: need 1 <= T <= 2^30 and H a multiple of 8 in [8, 8192] (T=%d H=%d)", who, T, H);
  return MOE_OK;
}

int moe_block_norm(const void* residual, const void* y, const void* gate, int gate_kind,
                   const float* w_post, const float* w_pre, float res_scale, float out_scale,
                   float eps, int T, int H, int dtype, void* r_out, void* n_out, float* rstd_post,
                   float* rstd_pre, void* stream) {
  if (!residual) return fail(MOE_EINVAL, "moe_block_norm: null pointer");
  int rc = norm_sizes("moe_block_norm", T, H, dtype, gate_kind);
  if (rc != MOE_OK) return rc;
  if (!grid_ok(moe::block_norm_threads(T, H, dtype))) return too_many_rows("moe_block_norm", T);
  if ((gate_kind == MOE_GATE_NONE) != (gate == nullptr))
    return fail(MOE_EINVAL, "moe_block_norm: gate and gate_kind do not agree");
  if (!y && (gate || w_post || r_out || !w_pre))
    return fail(MOE_EINVAL, "moe_block_norm: without y only w_pre and n_out are given");
  if (y && !r_out) return fail(MOE_EINVAL, "moe_block_norm: r_out is missing");
  if ((w_pre != nullptr) != (n_out != nullptr))
    return fail(MOE_EINVAL, "moe_block_norm: w_pre and n_out are given together");
  if ((rstd_post && !w_post) || (rstd_pre && !w_pre))
    return fail(MOE_EINVAL, "moe_block_norm: statistics of a norm that is not computed");
  if (!(eps >= 0.f)) return fail(MOE_EINVAL, "moe_block_norm: eps must be >= 0");
  if (!aligned16((const char*)residual, (const char*)y, (const char*)w_post, (const char*)w_pre,
                 (const char*)r_out, (const char*)n_out) ||
      (gate_kind == MOE_GATE_ELEMENT && !aligned16((const char*)gate)))
    return fail(MOE_EINVAL, "moe_block_norm: rows and weights must be aligned to 16 bytes");
  rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_block_norm(residual, y, gate, gate_kind, w_post, w_pre, res_scale,
                                         out_scale, eps, T, H, dtype, r_out, n_out, rstd_post,
                                         rstd_pre, (hipStream_t)stream),
                  "moe_block_norm launch");
}

size_t moe_block_norm_workspace_bytes(int T, int H, int dtype) {
  if (!dtype_ok(dtype) || T < 1 || T > (1 << 30) || H < 8 || H > 8192 || H % 8 != 0) return 0;
  return moe::block_norm_workspace_bytes(T, H, dtype);
}

int moe_block_norm_grad(const void* dr, const void* dn, const void* r_out, const void* y,
                        const void* gate, int gate_kind, const float* w_post, const float* w_pre,
                        const float* rstd_post, const float* rstd_pre, float res_scale,
                        float out_scale, int T, int H, int dtype, void* dres, void* dy,
                        void* dgate, float* dw_post, float* dw_pre, void* ws, size_t ws_bytes,
                        void* stream) {
  if (!dres || (!dr && !dn)) return fail(MOE_EINVAL, "moe_block_norm_grad: null pointer");
  int rc = norm_sizes("moe_block_norm_grad", T, H, dtype, gate_kind);
  if (rc != MOE_OK) return rc;
  if ((gate_kind == MOE_GATE_NONE) != (gate == nullptr) || (gate != nullptr) != (dgate != nullptr))
    return fail(MOE_EINVAL, "moe_block_norm_grad: gate, gate_kind and dgate do not agree");
  if (!y && (gate || w_post || dy))
    return fail(MOE_EINVAL, "moe_block_norm_grad: without y there is no gate, w_post or dy");
  if (y && !dy) return fail(MOE_EINVAL, "moe_block_norm_grad: dy is missing");
  if (w_pre ? !(dn && r_out && rstd_pre && dw_pre) : (dn || dw_pre))
    return fail(MOE_EINVAL, "moe_block_norm_grad: w_pre, dn, r_out, rstd_pre and dw_pre are given together");
  if (w_post ? !(rstd_post && dw_post) : dw_post != nullptr)
    return fail(MOE_EINVAL, "moe_block_norm_grad: w_post, rstd_post and dw_post are given together");
  if (!aligned16((const char*)dr, (const char*)dn, (const char*)r_out, (const char*)y,
                 (const char*)w_post, (const char*)w_pre, (const char*)dres, (const char*)dy,
                 (const char*)ws) ||
      (gate_kind == MOE_GATE_ELEMENT && !aligned16((const char*)gate, (const char*)dgate)))
    return fail(MOE_EINVAL, "moe_block_norm_grad: rows, weights and workspace must be aligned to 16 bytes");
  const size_t need = moe::block_norm_workspace_bytes(T, H, dtype);
  if (!ws || ws_bytes < need)
    return fail(MOE_EWORKSPACE, "moe_block_norm_grad: workspace of %zu bytes needed, %zu given", need, ws_bytes);
  rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_block_norm_grad(dr, dn, r_out, y, gate, gate_kind, w_post, w_pre,
                                              rstd_post, rstd_pre, res_scale, out_scale, T, H,
                                              dtype, dres, dy, dgate, dw_post, dw_pre, ws,
                                              (hipStream_t)stream),
                  "moe_block_norm_grad launch");
}

static bool fp8_k_ok(int T, int K) {
  return T >= 1 && T <= (1 << 30) && K >= 16 && K <= 65536 && K % 16 == 0;
}

int moe_fp8_quant(const void* x, int T, int K, int dtype, uint8_t* codes, float* scales,
                  void* stream) {
  if (!x || !codes || !scales) return fail(MOE_EINVAL, "moe_fp8_quant: null pointer");
  if (!dtype_ok(dtype)) return fail(MOE_EUNSUPPORTED, "moe_fp8_quant: unknown dtype %d", dtype);
  if (!fp8_k_ok(T, K))
    return fail(MOE_EINVAL, "moe_fp8_quant: need 1 <= T <= 2^30 and K a multiple of 16 in [16, 65536] (T=%d K=%d)", T, K);
  if (!grid_ok(moe::fp8_quant_threads(T, K))) return too_many_rows("moe_fp8_quant", T);
  if (!aligned16((const char*)x, codes))
    return fail(MOE_EINVAL, "moe_fp8_quant: rows must be aligned to 16 bytes");
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_fp8_quant(x, T, K, dtype, codes, scales, (hipStream_t)stream),
                  "moe_fp8_quant launch");
}

static bool fp8_matrix_ok(int T, int N, int K) {
  return fp8_k_ok(T, K) && N >= 8 && N <= 65536 && N % 8 == 0;
}

size_t moe_fp8_linear_workspace_bytes(int T, int N, int K) {
  return fp8_matrix_ok(T, N, K) ? moe::fp8_linear_workspace_bytes(T, N, K) : 0;
}

int moe_fp8_linear(const moe_fp8_matrix* M, const void* x, int T, int dtype, void* out, void* ws,
                   size_t ws_bytes, void* stream) {
  if (!M || !x || !out) return fail(MOE_EINVAL, "moe_fp8_linear: null pointer");
  if (!M->codes || !M->scales) return fail(MOE_EINVAL, "moe_fp8_linear: null weight pointer");
  if (!dtype_ok(dtype)) return fail(MOE_EUNSUPPORTED, "moe_fp8_linear: unknown dtype %d", dtype);
  if (!fp8_matrix_ok(T, M->N, M->K))
    return fail(MOE_EINVAL, "moe_fp8_linear: need 1 <= T <= 2^30, K a multiple of 16 in [16, 65536] and N a multiple of 8 in [8, 65536] (T=%d N=%d K=%d)", T, M->N, M->K);
  if (!grid_ok(moe::fp8_linear_threads(T, M->N, M->K))) return too_many_rows("moe_fp8_linear", T);
  if (!aligned16((const char*)x, (const char*)out, M->codes, (const char*)ws))
    return fail(MOE_EINVAL, "moe_fp8_linear: codes, rows and workspace must be aligned to 16 bytes");
  const size_t need = moe::fp8_linear_workspace_bytes(T, M->N, M->K);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(MOE_EWORKSPACE, "moe_fp8_linear: workspace of %zu bytes needed, %zu given", need, ws_bytes);
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_fp8_linear(*M, x, T, dtype, out, ws, (hipStream_t)stream),
                  "moe_fp8_linear launch");
}

static bool fp8_bank_ok(int H, int I) {
  return H >= 128 && H <= 8192 && H % 128 == 0 && I >= 128 && I <= 8192 && I % 128 == 0;
}

size_t moe_fp8_expert_ffn_workspace_bytes(int T, int K, int H, int I, int has_shared) {
  if (T < 1 || K < 1 || K > 32 || (long long)T * K > (1LL << 30) || !fp8_bank_ok(H, I) ||
      (has_shared != 0 && has_shared != 1))
    return 0;
  return moe::fp8_expert_ffn_workspace_bytes(T, K, H, I, has_shared);
}

int moe_fp8_expert_ffn(const moe_fp8_weights* W, const uint16_t* x, int T, int K,
                       const int32_t* offsets, const int32_t* sorted_slot, const int32_t* groups,
                       uint16_t* y_slots, void* ws, size_t ws_bytes, void* stream) {
  if (!W || !x || !offsets || !sorted_slot || !groups || !y_slots)
    return fail(MOE_EINVAL, "moe_fp8_expert_ffn: null pointer");
  if (!W->gu_codes || !W->gu_scales || !W->dn_codes || !W->dn_scales)
    return fail(MOE_EINVAL, "moe_fp8_expert_ffn: null weight pointer");
  if (!sizes_ok_common(T, W->E, K) || (W->has_shared != 0 && W->has_shared != 1))
    return fail(MOE_EINVAL, "moe_fp8_expert_ffn: need T >= 1, 1 <= K <= min(E, 32), E <= 1024, has_shared in {0,1}");
  if (!fp8_bank_ok(W->H, W->I) || (long long)T * W->H >= (1LL << 32))
    return fail(MOE_EINVAL, "moe_fp8_expert_ffn: need H and I multiples of 128 in [128, 8192] and T*H < 2^32 (T=%d H=%d I=%d)", T, W->H, W->I);
  if (!grid_ok(moe::fp8_expert_ffn_threads(*W, T, K))) return too_many_rows("moe_fp8_expert_ffn", T);
  if (!aligned16((const char*)x, (const char*)y_slots, W->gu_codes, W->dn_codes, (const char*)ws))
    return fail(MOE_EINVAL, "moe_fp8_expert_ffn: codes, rows and workspace must be aligned to 16 bytes");
  const size_t need = moe::fp8_expert_ffn_workspace_bytes(T, K, W->H, W->I, W->has_shared);
  if (!ws || ws_bytes < need)
    return fail(MOE_EWORKSPACE, "moe_fp8_expert_ffn: workspace of %zu bytes needed, %zu given", need, ws_bytes);
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_fp8_expert_ffn(*W, x, T, K, offsets, sorted_slot, groups, y_slots, ws,
                                             (hipStream_t)stream),
                  "moe_fp8_expert_ffn launch");
}

static bool dense_sizes_ok(int T, int H, int I) {
  return T >= 1 && T <= (1 << 30) && H >= 8 && H <= 65536 && H % 8 == 0 && I >= 8 && I <= 65536 &&
         I % 8 == 0;
}

// What both dense entry points ask of the weights and the sizes.
static int dense_ok(const char* what, const moe_dense_weights& W, int T,
                    uint64_t (*threads)(int, int, int)) {
  if (!W.gu || !W.dn) return fail(MOE_EINVAL, "%s: null weight pointer", what);
  if (W.dtype != MOE_DT_BF16 && W.dtype != MOE_DT_F16)
    return fail(MOE_EUNSUPPORTED, "%s: dtype %d is not bf16 or f16", what, W.dtype);
  if (!dense_sizes_ok(T, W.H, W.I))
    return fail(MOE_EINVAL, "%s: need 1 <= T <= 2^30, H and I multiples of 8 in [8, 65536] (T=%d H=%d I=%d)", what, T, W.H, W.I);
  if (!grid_ok(threads(T, W.H, W.I))) return too_many_rows(what, T);
  return MOE_OK;
}

size_t moe_dense_ffn_workspace_bytes(int T, int H, int I) {
  return dense_sizes_ok(T, H, I) ? moe::dense_ffn_workspace_bytes(T, H, I) : 0;
}

int moe_dense_ffn(const moe_dense_weights* W, const void* x, int T, void* y, void* gu_out,
                  void* ws, size_t ws_bytes, void* stream) {
  if (!W || !x || !y) return fail(MOE_EINVAL, "moe_dense_ffn: null pointer");
  int rc = dense_ok("moe_dense_ffn", *W, T, moe::dense_ffn_threads);
  if (rc != MOE_OK) return rc;
  if (!aligned16((const char*)x, (const char*)y, (const char*)gu_out, (const char*)W->gu,
                 (const char*)W->dn, (const char*)ws))
    return fail(MOE_EINVAL, "moe_dense_ffn: weights, rows and workspace must be aligned to 16 bytes");
  const size_t need = moe::dense_ffn_workspace_bytes(T, W->H, W->I);
  if (!ws || ws_bytes < need)
    return fail(MOE_EWORKSPACE, "moe_dense_ffn: workspace of %zu bytes needed, %zu given", need, ws_bytes);
  rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_dense_ffn(*W, x, T, y, gu_out, ws, (hipStream_t)stream),
                  "moe_dense_ffn launch");
}

size_t moe_dense_ffn_grad_workspace_bytes(int T, int H, int I) {
  return dense_sizes_ok(T, H, I) ? moe::dense_ffn_grad_workspace_bytes(T, H, I) : 0;
}

int moe_dense_ffn_grad(const moe_dense_weights* W, const void* dy, const void* x, const void* gu,
                       int T, void* dx, void* dw_gu, void* dw_dn, void* ws, size_t ws_bytes,
                       void* stream) {
  if (!W || !dy || !x || !gu || !dx || !dw_gu || !dw_dn)
    return fail(MOE_EINVAL, "moe_dense_ffn_grad: null pointer");
  int rc = dense_ok("moe_dense_ffn_grad", *W, T, moe::dense_ffn_grad_threads);
  if (rc != MOE_OK) return rc;
  if (!aligned16((const char*)dy, (const char*)x, (const char*)gu, (const char*)dx,
                 (const char*)dw_gu, (const char*)dw_dn, (const char*)W->gu, (const char*)W->dn,
                 (const char*)ws))
    return fail(MOE_EINVAL, "moe_dense_ffn_grad: weights, rows and workspace must be aligned to 16 bytes");
  const size_t need = moe::dense_ffn_grad_workspace_bytes(T, W->H, W->I);
  if (!ws || ws_bytes < need)
    return fail(MOE_EWORKSPACE, "moe_dense_ffn_grad: workspace of %zu bytes needed, %zu given", need, ws_bytes);
  rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_dense_ffn_grad(*W, dy, x, gu, T, dx, dw_gu, dw_dn, ws, (hipStream_t)stream),
                  "moe_dense_ffn_grad launch");
}

static bool int8_k_ok(int T, int K) { return T >= 1 && K >= 16 && K <= 65536 && K % 16 == 0; }
static bool int8_matrix_ok(int T, int N, int K) {
  return int8_k_ok(T, K) && N >= 8 && N <= 131072 && N % 8 == 0;
}

int moe_int8_quant(const void* x, int T, int K, int dtype, int8_t* codes, float* scales,
                   void* stream) {
  if (!x || !codes || !scales) return fail(MOE_EINVAL, "moe_int8_quant: null pointer");
  if (!dtype_ok(dtype)) return fail(MOE_EUNSUPPORTED, "moe_int8_quant: unknown dtype %d", dtype);
  if (!int8_k_ok(T, K))
    return fail(MOE_EINVAL, "moe_int8_quant: need T >= 1 and K a multiple of 16 in [16, 65536] (T=%d K=%d)", T, K);
  if (!grid_ok(moe::int8_quant_threads(T, K, dtype))) return too_many_rows("moe_int8_quant", T);
  if (!aligned16((const char*)x, (const char*)codes))
    return fail(MOE_EINVAL, "moe_int8_quant: rows must be aligned to 16 bytes");
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_int8_quant(x, T, K, dtype, codes, scales, (hipStream_t)stream),
                  "moe_int8_quant launch");
}

size_t moe_int8_linear_workspace_bytes(int T, int N, int K) {
  return int8_matrix_ok(T, N, K) ? moe::int8_linear_workspace_bytes(T, N, K) : 0;
}

int moe_int8_linear(const moe_int8_matrix* M, const void* x, int T, int dtype, int gated,
                    void* out, void* ws, size_t ws_bytes, void* stream) {
  if (!M || !x || !out) return fail(MOE_EINVAL, "moe_int8_linear: null pointer");
  if (!M->codes || !M->scales) return fail(MOE_EINVAL, "moe_int8_linear: null weight pointer");
  if (!dtype_ok(dtype)) return fail(MOE_EUNSUPPORTED, "moe_int8_linear: unknown dtype %d", dtype);
  if (gated != 0 && gated != 1) return fail(MOE_EINVAL, "moe_int8_linear: gated must be 0 or 1");
  if (!int8_matrix_ok(T, M->N, M->K) || (gated && M->N % 16))
    return fail(MOE_EINVAL, "moe_int8_linear: need T >= 1, K a multiple of 16 in [16, 65536] and N a multiple of 8 (gated: 16) in [8, 131072] (T=%d N=%d K=%d)", T, M->N, M->K);
  if (!grid_ok(moe::int8_linear_threads(T, M->N, M->K, dtype))) return too_many_rows("moe_int8_linear", T);
  if (!aligned16((const char*)x, (const char*)out, (const char*)M->codes, (const char*)ws))
    return fail(MOE_EINVAL, "moe_int8_linear: codes, rows and workspace must be aligned to 16 bytes");
  const size_t need = moe::int8_linear_workspace_bytes(T, M->N, M->K);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(MOE_EWORKSPACE, "moe_int8_linear: workspace of %zu bytes needed, %zu given", need, ws_bytes);
  int rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_int8_linear(*M, x, T, dtype, gated, out, ws, (hipStream_t)stream),
                  "moe_int8_linear launch");
}

// What both gradient entry points ask of the list; outs: its outputs too.
static int grad_list_ok(const char* what, const moe_grad_tensor* list, int count, bool outs) {
  if (!list) return fail(MOE_EINVAL, "%s: null pointer", what);
  if (count < 1 || count > (1 << 20))
    return fail(MOE_EINVAL, "%s: need between 1 and 2^20 tensors, got %d", what, count);
  for (int i = 0; i < count; ++i) {
    const moe_grad_tensor& g = list[i];
    if (!dtype_ok(g.dtype)) return fail(MOE_EUNSUPPORTED, "%s: tensor %d: unknown dtype %d", what, i, g.dtype);
    if (g.n < 0 || g.n > (1LL << 37))
      return fail(MOE_EINVAL, "%s: tensor %d: need 0 <= n <= 2^37, got %lld", what, i, (long long)g.n);
    if (g.n == 0) continue;
    if (!g.grad || (outs && !g.out)) return fail(MOE_EINVAL, "%s: tensor %d: null pointer", what, i);
    const uintptr_t es = g.dtype == MOE_DT_F32 ? 4 : 2;
    if ((uintptr_t)g.grad % es || (outs && (uintptr_t)g.out % es))
      return fail(MOE_EINVAL, "%s: tensor %d: not aligned to its type", what, i);
  }
  return MOE_OK;
}

// Two outputs of a list may not share memory (a tensor named twice), nor an output and a
// gradient but its own in place: the launches would read and scale them in an order of
// their own.
static int grad_outs_ok(const moe_grad_tensor* list, int count) {
  struct Range {
    uintptr_t from, to;
    int of;
  };
  const auto range = [&](const void* p, int i) {
    const uintptr_t at = (uintptr_t)p;
    return Range{at, at + (uintptr_t)list[i].n * (list[i].dtype == MOE_DT_F32 ? 4 : 2), i};
  };
  std::vector<Range> r;
  r.reserve((size_t)count);
  bool sorted = true, in_place = true;
  for (int i = 0; i < count; ++i) {
    if (list[i].n == 0) continue;
    r.push_back(range(list[i].out, i));
    sorted = sorted && (r.size() == 1 || r[r.size() - 2].from <= r.back().from);
    in_place = in_place && list[i].grad == list[i].out;
  }
  if (!sorted) std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.from < b.from; });
  for (size_t i = 1; i < r.size(); ++i)
    if (r[i].from < r[i - 1].to) return fail(MOE_EINVAL, "moe_grad_clip: two outputs overlap");
  for (int i = 0; i < count && !in_place; ++i) {
    if (list[i].n == 0) continue;
    const Range g = range(list[i].grad, i);
    // the first output that ends behind the gradient's begin, and those after it
    for (auto o = std::partition_point(r.begin(), r.end(), [&](const Range& o) { return o.to <= g.from; });
         o != r.end() && o->from < g.to; ++o)
      if (o->of != i || o->from != g.from)
        return fail(MOE_EINVAL, "moe_grad_clip: an output overlaps a gradient that is not its own");
  }
  return MOE_OK;
}

size_t moe_grad_norm_workspace_bytes(int count) {
  return count >= 1 && count <= (1 << 20) ? moe::grad_norm_workspace_bytes(count) : 0;
}

int moe_grad_norm(const moe_grad_tensor* list, int count, float* norm, void* ws, size_t ws_bytes,
                  void* stream) {
  if (!norm) return fail(MOE_EINVAL, "moe_grad_norm: null pointer");
  int rc = grad_list_ok("moe_grad_norm", list, count, false);
  if (rc != MOE_OK) return rc;
  const size_t need = moe::grad_norm_workspace_bytes(count);
  if (!ws || ws_bytes < need || (uintptr_t)ws % 8)
    return fail(MOE_EWORKSPACE, "moe_grad_norm: workspace of %zu bytes, aligned to 8, needed, %zu given", need, ws_bytes);
  rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_grad_norm(list, count, norm, (double*)ws, (hipStream_t)stream),
                  "moe_grad_norm launch");
}

int moe_grad_clip(const moe_grad_tensor* list, int count, const float* norm, float max_norm,
                  void* stream) {
  if (!norm) return fail(MOE_EINVAL, "moe_grad_clip: null pointer");
  if (!(max_norm >= 0.f && max_norm <= FLT_MAX))
    return fail(MOE_EINVAL, "moe_grad_clip: max_norm must be finite and not negative");
  int rc = grad_list_ok("moe_grad_clip", list, count, true);
  if (rc == MOE_OK) rc = grad_outs_ok(list, count);
  if (rc != MOE_OK) return rc;
  rc = ensure_init();
  if (rc != MOE_OK) return rc;
  return launched(moe::launch_grad_clip(list, count, norm, max_norm, (hipStream_t)stream),
                  "moe_grad_clip launch");
}

int moe_timing_enable(int on) {
  g_timing_on.store(on != 0);
  return ok();
}

int moe_timing_reset(void) {
  std::lock_guard<std::mutex> lk(g_tmu);
  g_used = 0;
  g_dropped = 0;
  return ok();
}

int moe_timing_read(const char** names, int* launches, double* total_ms, int max_names,
                    int* dropped) {
  if (max_names < 0 || (max_names > 0 && (!names || !launches || !total_ms)))
    return fail(MOE_EINVAL, "moe_timing_read: bad output arrays");
  std::lock_guard<std::mutex> lk(g_tmu);
  int n = 0;
  for (size_t i = 0; i < g_used; ++i) {
    TimingRec& r = g_pool[i];
    hipError_t e = hipEventSynchronize(r.b);
    if (e != hipSuccess) return hip_fail(e, "moe_timing_read: hipEventSynchronize");
    float ms = 0.f;
    e = hipEventElapsedTime(&ms, r.a, r.b);
    if (e != hipSuccess) return hip_fail(e, "moe_timing_read: hipEventElapsedTime");
    int j = 0;
    while (j < n && strcmp(names[j], r.name) != 0) ++j;
    if (j == n) {
      if (n == max_names) continue;
      names[n] = r.name;
      launches[n] = 0;
      total_ms[n] = 0.0;
      ++n;
    }
    launches[j] += 1;
    total_ms[j] += ms;
  }
  if (dropped) *dropped = (int)g_dropped;
  g_err.clear();
  return n;
}

}  // extern "C"
