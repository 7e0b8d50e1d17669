// C ABI of the routed MoE FFN layer (declared in include/moe.h): argument checking,
// workspace layout and dispatch to the kernels. No call allocates, frees or synchronises.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include "../../include/moe.h"
#include "kernels.hpp"

namespace {

thread_local char g_err[512] = "";

moe_status fail(moe_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return s;
}

moe_status ok() {
  g_err[0] = 0;
  return MOE_OK;
}

moe_status hip_status(hipError_t e, const char* where) {
  if (e == hipSuccess) return ok();
  return fail(MOE_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

bool known_fmt(int fmt) {
  return fmt == MOE_W_MXFP4 || fmt == MOE_W_Q8_0 || fmt == MOE_W_Q4_K || fmt == MOE_W_Q5_K ||
         fmt == MOE_W_Q6_K;
}
// k-quant formats: the reduction dimension must be a multiple of the 256-element super-block
bool superblocked(int fmt) { return fmt == MOE_W_Q4_K || fmt == MOE_W_Q5_K || fmt == MOE_W_Q6_K; }

// Launch errors are read back with hipGetLastError; drop any error an earlier, unrelated
// HIP call left behind so it is not reported as this call's failure.
void clear_stale_error() { (void)hipGetLastError(); }

#define CHECK_PTR(p)                                                                 \
  do {                                                                               \
    if ((p) == nullptr) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", #p);          \
    if (!aligned16(p)) return fail(MOE_ERR_INVALID_ARG, "%s is not 16-byte aligned", #p); \
  } while (0)

moe_status check_shape(int32_t T, int32_t H, int32_t E, int32_t k) {
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T = %d < 0", T);
  if (H <= 0 || H % 32) return fail(MOE_ERR_INVALID_ARG, "H = %d is not a positive multiple of 32", H);
  if (E < 1 || E > moe::kMaxE) return fail(MOE_ERR_INVALID_ARG, "E = %d outside [1, %d]", E, moe::kMaxE);
  if (k < 1 || k > moe::kMaxK) return fail(MOE_ERR_INVALID_ARG, "k = %d outside [1, %d]", k, moe::kMaxK);
  if (k > E) return fail(MOE_ERR_INVALID_ARG, "k = %d > E = %d", k, E);
  if ((int64_t)T * k > 0x3FFFFFFF) return fail(MOE_ERR_INVALID_ARG, "T*k too large");
  return MOE_OK;
}

// The grouped GEMM addresses gathered activation rows (x, and h for the down projection)
// as 32-bit indices of 16-byte units, so each of x [T x H] and h [T*k x I] must hold fewer
// than 2^35 bf16 elements (64 GiB).
constexpr int64_t kMaxActElems = int64_t(1) << 35;
moe_status check_extent(int32_t T, int32_t k, int32_t H, int32_t I) {
  if ((int64_t)T * H >= kMaxActElems)
    return fail(MOE_ERR_INVALID_ARG, "x holds T*H = %lld elements, limit 2^35",
                (long long)T * H);
  if ((int64_t)T * k * I >= kMaxActElems)
    return fail(MOE_ERR_INVALID_ARG, "h holds T*k*I = %lld elements, limit 2^35",
                (long long)T * k * I);
  return MOE_OK;
}

moe_status check_pool(const moe_pool* pool) {
  if (pool == nullptr) return fail(MOE_ERR_INVALID_ARG, "pool is NULL");
  if (!known_fmt(pool->fmt))
    return fail(MOE_ERR_UNSUPPORTED, "unknown weight format %d", pool->fmt);
  if (pool->n_slots < 1) return fail(MOE_ERR_INVALID_ARG, "n_slots = %d < 1", pool->n_slots);
  if (pool->H <= 0 || pool->H % 32) return fail(MOE_ERR_INVALID_ARG, "pool H = %d", pool->H);
  if (pool->I <= 0 || pool->I % 32) return fail(MOE_ERR_INVALID_ARG, "pool I = %d", pool->I);
  if (superblocked(pool->fmt) && (pool->H % 256 || pool->I % 256))
    return fail(MOE_ERR_INVALID_ARG, "k-quant pools need H and I to be multiples of 256 (H = %d, I = %d)",
                pool->H, pool->I);
  CHECK_PTR(pool->gate_q);
  CHECK_PTR(pool->up_q);
  CHECK_PTR(pool->down_q);
  CHECK_PTR(pool->gate_s);
  CHECK_PTR(pool->up_s);
  CHECK_PTR(pool->down_s);
  return MOE_OK;
}

size_t plane_bytes(int fmt, int64_t rows, int64_t K, bool scales) {
  if (scales) return (size_t)moe::scale_plane_bytes(fmt, rows, K);
  return (size_t)moe::code_plane_bytes(fmt, rows, K);
}

void pool_views(const moe_pool* p, moe::PoolView* g, moe::PoolView* u, moe::PoolView* d) {
  const int fmt = p->fmt;
  const int64_t gq = plane_bytes(fmt, p->I, p->H, false), gs = plane_bytes(fmt, p->I, p->H, true);
  const int64_t dq = plane_bytes(fmt, p->H, p->I, false), ds = plane_bytes(fmt, p->H, p->I, true);
  *g = {(const uint8_t*)p->gate_q, (const uint8_t*)p->gate_s, gq, gs};
  *u = {(const uint8_t*)p->up_q, (const uint8_t*)p->up_s, gq, gs};
  *d = {(const uint8_t*)p->down_q, (const uint8_t*)p->down_s, dq, ds};
}

size_t route_scratch(int32_t T, int32_t H, int32_t E) {
  if (moe::route_fused_ok(T, H, E))          // split router, finished by a later kernel
    return (size_t)moe::route_fused_split(H) * T * E * sizeof(float);
  if (moe::route_small_ok(T, E)) return 0;   // one workgroup, no partials
  const int ks = moe::route_ksplit(T, H);
  return ks > 1 ? (size_t)ks * T * E * sizeof(float) : 0;
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

bool use_gemv(int32_t path, int32_t T) {
  return path == MOE_PATH_GEMV || path == MOE_PATH_PERSISTENT ||
         (path == MOE_PATH_AUTO && T <= 16);
}

moe_status gate_up_dispatch(const moe_pool* pool, const int32_t* slot_map, int32_t E,
                            const uint16_t* x, int32_t T, int32_t k, const int32_t* offsets,
                            const int32_t* perm, uint16_t* h, uint32_t* err, int32_t path,
                            hipStream_t stream, const int32_t* act = nullptr) {
  clear_stale_error();
  moe::PoolView g, u, d;
  pool_views(pool, &g, &u, &d);
  if (use_gemv(path, T))
    return hip_status(moe::launch_gate_up_gemv(pool->fmt, g, u, slot_map, pool->n_slots, E, x, T,
                                               k, pool->H, pool->I, offsets, perm, h, err, act,
                                               stream),
                      "gate/up (GEMV)");
  return hip_status(moe::launch_gate_up_grouped(pool->fmt, g, u, slot_map, pool->n_slots, E, x, T,
                                                k, pool->H, pool->I, offsets, perm, h, err, stream),
                    "gate/up (grouped GEMM)");
}

moe_status down_dispatch(const moe_pool* pool, const int32_t* slot_map, int32_t E, int32_t T,
                         int32_t k, const int32_t* offsets, const uint16_t* h, float* y,
                         uint32_t* err, int32_t path, hipStream_t stream) {
  clear_stale_error();
  moe::PoolView g, u, d;
  pool_views(pool, &g, &u, &d);
  if (use_gemv(path, T))
    return hip_status(moe::launch_down_gemv(pool->fmt, d, slot_map, pool->n_slots, E, T, k,
                                            pool->H, pool->I, offsets, h, y, err, stream),
                      "down (GEMV)");
  return hip_status(moe::launch_down_grouped(pool->fmt, d, slot_map, pool->n_slots, E, T, k,
                                             pool->H, pool->I, offsets, h, y, err, stream),
                    "down (grouped GEMM)");
}

moe_status ffn_dispatch(const moe_pool* pool, const int32_t* slot_map, int32_t E,
                        const uint16_t* x, int32_t T, int32_t k, const int32_t* offsets,
                        const int32_t* perm, uint16_t* h, float* y, uint32_t* err,
                        int32_t path, hipStream_t stream) {
  moe_status s = gate_up_dispatch(pool, slot_map, E, x, T, k, offsets, perm, h, err, path, stream);
  if (s != MOE_OK) return s;
  return down_dispatch(pool, slot_map, E, T, k, offsets, h, y, err, path, stream);
}

// Shared argument checks of the expert-FFN entry points.
moe_status check_ffn_args(const moe_pool* pool, const int32_t* slot_map, int32_t E, int32_t T,
                          int32_t k, const int32_t* offsets, uint32_t* err_flags, int32_t path) {
  moe_status s = check_pool(pool);
  if (s != MOE_OK) return s;
  s = check_shape(T, pool->H, E, k);
  if (s != MOE_OK) return s;
  s = check_extent(T, k, pool->H, pool->I);
  if (s != MOE_OK) return s;
  if (path < MOE_PATH_AUTO || path > MOE_PATH_PERSISTENT)
    return fail(MOE_ERR_INVALID_ARG, "path = %d", path);
  if (T == 0) return MOE_OK;
  CHECK_PTR(slot_map);
  CHECK_PTR(offsets);
  if (err_flags != nullptr && ((uintptr_t)err_flags & 3))
    return fail(MOE_ERR_INVALID_ARG, "err_flags misaligned");
  return MOE_OK;
}

}  // namespace

// ---- moe_layer_noalloc: moe_layer with its workspace in a file-scope device array

// One array per device, held for the life of the process. In host code its name is only a
// stand-in for the symbol: kernels are given the device address that hipGetSymbolAddress
// returns for the current device, never the name itself.
static __device__ __align__(256) unsigned char scratch[MOE_NOALLOC_WS_BYTES];

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];   // address of `scratch` on each device, looked up once

// The device address of `scratch` on the device that `stream` belongs to, looked up (with
// that device current) on the first call for the device.
moe_status noalloc_workspace(hipStream_t stream, void** out) {
  int cur = -1;
  hipError_t e = hipGetDevice(&cur);
  if (e != hipSuccess) return hip_status(e, "hipGetDevice");
  int dev = cur;
  if (stream != nullptr) {
    hipDevice_t d = -1;
    e = hipStreamGetDevice(stream, &d);
    if (e != hipSuccess) return hip_status(e, "hipStreamGetDevice");
    dev = (int)d;
  }
  if (dev < 0 || dev >= kMaxDevices)
    return fail(MOE_ERR_INVALID_ARG, "device %d outside [0, %d)", dev, kMaxDevices);
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_ptr[dev] == nullptr) {
    if (dev != cur && (e = hipSetDevice(dev)) != hipSuccess) return hip_status(e, "hipSetDevice");
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    const hipError_t back = dev != cur ? hipSetDevice(cur) : hipSuccess;
    if (e != hipSuccess) return hip_status(e, "hipGetSymbolAddress(scratch)");
    if (back != hipSuccess) return hip_status(back, "hipSetDevice (restore)");
    if (p == nullptr || ((uintptr_t)p & 255))
      return fail(MOE_ERR_HIP, "static workspace at %p is not 256-byte aligned", p);
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return MOE_OK;
}
}  // namespace

extern "C" {

const char* moe_status_string(moe_status s) {
  switch (s) {
    case MOE_OK: return "MOE_OK";
    case MOE_ERR_INVALID_ARG: return "MOE_ERR_INVALID_ARG";
    case MOE_ERR_UNSUPPORTED: return "MOE_ERR_UNSUPPORTED";
    case MOE_ERR_HIP: return "MOE_ERR_HIP";
  }
  return "unknown moe_status";
}

const char* moe_last_error(void) { return g_err; }

size_t moe_plane_bytes(int32_t fmt, int32_t rows, int32_t K, int32_t scales) {
  if (!known_fmt(fmt) || rows < 0 || K < 0 || (superblocked(fmt) && K % 256)) return 0;
  return plane_bytes(fmt, rows, K, scales != 0);
}

moe_status moe_pool_pack(int32_t fmt, int32_t n_mats, int32_t rows, int32_t K,
                         const void* src_q, const void* src_s, void* dst_q, void* dst_s,
                         void* stream) {
  if (!known_fmt(fmt)) return fail(MOE_ERR_UNSUPPORTED, "unknown weight format %d", fmt);
  if (n_mats < 0 || rows < 0 || K < 0) return fail(MOE_ERR_INVALID_ARG, "negative size");
  if (rows % 16) return fail(MOE_ERR_INVALID_ARG, "rows = %d is not a multiple of 16", rows);
  if (K % 32) return fail(MOE_ERR_INVALID_ARG, "K = %d is not a multiple of 32", K);
  if (superblocked(fmt) && K % 256)
    return fail(MOE_ERR_INVALID_ARG, "k-quants need K = %d to be a multiple of 256", K);
  if (n_mats == 0 || rows == 0 || K == 0) return ok();
  CHECK_PTR(src_q);
  CHECK_PTR(dst_q);
  if (src_s == nullptr || dst_s == nullptr) return fail(MOE_ERR_INVALID_ARG, "scale plane is NULL");
  if (fmt == MOE_W_Q8_0 && (((uintptr_t)src_s | (uintptr_t)dst_s) & 1))
    return fail(MOE_ERR_INVALID_ARG, "fp16 scale plane is not 2-byte aligned");
  clear_stale_error();
  return hip_status(moe::launch_pack(fmt, n_mats, rows, K, src_q, src_s, dst_q, dst_s,
                                     (hipStream_t)stream),
                    "pool pack");
}

size_t moe_route_scratch_bytes(int32_t T, int32_t H, int32_t E) {
  if (T <= 0 || H <= 0 || E <= 0) return 0;
  return route_scratch(T, H, E);
}

moe_status moe_route(const uint16_t* x, const uint16_t* w_router, const float* bias, int32_t T,
                     int32_t H, int32_t E, int32_t k, int32_t* topk_ids, float* topk_w,
                     void* scratch, size_t scratch_bytes, void* stream) {
  moe_status s = check_shape(T, H, E, k);
  if (s != MOE_OK) return s;
  if (T == 0) return ok();
  CHECK_PTR(x);
  CHECK_PTR(w_router);
  CHECK_PTR(topk_ids);
  CHECK_PTR(topk_w);
  if (bias != nullptr && ((uintptr_t)bias & 3)) return fail(MOE_ERR_INVALID_ARG, "bias misaligned");
  const size_t need = route_scratch(T, H, E);
  if (need) {
    CHECK_PTR(scratch);
    if (scratch_bytes < need)
      return fail(MOE_ERR_INVALID_ARG, "route scratch %zu bytes < %zu needed", scratch_bytes, need);
  }
  clear_stale_error();
  return hip_status(moe::launch_route(x, w_router, bias, T, H, E, k, topk_ids, topk_w,
                                      (float*)scratch, (hipStream_t)stream),
                    "route");
}

size_t moe_bucket_scratch_bytes(int32_t T, int32_t k, int32_t E) {
  if (T <= 0 || k <= 0 || E <= 0) return 0;
  return moe::bucket_scratch_bytes(T * k, E);
}

moe_status moe_bucket(const int32_t* topk_ids, int32_t T, int32_t k, int32_t E, int32_t* counts,
                      int32_t* offsets, int32_t* perm, int32_t* inv_perm, void* scratch,
                      size_t scratch_bytes, void* stream) {
  moe_status s = check_shape(T, 32, E, k);
  if (s != MOE_OK) return s;
  CHECK_PTR(counts);
  CHECK_PTR(offsets);
  clear_stale_error();
  if (T == 0)   // empty input: one small kernel still writes all-zero counts and offsets
    return hip_status(moe::launch_bucket(nullptr, 0, E, counts, offsets, nullptr, nullptr,
                                         nullptr, (hipStream_t)stream),
                      "bucket");
  CHECK_PTR(topk_ids);
  CHECK_PTR(perm);
  CHECK_PTR(inv_perm);
  const size_t need = moe::bucket_scratch_bytes(T * k, E);
  if (need) {
    CHECK_PTR(scratch);
    if (scratch_bytes < need)
      return fail(MOE_ERR_INVALID_ARG, "bucket scratch %zu bytes < %zu needed", scratch_bytes, need);
  }
  return hip_status(moe::launch_bucket(topk_ids, T * k, E, counts, offsets, perm, inv_perm,
                                       scratch, (hipStream_t)stream),
                    "bucket");
}

moe_status moe_expert_ffn(const moe_pool* pool, const int32_t* slot_map, int32_t E,
                          const uint16_t* x, int32_t T, int32_t k, const int32_t* offsets,
                          const int32_t* perm, uint16_t* h, float* y, uint32_t* err_flags,
                          int32_t path, void* stream) {
  moe_status s = check_ffn_args(pool, slot_map, E, T, k, offsets, err_flags, path);
  if (s != MOE_OK || T == 0) return s == MOE_OK ? ok() : s;
  CHECK_PTR(x);
  CHECK_PTR(perm);
  CHECK_PTR(h);
  CHECK_PTR(y);
  return ffn_dispatch(pool, slot_map, E, x, T, k, offsets, perm, h, y, err_flags, path,
                      (hipStream_t)stream);
}

moe_status moe_expert_gate_up(const moe_pool* pool, const int32_t* slot_map, int32_t E,
                              const uint16_t* x, int32_t T, int32_t k, const int32_t* offsets,
                              const int32_t* perm, uint16_t* h, uint32_t* err_flags,
                              int32_t path, void* stream) {
  moe_status s = check_ffn_args(pool, slot_map, E, T, k, offsets, err_flags, path);
  if (s != MOE_OK || T == 0) return s == MOE_OK ? ok() : s;
  CHECK_PTR(x);
  CHECK_PTR(perm);
  CHECK_PTR(h);
  return gate_up_dispatch(pool, slot_map, E, x, T, k, offsets, perm, h, err_flags, path,
                          (hipStream_t)stream);
}

moe_status moe_expert_down(const moe_pool* pool, const int32_t* slot_map, int32_t E, int32_t T,
                           int32_t k, const int32_t* offsets, const uint16_t* h, float* y,
                           uint32_t* err_flags, int32_t path, void* stream) {
  moe_status s = check_ffn_args(pool, slot_map, E, T, k, offsets, err_flags, path);
  if (s != MOE_OK || T == 0) return s == MOE_OK ? ok() : s;
  CHECK_PTR(h);
  CHECK_PTR(y);
  return down_dispatch(pool, slot_map, E, T, k, offsets, h, y, err_flags, path,
                       (hipStream_t)stream);
}

moe_status moe_combine(const float* y, const int32_t* inv_perm, const float* topk_w, int32_t T,
                       int32_t k, int32_t H, float* out, void* stream) {
  moe_status s = check_shape(T, H, moe::kMaxE, k);
  if (s != MOE_OK) return s;
  if (T == 0) return ok();
  CHECK_PTR(y);
  CHECK_PTR(inv_perm);
  CHECK_PTR(topk_w);
  CHECK_PTR(out);
  clear_stale_error();
  return hip_status(moe::launch_combine(y, inv_perm, topk_w, T, k, H, out, (hipStream_t)stream),
                    "combine");
}

moe_status moe_miss_list(const int32_t* slot_map, int32_t E, const int32_t* offsets,
                         const int32_t* perm, int32_t T, int32_t k, int32_t* miss_pos,
                         int32_t* miss_of_pair, int32_t* counters, void* stream) {
  moe_status s = check_shape(T, 32, E, k);
  if (s != MOE_OK) return s;
  CHECK_PTR(slot_map);
  CHECK_PTR(offsets);
  CHECK_PTR(counters);
  if (T > 0) {
    CHECK_PTR(perm);
    CHECK_PTR(miss_pos);
    CHECK_PTR(miss_of_pair);
  }
  clear_stale_error();
  return hip_status(moe::launch_miss_list(slot_map, E, offsets, perm, T * k, miss_pos,
                                          miss_of_pair, counters, (hipStream_t)stream),
                    "miss list");
}

moe_status moe_merge_misses(float* out, const float* y_miss, const int32_t* miss_of_pair,
                            const float* topk_w, int32_t T, int32_t k, int32_t H,
                            void* stream) {
  moe_status s = check_shape(T, H, moe::kMaxE, k);
  if (s != MOE_OK) return s;
  if (T == 0) return ok();
  CHECK_PTR(out);
  CHECK_PTR(y_miss);
  CHECK_PTR(miss_of_pair);
  CHECK_PTR(topk_w);
  clear_stale_error();
  return hip_status(moe::launch_merge_misses(out, y_miss, miss_of_pair, topk_w, T, k, H,
                                             (hipStream_t)stream),
                    "merge misses");
}

moe_status moe_stage_plan(const int32_t* counts, const int32_t* slot_map, int32_t E,
                          int32_t first_slot, int32_t n_stage, int32_t* slot_map_out,
                          int32_t* copy_list, int32_t* counters, void* stream) {
  if (E < 1 || E > moe::kMaxE) return fail(MOE_ERR_INVALID_ARG, "E = %d outside [1, %d]", E, moe::kMaxE);
  if (first_slot < 0 || n_stage < 0)
    return fail(MOE_ERR_INVALID_ARG, "first_slot = %d, n_stage = %d", first_slot, n_stage);
  if ((int64_t)first_slot + n_stage > 0x7fffffff) return fail(MOE_ERR_INVALID_ARG, "window too large");
  CHECK_PTR(counts);
  CHECK_PTR(slot_map);
  CHECK_PTR(slot_map_out);
  CHECK_PTR(copy_list);
  CHECK_PTR(counters);
  clear_stale_error();
  return hip_status(moe::launch_stage_plan(counts, slot_map, E, first_slot, n_stage,
                                           slot_map_out, copy_list, counters,
                                           (hipStream_t)stream),
                    "stage plan");
}

moe_status moe_stage_copy(const moe_pool* pool, const moe_pool* backing,
                          const int32_t* copy_list, const int32_t* counters, int32_t first_slot,
                          int32_t max_copies, uint32_t* err_flags, void* stream) {
  moe_status s = check_pool(pool);
  if (s != MOE_OK) return s;
  s = check_pool(backing);
  if (s != MOE_OK) return s;
  if (backing->fmt != pool->fmt || backing->H != pool->H || backing->I != pool->I)
    return fail(MOE_ERR_INVALID_ARG, "backing store and pool differ in format or shape");
  if (first_slot < 0 || max_copies < 0 || (int64_t)first_slot + max_copies > pool->n_slots)
    return fail(MOE_ERR_INVALID_ARG, "window [%d, %d + %d) outside the pool's %d slots",
                first_slot, first_slot, max_copies, pool->n_slots);
  if (max_copies > moe::kMaxE)
    return fail(MOE_ERR_INVALID_ARG, "max_copies = %d > %d", max_copies, moe::kMaxE);
  if (max_copies == 0) return ok();
  CHECK_PTR(copy_list);
  CHECK_PTR(counters);
  const int fmt = pool->fmt, H = pool->H, I = pool->I;
  moe::StagePlanes pl;
  const void* src[6] = {backing->gate_q, backing->gate_s, backing->up_q,
                        backing->up_s,   backing->down_q, backing->down_s};
  const void* dst[6] = {pool->gate_q, pool->gate_s, pool->up_q,
                        pool->up_s,   pool->down_q, pool->down_s};
  for (int p = 0; p < moe::kStagePlanes; ++p) {
    const bool down = p >= 4, scales = p % 2 == 1;
    pl.src[p] = (const uint8_t*)src[p];
    pl.dst[p] = (uint8_t*)const_cast<void*>(dst[p]);
    pl.bytes[p] = (int64_t)plane_bytes(fmt, down ? H : I, down ? I : H, scales);
  }
  clear_stale_error();
  return hip_status(moe::launch_stage_copy(pl, copy_list, counters, first_slot, max_copies,
                                           backing->n_slots, err_flags, (hipStream_t)stream),
                    "stage copy");
}

moe_status moe_layer_workspace(int32_t T, int32_t H, int32_t I, int32_t E, int32_t k,
                               moe_ws_layout* out) {
  if (out == nullptr) return fail(MOE_ERR_INVALID_ARG, "out is NULL");
  moe_status s = check_shape(T, H, E, k);
  if (s != MOE_OK) return s;
  if (I <= 0 || I % 32) return fail(MOE_ERR_INVALID_ARG, "I = %d", I);
  s = check_extent(T, k, H, I);
  if (s != MOE_OK) return s;
  const size_t n = (size_t)T * k;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align256(off + bytes);
    return at;
  };
  out->topk_ids = take(n * 4);
  out->topk_w = take(n * 4);
  out->counts = take((size_t)E * 4);
  out->offsets = take((size_t)(E + 1) * 4);
  out->perm = take(n * 4);
  out->inv_perm = take(n * 4);
  out->h = take(n * I * 2);
  out->y = take(n * H * 4);
  const size_t rs = T > 0 ? route_scratch(T, H, E) : 0;
  const size_t bs = T > 0 ? moe::bucket_scratch_bytes((int)n, E) : 0;
  out->scratch = take(rs > bs ? rs : bs);
  out->act = take((size_t)moe::act_ints(E) * sizeof(int32_t));
  out->sync = take((size_t)moe::sync_ints(H) * sizeof(int32_t));
  out->total = off;
  return ok();
}

// Down projection and combine of the fused layer. With the small-batch active-expert list
// (act != NULL) and few pairs, one kernel does both.
static moe_status down_combine_tail(const moe_pool* pool, const int32_t* slot_map, int32_t E,
                                    int32_t T, int32_t k, const int32_t* offsets,
                                    const int32_t* act, const uint16_t* h,
                                    const int32_t* inv_perm, const float* w, float* y,
                                    float* out, uint32_t* err_flags, int32_t path,
                                    hipStream_t st, int32_t* tickets = nullptr) {
  const bool small = moe::down_small_preferred(pool->fmt, T, k, E, pool->I);
  if (act != nullptr && tickets != nullptr && use_gemv(path, T) && !small &&
      moe::down_ticket_ok(T, k, E)) {
    // decode: the tickets were zeroed by the routed gate/up kernel
    clear_stale_error();
    moe::PoolView g, u, d;
    pool_views(pool, &g, &u, &d);
    return hip_status(moe::launch_down_ticket(pool->fmt, d, pool->n_slots, E, T, k, pool->H,
                                              pool->I, act, h, inv_perm, w, y, out, tickets,
                                              err_flags, st),
                      "down+combine (tickets)");
  }
  if (act != nullptr && use_gemv(path, T) && small) {
    clear_stale_error();
    moe::PoolView g, u, d;
    pool_views(pool, &g, &u, &d);
    return hip_status(moe::launch_down_combine_small(pool->fmt, d, pool->n_slots, E, T, k, pool->H,
                                                     pool->I, act, h, inv_perm, w, y, out,
                                                     err_flags, st),
                      "down+combine");
  }
  moe_status s = down_dispatch(pool, slot_map, E, T, k, offsets, h, y, err_flags, path, st);
  if (s != MOE_OK) return s;
  clear_stale_error();
  return hip_status(moe::launch_combine(y, inv_perm, w, T, k, pool->H, out, st), "combine");
}

// Record a timing event; inside a stream capture it becomes an event-record node of the
// graph (so replays can still be timed).
static moe_status record_event(hipEvent_t ev, hipStream_t st) {
  hipStreamCaptureStatus cs = hipStreamCaptureStatusNone;
  hipError_t e = hipStreamIsCapturing(st, &cs);
  if (e != hipSuccess) return hip_status(e, "event record: stream capture query");
  if (cs == hipStreamCaptureStatusActive)
    return hip_status(hipEventRecordWithFlags(ev, st, hipEventRecordExternal),
                      "event record (external, in capture)");
  return hip_status(hipEventRecord(ev, st), "event record");
}

static moe_status layer_impl(const moe_pool* pool, const int32_t* slot_map,
                             const uint16_t* w_router, const float* bias, const uint16_t* x,
                             int32_t T, int32_t E, int32_t k, float* out, void* workspace,
                             size_t workspace_bytes, uint32_t* err_flags, int32_t path,
                             void* stream, void* ev_begin, void* ev_end) {
  moe_status s = check_pool(pool);
  if (s != MOE_OK) return s;
  s = check_shape(T, pool->H, E, k);
  if (s != MOE_OK) return s;
  s = check_extent(T, k, pool->H, pool->I);
  if (s != MOE_OK) return s;
  if (path < MOE_PATH_AUTO || path > MOE_PATH_PERSISTENT)
    return fail(MOE_ERR_INVALID_ARG, "path = %d", path);
  if (T == 0) return ok();
  CHECK_PTR(slot_map);
  CHECK_PTR(w_router);
  CHECK_PTR(x);
  CHECK_PTR(out);
  if (bias != nullptr && ((uintptr_t)bias & 3)) return fail(MOE_ERR_INVALID_ARG, "bias misaligned");
  if (workspace == nullptr || ((uintptr_t)workspace & 255))
    return fail(MOE_ERR_INVALID_ARG, "workspace is NULL or not 256-byte aligned");
  if (err_flags != nullptr && ((uintptr_t)err_flags & 3))
    return fail(MOE_ERR_INVALID_ARG, "err_flags misaligned");
  moe_ws_layout L;
  s = moe_layer_workspace(T, pool->H, pool->I, E, k, &L);
  if (s != MOE_OK) return s;
  if (workspace_bytes < L.total)
    return fail(MOE_ERR_INVALID_ARG, "workspace %zu bytes < %zu needed", workspace_bytes, L.total);
  char* ws = (char*)workspace;
  int32_t* ids = (int32_t*)(ws + L.topk_ids);
  float* w = (float*)(ws + L.topk_w);
  int32_t* counts = (int32_t*)(ws + L.counts);
  int32_t* offsets = (int32_t*)(ws + L.offsets);
  int32_t* perm = (int32_t*)(ws + L.perm);
  int32_t* inv_perm = (int32_t*)(ws + L.inv_perm);
  uint16_t* h = (uint16_t*)(ws + L.h);
  float* y = (float*)(ws + L.y);
  void* scratch = ws + L.scratch;
  int32_t* act = (int32_t*)(ws + L.act);
  int32_t* sync = (int32_t*)(ws + L.sync);   // tickets first, then the hand-off counters
  hipStream_t st = (hipStream_t)stream;
  hipError_t e;
  bool have_act = false;
  clear_stale_error();
  // route + bucket: for small batches the split router is finished (top-k and counting
  // sort) by one single-workgroup kernel; otherwise router, then the counting sort
  const bool gemv = use_gemv(path, T);
  if (moe::route_fused_ok(T, pool->H, E)) {
    // router partials over slices of H; the gate/up GEMV finishes the routing itself (or,
    // for the grouped path, one workgroup finishes it and bucket-sorts)
    const int ns = moe::route_fused_split(pool->H);
    const bool fused = path == MOE_PATH_PERSISTENT && moe::decode_fused_ok(T, pool->H, E);
    e = moe::launch_router_partials(x, w_router, T, pool->H, E, ns, (float*)scratch, st,
                                    fused ? sync : nullptr, moe::sync_ints(pool->H));
    if (e != hipSuccess) return hip_status(e, "router");
    if (fused) {
      // one persistent kernel: routing, gate/up + SwiGLU, down and combine
      if (ev_begin != nullptr) {
        s = record_event((hipEvent_t)ev_begin, st);
        if (s != MOE_OK) return s;
      }
      moe::PoolView g, u, d;
      pool_views(pool, &g, &u, &d);
      const moe::RouteIn rin{(const float*)scratch, ns, bias, T, ids, w, counts, offsets, perm,
                             inv_perm, act, nullptr, 0};
      clear_stale_error();
      e = moe::launch_decode_fused(pool->fmt, g, u, d, slot_map, pool->n_slots, E, x, T, k,
                                   pool->H, pool->I, rin, h, y, out, sync, err_flags, st);
      if (e != hipSuccess) return hip_status(e, "fused decode layer");
      if (ev_end != nullptr) return record_event((hipEvent_t)ev_end, st);
      return ok();
    }
    if (gemv) {
      if (ev_begin != nullptr) {
        s = record_event((hipEvent_t)ev_begin, st);
        if (s != MOE_OK) return s;
      }
      moe::PoolView g, u, d;
      pool_views(pool, &g, &u, &d);
      const moe::RouteIn rin{(const float*)scratch, ns, bias, T, ids, w, counts, offsets, perm,
                             inv_perm, act, sync, pool->H / 16};
      clear_stale_error();
      e = moe::launch_gate_up_route(pool->fmt, g, u, slot_map, pool->n_slots, E, x, T, k,
                                    pool->H, pool->I, rin, h, err_flags, st);
      if (e != hipSuccess) return hip_status(e, "route + gate/up (GEMV)");
      if (ev_end != nullptr) {
        s = record_event((hipEvent_t)ev_end, st);
        if (s != MOE_OK) return s;
      }
      return down_combine_tail(pool, slot_map, E, T, k, offsets, act, h, inv_perm, w, y, out,
                               err_flags, path, st, sync);
    }
    e = moe::launch_router_finish((const float*)scratch, ns, bias, T, E, k, ids, w, counts,
                                  offsets, perm, inv_perm, st);
    if (e != hipSuccess) return hip_status(e, "route+bucket");
  } else if (moe::route_small_ok(T, E)) {
    // one workgroup: router, top-k, counting sort and the active-expert list
    e = moe::launch_route_small(x, w_router, bias, T, pool->H, E, k, slot_map, ids, w, counts,
                                offsets, perm, inv_perm, act, st);
    if (e != hipSuccess) return hip_status(e, "route+bucket");
    have_act = true;
  } else if (moe::route_bucket_fusable(T, E)) {
    e = moe::launch_route_bucket_small(x, w_router, bias, T, pool->H, E, k, (float*)scratch, ids,
                                       w, counts, offsets, perm, inv_perm, st);
    if (e != hipSuccess) return hip_status(e, "route+bucket");
  } else {
    e = moe::launch_route(x, w_router, bias, T, pool->H, E, k, ids, w, (float*)scratch, st);
    if (e != hipSuccess) return hip_status(e, "route");
    e = moe::launch_bucket(ids, T * k, E, counts, offsets, perm, inv_perm, scratch, st);
    if (e != hipSuccess) return hip_status(e, "bucket");
  }
  if (ev_begin != nullptr) {
    s = record_event((hipEvent_t)ev_begin, st);
    if (s != MOE_OK) return s;
  }
  s = gate_up_dispatch(pool, slot_map, E, x, T, k, offsets, perm, h, err_flags, path, st,
                       have_act ? act : nullptr);
  if (s != MOE_OK) return s;
  if (ev_end != nullptr) {
    s = record_event((hipEvent_t)ev_end, st);
    if (s != MOE_OK) return s;
  }
  return down_combine_tail(pool, slot_map, E, T, k, offsets, have_act ? act : nullptr, h,
                           inv_perm, w, y, out, err_flags, path, st);
}

moe_status moe_layer(const moe_pool* pool, const int32_t* slot_map, const uint16_t* w_router,
                     const float* bias, const uint16_t* x, int32_t T, int32_t E, int32_t k,
                     float* out, void* workspace, size_t workspace_bytes, uint32_t* err_flags,
                     int32_t path, void* stream) {
  return layer_impl(pool, slot_map, w_router, bias, x, T, E, k, out, workspace, workspace_bytes,
                    err_flags, path, stream, nullptr, nullptr);
}

moe_status moe_layer_noalloc(const moe_pool* pool, const int32_t* slot_map,
                             const uint16_t* w_router, const float* bias, const uint16_t* x,
                             int32_t T, int32_t E, int32_t k, float* out, uint32_t* err_flags,
                             int32_t path, void* stream) {
  moe_status s = check_pool(pool);
  if (s != MOE_OK) return s;
  s = check_shape(T, pool->H, E, k);
  if (s != MOE_OK) return s;
  if (T == 0) return ok();
  moe_ws_layout L;
  s = moe_layer_workspace(T, pool->H, pool->I, E, k, &L);
  if (s != MOE_OK) return s;
  if (L.total > (size_t)MOE_NOALLOC_WS_BYTES)
    return fail(MOE_ERR_INVALID_ARG,
                "moe_layer_noalloc: the layer needs %zu bytes of workspace, more than the "
                "%zu-byte static workspace (T = %d; use moe_layer with a caller workspace)",
                L.total, (size_t)MOE_NOALLOC_WS_BYTES, T);
  void* ws = nullptr;
  s = noalloc_workspace((hipStream_t)stream, &ws);
  if (s != MOE_OK) return s;
  return layer_impl(pool, slot_map, w_router, bias, x, T, E, k, out, ws, MOE_NOALLOC_WS_BYTES,
                    err_flags, path, stream, nullptr, nullptr);
}

moe_status moe_layer_timed(const moe_pool* pool, const int32_t* slot_map,
                           const uint16_t* w_router, const float* bias, const uint16_t* x,
                           int32_t T, int32_t E, int32_t k, float* out, void* workspace,
                           size_t workspace_bytes, uint32_t* err_flags, int32_t path,
                           void* stream, void* ev_gate_up_begin, void* ev_gate_up_end) {
  return layer_impl(pool, slot_map, w_router, bias, x, T, E, k, out, workspace, workspace_bytes,
                    err_flags, path, stream, ev_gate_up_begin, ev_gate_up_end);
}

// ---- microscaled formats and the block's two ends

namespace {

moe_status check_mx(int32_t fmt, int32_t K) {
  if (fmt != MOE_MX_FP4 && fmt != MOE_MX_FP6)
    return fail(MOE_ERR_UNSUPPORTED, "unknown microscaled format %d", fmt);
  if (K <= 0 || K % 32) return fail(MOE_ERR_INVALID_ARG, "K = %d is not a positive multiple of 32", K);
  return MOE_OK;
}

moe_status check_type(const char* what, int32_t type, bool fp16) {
  if (type == MOE_T_BF16 || type == MOE_T_FP32 || (fp16 && type == MOE_T_FP16)) return MOE_OK;
  return fail(MOE_ERR_UNSUPPORTED, "%s type %d", what, type);
}

// rows x K values, one thread per 8 of them
moe_status check_mx_rows(int32_t rows, int32_t K) {
  if (rows < 0) return fail(MOE_ERR_INVALID_ARG, "rows = %d < 0", rows);
  if ((int64_t)rows * K >= (int64_t(1) << 40))
    return fail(MOE_ERR_INVALID_ARG, "rows*K = %lld values, limit 2^40", (long long)rows * K);
  return MOE_OK;
}

// Sizes and parameters that both norms share; H as everywhere a multiple of 32.
moe_status check_norm(int32_t T, int32_t H, int32_t k, int32_t resid_type, int32_t weight_type,
                      float eps) {
  moe_status s = check_shape(T, H, moe::kMaxE, k);
  if (s != MOE_OK) return s;
  if (!(eps >= 0.f && eps <= FLT_MAX))
    return fail(MOE_ERR_INVALID_ARG, "eps = %g is negative or not finite", (double)eps);
  s = check_type("resid", resid_type, false);
  if (s != MOE_OK) return s;
  return check_type("weight", weight_type, false);
}

// Arguments of the products on microscaled rows.
moe_status check_mx_product(const moe_pool* pool, const int32_t* slot_map, int32_t E, int32_t fmt,
                            int32_t T, int32_t k, const int32_t* offsets, uint32_t* err_flags,
                            int32_t path) {
  moe_status s = check_ffn_args(pool, slot_map, E, T, k, offsets, err_flags, path);
  if (s != MOE_OK) return s;
  if (pool->fmt != MOE_W_MXFP4)
    return fail(MOE_ERR_UNSUPPORTED, "products on microscaled rows need an MXFP4 pool, not format %d",
                pool->fmt);
  // the kernels step through a row group's units in 32 bits: 256 bytes a block, two groups
  if (pool->H >= 1 << 27 || pool->I >= 1 << 27)
    return fail(MOE_ERR_INVALID_ARG, "H = %d, I = %d, limit 2^27", pool->H, pool->I);
  return check_mx(fmt, pool->H);
}

// AUTO for the products on microscaled rows: the few-token kernel for up to 16 tokens (one
// column tile an expert) and where experts have at most 4 rows on average. Measured,
// us of it against the 32-row tiles, uniform load and one where the r-th expert is wanted r^-1.2
// times as often: H = I = 2880, 32 experts, MXFP6, gate/up, mean 2: 48 against 58, 28 against 35;
// mean 4: 52 against 61, 41 against 43; mean 8: 59 against 62, 54 against 50; H 2048, I 768, 128
// experts, MXFP4, gate/up, mean 4: 41 against 48, 23 against 23; mean 8: 44 against 48, 39 against
// 21. Down gains less: mean 2: 30 against 30, 14 against 23; mean 4: 34 against 32, 23 against
// 27; the 128 experts, mean 4: 30 against 21, 16 against 12.
bool use_mx_gemv(int32_t path, int32_t T, int32_t k, int32_t E) {
  return use_gemv(path, T) || (path == MOE_PATH_AUTO && (int64_t)T * k <= 4 * E);
}

moe_status mx_gate_up(const moe_pool* pool, const int32_t* slot_map, int32_t E, const void* x_q,
                      const uint8_t* x_s, int32_t x_fmt, int32_t T, int32_t k,
                      const int32_t* offsets, const int32_t* perm, uint16_t* h, uint32_t* err,
                      int32_t path, hipStream_t st) {
  moe::PoolView g, u, d;
  pool_views(pool, &g, &u, &d);
  const moe::MxProduct p{g, u, slot_map, pool->n_slots, E, T, k, offsets, perm,
                         (const uint8_t*)x_q, x_s, pool->H, pool->I, h, nullptr, err};
  clear_stale_error();
  return hip_status(moe::launch_mx_product(p, x_fmt, true, use_mx_gemv(path, T, k, E), st),
                    "microscaled gate/up");
}

moe_status mx_down(const moe_pool* pool, const int32_t* slot_map, int32_t E, const void* h_q,
                   const uint8_t* h_s, int32_t h_fmt, int32_t T, int32_t k,
                   const int32_t* offsets, float* y, uint32_t* err, int32_t path,
                   hipStream_t st) {
  moe::PoolView g, u, d;
  pool_views(pool, &g, &u, &d);
  const moe::MxProduct p{d, d, slot_map, pool->n_slots, E, T, k, offsets, nullptr,
                         (const uint8_t*)h_q, h_s, pool->I, pool->H, nullptr, y, err};
  clear_stale_error();
  return hip_status(moe::launch_mx_product(p, h_fmt, false, use_mx_gemv(path, T, k, E), st),
                    "microscaled down");
}

}  // namespace

size_t moe_mx_row_bytes(int32_t fmt, int32_t K) {
  if ((fmt != MOE_MX_FP4 && fmt != MOE_MX_FP6) || K < 0 || K % 32) return 0;
  return (size_t)(K / 32) * moe::mx_block_bytes(fmt);
}

moe_status moe_mx_quantize(const void* src, int32_t src_type, int32_t rows, int32_t K,
                           int32_t fmt, void* q, uint8_t* s, void* stream) {
  moe_status st = check_mx(fmt, K);
  if (st != MOE_OK) return st;
  st = check_type("src", src_type, true);
  if (st != MOE_OK) return st;
  st = check_mx_rows(rows, K);
  if (st != MOE_OK) return st;
  if (rows == 0) return ok();
  CHECK_PTR(src);
  CHECK_PTR(q);
  if (s == nullptr) return fail(MOE_ERR_INVALID_ARG, "s is NULL");
  clear_stale_error();
  return hip_status(moe::launch_mx_quantize(src, src_type, (int64_t)rows * K, fmt, (uint8_t*)q, s,
                                            (hipStream_t)stream),
                    "microscaled quantise");
}

moe_status moe_mx_dequantize(const void* q, const uint8_t* s, int32_t fmt, int32_t rows,
                             int32_t K, void* dst, int32_t dst_type, void* stream) {
  moe_status st = check_mx(fmt, K);
  if (st != MOE_OK) return st;
  st = check_type("dst", dst_type, true);
  if (st != MOE_OK) return st;
  st = check_mx_rows(rows, K);
  if (st != MOE_OK) return st;
  if (rows == 0) return ok();
  CHECK_PTR(q);
  CHECK_PTR(dst);
  if (s == nullptr) return fail(MOE_ERR_INVALID_ARG, "s is NULL");
  clear_stale_error();
  return hip_status(moe::launch_mx_dequantize((const uint8_t*)q, s, (int64_t)rows * K, fmt, dst,
                                              dst_type, (hipStream_t)stream),
                    "microscaled dequantise");
}

moe_status moe_mx_expert_gate_up(const moe_pool* pool, const int32_t* slot_map, int32_t E,
                                 const void* x_q, const uint8_t* x_s, int32_t x_fmt, int32_t T,
                                 int32_t k, const int32_t* offsets, const int32_t* perm,
                                 uint16_t* h, uint32_t* err_flags, int32_t path, void* stream) {
  moe_status s = check_mx_product(pool, slot_map, E, x_fmt, T, k, offsets, err_flags, path);
  if (s != MOE_OK || T == 0) return s == MOE_OK ? ok() : s;
  CHECK_PTR(x_q);
  CHECK_PTR(perm);
  CHECK_PTR(h);
  if (x_s == nullptr) return fail(MOE_ERR_INVALID_ARG, "x_s is NULL");
  return mx_gate_up(pool, slot_map, E, x_q, x_s, x_fmt, T, k, offsets, perm, h, err_flags, path,
                    (hipStream_t)stream);
}

moe_status moe_mx_expert_down(const moe_pool* pool, const int32_t* slot_map, int32_t E,
                              const void* h_q, const uint8_t* h_s, int32_t h_fmt, int32_t T,
                              int32_t k, const int32_t* offsets, float* y, uint32_t* err_flags,
                              int32_t path, void* stream) {
  moe_status s = check_mx_product(pool, slot_map, E, h_fmt, T, k, offsets, err_flags, path);
  if (s != MOE_OK || T == 0) return s == MOE_OK ? ok() : s;
  CHECK_PTR(h_q);
  CHECK_PTR(y);
  if (h_s == nullptr) return fail(MOE_ERR_INVALID_ARG, "h_s is NULL");
  return mx_down(pool, slot_map, E, h_q, h_s, h_fmt, T, k, offsets, y, err_flags, path,
                 (hipStream_t)stream);
}

moe_status moe_mx_expert_ffn(const moe_pool* pool, const int32_t* slot_map, int32_t E,
                             const void* x_q, const uint8_t* x_s, int32_t x_fmt, int32_t T,
                             int32_t k, const int32_t* offsets, const int32_t* perm, uint16_t* h,
                             void* h_q, uint8_t* h_s, int32_t h_fmt, float* y,
                             uint32_t* err_flags, int32_t path, void* stream) {
  moe_status s = check_mx_product(pool, slot_map, E, x_fmt, T, k, offsets, err_flags, path);
  if (s != MOE_OK) return s;
  s = check_mx(h_fmt, pool->I);
  if (s != MOE_OK) return s;
  s = check_mx_rows(T * k, pool->I);
  if (s != MOE_OK) return s;
  if (T == 0) return ok();
  CHECK_PTR(x_q);
  CHECK_PTR(perm);
  CHECK_PTR(h);
  CHECK_PTR(h_q);
  CHECK_PTR(y);
  if (x_s == nullptr || h_s == nullptr)
    return fail(MOE_ERR_INVALID_ARG, "%s is NULL", x_s == nullptr ? "x_s" : "h_s");
  const hipStream_t st = (hipStream_t)stream;
  s = mx_gate_up(pool, slot_map, E, x_q, x_s, x_fmt, T, k, offsets, perm, h, err_flags, path, st);
  if (s != MOE_OK) return s;
  s = hip_status(moe::launch_mx_quantize(h, MOE_T_BF16, (int64_t)T * k * pool->I, h_fmt,
                                         (uint8_t*)h_q, h_s, st),
                 "microscaled quantise");
  if (s != MOE_OK) return s;
  return mx_down(pool, slot_map, E, h_q, h_s, h_fmt, T, k, offsets, y, err_flags, path, st);
}

moe_status moe_add_norm(const void* resid, int32_t resid_type, const void* delta,
                        int32_t delta_type, float scale, const void* weight, int32_t weight_type,
                        float eps, int32_t T, int32_t H, void* resid_out, uint16_t* x,
                        void* stream) {
  moe_status s = check_norm(T, H, 1, resid_type, weight_type, eps);
  if (s != MOE_OK) return s;
  if (delta != nullptr && (s = check_type("delta", delta_type, false)) != MOE_OK) return s;
  if (T == 0) return ok();
  CHECK_PTR(resid);
  if (delta != nullptr) {
    CHECK_PTR(delta);
    CHECK_PTR(resid_out);
  } else if (resid_out != nullptr) {
    CHECK_PTR(resid_out);
  }
  CHECK_PTR(weight);
  CHECK_PTR(x);
  moe::BlockNorm a{};
  a.T = T, a.H = H, a.k = 1;
  a.resid = resid, a.delta = delta, a.weight = weight;
  a.eps = eps;
  a.scale = delta != nullptr ? scale : -0.f;   // -0 * 0 + resid is resid, bit by bit
  a.resid_out = resid_out, a.x = x;
  a.delta_f32 = delta_type == MOE_T_FP32, a.par_f32 = weight_type == MOE_T_FP32;
  clear_stale_error();
  return hip_status(moe::launch_block_norm(a, false, resid_type == MOE_T_FP32, (hipStream_t)stream),
                    "add + norm");
}

moe_status moe_combine_norm(const float* y, const int32_t* inv_perm, const float* topk_w,
                            int32_t T, int32_t k, int32_t H, const void* resid,
                            int32_t resid_type, const void* post_weight, const void* gate,
                            int32_t gate_rows, float scale, const void* next_weight,
                            int32_t weight_type, float eps, void* resid_out, uint16_t* x,
                            void* stream) {
  moe_status s = check_norm(T, H, k, resid_type, weight_type, eps);
  if (s != MOE_OK) return s;
  if (gate != nullptr && gate_rows != 1 && gate_rows != T)
    return fail(MOE_ERR_INVALID_ARG, "gate_rows = %d, neither 1 nor T = %d", gate_rows, T);
  if (T == 0) return ok();
  if ((next_weight == nullptr) != (x == nullptr))
    return fail(MOE_ERR_INVALID_ARG, "next_weight and x go together: one of them is NULL");
  CHECK_PTR(y);
  CHECK_PTR(inv_perm);
  CHECK_PTR(topk_w);
  CHECK_PTR(resid);
  CHECK_PTR(resid_out);
  if (post_weight != nullptr) CHECK_PTR(post_weight);
  if (gate != nullptr) CHECK_PTR(gate);
  if (x != nullptr) {
    CHECK_PTR(next_weight);
    CHECK_PTR(x);
  }
  moe::BlockNorm a{};
  a.T = T, a.H = H, a.k = k;
  a.resid = resid, a.y = y, a.inv_perm = inv_perm, a.w = topk_w;
  a.post = post_weight, a.gate = gate, a.gate_stride = gate_rows == 1 ? 0 : H;
  a.weight = next_weight;
  a.eps = eps, a.scale = scale;
  a.resid_out = resid_out, a.x = x;
  a.par_f32 = weight_type == MOE_T_FP32;
  clear_stale_error();
  return hip_status(moe::launch_block_norm(a, true, resid_type == MOE_T_FP32, (hipStream_t)stream),
                    "combine + norm");
}

namespace {

// The rows of the attention half of a block.
moe_status check_heads(const char* name, const moe_heads* h, int align, int64_t stride) {
  if (h == nullptr || h->p == nullptr) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", name);
  if ((uintptr_t)h->p & (align - 1))
    return fail(MOE_ERR_INVALID_ARG, "%s is not %d-byte aligned", name, align);
  if (h->token < 0 || h->head < 0 || h->token % stride || h->head % stride)
    return fail(MOE_ERR_INVALID_ARG, "%s strides (%lld, %lld): not negative, multiples of %lld", name,
                (long long)h->token, (long long)h->head, (long long)stride);
  if (h->token >= (int64_t(1) << 32) || h->head >= (int64_t(1) << 32))
    return fail(MOE_ERR_INVALID_ARG, "%s strides: limit 2^32", name);
  return MOE_OK;
}
moe::HeadsView heads_view(const moe_heads* h) { return {(uint8_t*)h->p, h->token, h->head}; }
bool same_heads(const moe_heads* a, const moe_heads* b) {
  return a->p != b->p || (a->token == b->token && a->head == b->head);
}

// Rows that are written must not meet: those of (t, h) and (t', h') start at least D elements apart.
moe_status check_apart(const char* name, const moe_heads* h, int64_t T, int64_t n, int64_t D) {
  bool apart = (T <= 1 || h->token >= D) && (n <= 1 || h->head >= D);
  if (apart && T > 1 && n > 1 && h->token < (n - 1) * h->head + D && h->head < (T - 1) * h->token + D) {
    // heads between tokens and tokens between heads: the differences of one kind, next to those of the other
    const int64_t few = T < n ? T : n, many = T < n ? n : T;
    const int64_t step = T < n ? h->token : h->head, other = T < n ? h->head : h->token;
    for (int64_t i = 1; apart && i < few; ++i) {
      const int64_t at = i * step, j = at / other;
      apart = (j >= many || at - j * other >= D) && (j + 1 >= many || (j + 1) * other - at >= D);
    }
  }
  if (apart) return MOE_OK;
  return fail(MOE_ERR_INVALID_ARG, "%s strides (%lld, %lld): rows of %lld values overlap", name,
              (long long)h->token, (long long)h->head, (long long)D);
}

int type_bytes(int32_t type) { return type == MOE_T_FP32 ? 4 : type == MOE_T_E4M3 ? 1 : 2; }

moe_status check_rope(const moe_rope_plan* plan, int32_t D) {
  if (plan == nullptr) return fail(MOE_ERR_INVALID_ARG, "plan is NULL");
  if (plan->layout != MOE_ROPE_HALF && plan->layout != MOE_ROPE_INTERLEAVED)
    return fail(MOE_ERR_UNSUPPORTED, "unknown rope layout %d", plan->layout);
  if (plan->dim < 2 || plan->dim % 2 || plan->dim > D)
    return fail(MOE_ERR_INVALID_ARG, "rope dim = %d: even, in [2, D = %d]", plan->dim, D);
  if (plan->freq == nullptr || ((uintptr_t)plan->freq & 7))
    return fail(MOE_ERR_INVALID_ARG, "rope freq is %s",
                plan->freq ? "not 8-byte aligned" : "NULL");
  return MOE_OK;
}
moe::RopeView rope_view(const moe_rope_plan* p) {
  if (p == nullptr) return {nullptr, 0, false, 1.f};
  return {p->freq, p->dim, p->layout == MOE_ROPE_INTERLEAVED, p->scale};
}

moe_status check_cache(const moe_kv_cache* c) {
  if (c == nullptr) return fail(MOE_ERR_INVALID_ARG, "cache is NULL");
  if (c->type != MOE_T_BF16 && c->type != MOE_T_FP16 && c->type != MOE_T_E4M3)
    return fail(MOE_ERR_UNSUPPORTED, "unknown cache type %d", c->type);
  if (c->n_pages < 1 || c->page_size < 1 || c->n_heads < 1)
    return fail(MOE_ERR_INVALID_ARG, "cache of %d pages, %d tokens a page, %d heads", c->n_pages,
                c->page_size, c->n_heads);
  if (c->D < 16 || c->D > 256 || c->D % 16)
    return fail(MOE_ERR_INVALID_ARG, "cache D = %d: a multiple of 16, at most 256", c->D);
  CHECK_PTR(c->k);
  CHECK_PTR(c->v);
  const int64_t mult = 16 / type_bytes(c->type);
  for (const int64_t st : {c->k_page, c->k_token, c->k_head, c->v_page, c->v_token, c->v_head})
    if (st < 0 || st % mult || st >= (int64_t(1) << 32))
      return fail(MOE_ERR_INVALID_ARG, "cache stride %lld: not negative, a multiple of %lld, below 2^32",
                  (long long)st, (long long)mult);
  if ((c->k_scale != nullptr || c->v_scale != nullptr) && c->type != MOE_T_E4M3)
    return fail(MOE_ERR_INVALID_ARG, "scales go with an E4M3 cache");
  if (((uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 3)
    return fail(MOE_ERR_INVALID_ARG, "cache scales misaligned");
  return MOE_OK;
}
moe::KvCacheView cache_view(const moe_kv_cache* c) {
  return {(uint8_t*)c->k, (uint8_t*)c->v, c->k_page, c->k_token, c->k_head, c->v_page, c->v_token,
          c->v_head, c->k_scale, c->v_scale, c->type, c->n_pages, c->page_size, c->n_heads, c->D,
          0xFFFFFFFFu / (uint32_t)c->page_size};
}

// The sizes of a batch. Its pointers are checked where there are rows (check_batch_ptrs).
moe_status check_batch(const moe_kv_batch* b, const moe_kv_cache* c, int64_t n_q_heads) {
  if (b == nullptr) return fail(MOE_ERR_INVALID_ARG, "batch is NULL");
  if (b->n_seq < 0 || b->n_seq >= (1 << 24))
    return fail(MOE_ERR_INVALID_ARG, "n_seq = %d outside [0, 2^24)", b->n_seq);
  if (b->T < 0) return fail(MOE_ERR_INVALID_ARG, "T = %d < 0", b->T);
  const int64_t heads = n_q_heads > c->n_heads ? n_q_heads : c->n_heads;
  // fewer than 2^24 heads, a workgroup of 256 threads each: a grid's dimension has below 2^32 threads
  if (heads * c->D >= (1 << 28) || heads * (b->T > 0 ? b->T : 1) > (1 << 30))
    return fail(MOE_ERR_INVALID_ARG, "%lld heads, D = %d, T = %d: heads * D < 2^28, T * heads <= 2^30",
                (long long)heads, c->D, b->T);
  if (b->max_pages < 1 || (int64_t)b->max_pages * c->page_size > 0x7FFFF000)
    return fail(MOE_ERR_INVALID_ARG, "page table of %d pages of %d tokens: 1 to 2^31 - 4096 tokens",
                b->max_pages, c->page_size);
  if (b->table_stride < 0 || b->table_stride >= (int64_t(1) << 32))
    return fail(MOE_ERR_INVALID_ARG, "table_stride = %lld", (long long)b->table_stride);
  if (b->max_q < 0 || b->max_len < 0)
    return fail(MOE_ERR_INVALID_ARG, "max_q = %d, max_len = %d", b->max_q, b->max_len);
  return MOE_OK;
}
moe_status check_batch_ptrs(const moe_kv_batch* b, const uint32_t* err_flags) {
  const struct { const char* name; const void* p; } all[] = {
      {"q_start", b->q_start}, {"seq_len", b->seq_len}, {"page_table", b->page_table}};
  for (const auto& a : all) {
    if (a.p == nullptr) return fail(MOE_ERR_INVALID_ARG, "%s is NULL", a.name);
    if ((uintptr_t)a.p & 3) return fail(MOE_ERR_INVALID_ARG, "%s misaligned", a.name);
  }
  if ((uintptr_t)err_flags & 3) return fail(MOE_ERR_INVALID_ARG, "err_flags misaligned");
  return MOE_OK;
}
moe::KvBatchView batch_view(const moe_kv_batch* b) {
  return {b->q_start, b->seq_len, b->page_table, b->table_stride, b->n_seq, b->T, b->max_pages};
}

moe_status check_attend(const moe_kv_cache* c, const moe_kv_batch* b, int32_t n_q_heads,
                        int32_t window, int32_t keep_first) {
  moe_status s = check_cache(c);
  if (s != MOE_OK) return s;
  if (n_q_heads < 1 || n_q_heads % c->n_heads)
    return fail(MOE_ERR_INVALID_ARG, "n_q_heads = %d is not a multiple of the cache's %d", n_q_heads,
                c->n_heads);
  s = check_batch(b, c, n_q_heads);
  if (s != MOE_OK) return s;
  if (window < 0 || keep_first < 0)
    return fail(MOE_ERR_INVALID_ARG, "window = %d, keep_first = %d", window, keep_first);
  return MOE_OK;
}
moe::AttendPlan plan_of(const moe_kv_cache* c, const moe_kv_batch* b, int32_t n_q_heads,
                        int32_t window, int32_t keep_first) {
  return moe::attend_plan(cache_view(c), batch_view(b), n_q_heads, window, keep_first, b->max_q,
                          b->max_len);
}
// Rows of splits whose sums meet in scratch memory, of the sequences with many rows and with few. A row
// has D sums and two statistics.
int64_t part_rows(const moe::AttendPlan& p) {
  return p.few || p.splits <= 1 ? 0 : p.splits * p.rows;
}
int64_t part_rows_few(const moe::AttendPlan& p) {
  return !(p.few || p.both) || p.splits_few <= 1 ? 0 : p.splits_few * p.rows_few;
}
size_t attend_scratch(const moe_kv_cache* c, const moe::AttendPlan& p) {
  return (size_t)(part_rows(p) + part_rows_few(p)) * (c->D + 2) * sizeof(float);
}

moe_status check_16bit(const char* name, int32_t type) {
  if (type == MOE_T_BF16 || type == MOE_T_FP16) return MOE_OK;
  return fail(MOE_ERR_UNSUPPORTED, "%s type %d", name, type);
}

}  // namespace

moe_status moe_rope(const moe_rope_plan* plan, const moe_heads* x, int32_t type, int32_t T,
                    int32_t n_heads, int32_t D, const int32_t* positions, int32_t inverse,
                    const moe_heads* out, void* stream) {
  moe_status s = check_type("x", type, true);
  if (s != MOE_OK) return s;
  if (T < 0 || n_heads < 1 || D < 2 || D > 1024 || (int64_t)n_heads * D > (1 << 28) ||
      (int64_t)T * n_heads > (1 << 30))
    return fail(MOE_ERR_INVALID_ARG,
                "T = %d, n_heads = %d, D = %d: D in [2, 1024], n_heads * D <= 2^28, T * n_heads <= 2^30",
                T, n_heads, D);
  if ((s = check_rope(plan, D)) != MOE_OK) return s;
  if (T == 0) return ok();
  if ((s = check_heads("x", x, type_bytes(type), 1)) != MOE_OK) return s;
  if ((s = check_heads("out", out, type_bytes(type), 1)) != MOE_OK) return s;
  if (!same_heads(x, out)) return fail(MOE_ERR_INVALID_ARG, "out is x with other strides");
  if ((s = check_apart("out", out, T, n_heads, D)) != MOE_OK) return s;
  if (positions == nullptr || ((uintptr_t)positions & 3))
    return fail(MOE_ERR_INVALID_ARG, "positions is %s", positions ? "misaligned" : "NULL");
  moe::RopeCall a{};
  a.rope = rope_view(plan);
  a.x = heads_view(x), a.out = heads_view(out);
  a.positions = positions;
  a.type = type, a.T = T, a.n_heads = n_heads, a.D = D, a.inverse = inverse != 0;
  clear_stale_error();
  return hip_status(moe::launch_rope(a, (hipStream_t)stream), "rope");
}

moe_status moe_kv_append(const moe_kv_cache* cache, const moe_kv_batch* batch, const moe_heads* k,
                         const moe_heads* v, int32_t type, const moe_rope_plan* rope,
                         const int32_t* positions, const moe_heads* q, int32_t n_q_heads,
                         const moe_heads* q_out, uint32_t* err_flags, void* stream) {
  moe_status s = check_cache(cache);
  if (s != MOE_OK) return s;
  if ((s = check_type("k", type, true)) != MOE_OK) return s;
  if ((q == nullptr) != (q_out == nullptr))
    return fail(MOE_ERR_INVALID_ARG, "q and q_out go together: one of them is NULL");
  if (q != nullptr && n_q_heads < 1)
    return fail(MOE_ERR_INVALID_ARG, "n_q_heads = %d < 1", n_q_heads);
  if ((s = check_batch(batch, cache, q ? n_q_heads : 0)) != MOE_OK) return s;
  if (rope != nullptr && (s = check_rope(rope, cache->D)) != MOE_OK) return s;
  if (batch->T == 0 || batch->n_seq == 0) return ok();
  if ((s = check_batch_ptrs(batch, err_flags)) != MOE_OK) return s;
  const int bytes = type_bytes(type);
  if ((s = check_heads("k", k, bytes, 1)) != MOE_OK) return s;
  if ((s = check_heads("v", v, bytes, 1)) != MOE_OK) return s;
  if (q != nullptr) {
    if ((s = check_heads("q", q, bytes, 1)) != MOE_OK) return s;
    if ((s = check_heads("q_out", q_out, bytes, 1)) != MOE_OK) return s;
    if (!same_heads(q, q_out)) return fail(MOE_ERR_INVALID_ARG, "q_out is q with other strides");
    if ((s = check_apart("q_out", q_out, batch->T, n_q_heads, cache->D)) != MOE_OK) return s;
  }
  if (cache->n_heads > 1 && (cache->k_head < cache->D || cache->v_head < cache->D))
    return fail(MOE_ERR_INVALID_ARG, "cache head strides (%lld, %lld): heads of %d values overlap",
                (long long)cache->k_head, (long long)cache->v_head, cache->D);
  if ((uintptr_t)positions & 3) return fail(MOE_ERR_INVALID_ARG, "positions misaligned");
  moe::AppendCall a{};
  a.cache = cache_view(cache), a.batch = batch_view(batch);
  a.rope = rope_view(rope);
  a.k = heads_view(k), a.v = heads_view(v);
  if (q != nullptr) a.q = heads_view(q), a.q_out = heads_view(q_out);
  a.positions = positions;
  a.type = type, a.n_q_heads = n_q_heads, a.err = err_flags;
  clear_stale_error();
  return hip_status(moe::launch_append(a, (hipStream_t)stream), "append to the cache");
}

size_t moe_attend_scratch_bytes(const moe_kv_cache* cache, const moe_kv_batch* batch,
                                int32_t n_q_heads, int32_t window, int32_t keep_first) {
  if (check_attend(cache, batch, n_q_heads, window, keep_first) != MOE_OK) return 0;
  if (batch->T == 0 || batch->n_seq == 0) return 0;
  return attend_scratch(cache, plan_of(cache, batch, n_q_heads, window, keep_first));
}

moe_status moe_attend(const moe_kv_cache* cache, const moe_kv_batch* batch, const moe_heads* q,
                      int32_t type, int32_t n_q_heads, float scale, int32_t causal, int32_t window,
                      int32_t keep_first, const float* sinks, const moe_heads* out, void* scratch,
                      size_t scratch_bytes, uint32_t* err_flags, void* stream) {
  moe_status s = check_attend(cache, batch, n_q_heads, window, keep_first);
  if (s != MOE_OK) return s;
  if ((s = check_16bit("q", type)) != MOE_OK) return s;
  if (cache->type != MOE_T_E4M3 && cache->type != type)
    return fail(MOE_ERR_UNSUPPORTED, "q of type %d on a cache of type %d", type, cache->type);
  if (!std::isfinite(scale)) return fail(MOE_ERR_INVALID_ARG, "scale is not finite");
  if (window > 0 && !causal) return fail(MOE_ERR_INVALID_ARG, "a window needs causal");
  if (batch->T == 0 || batch->n_seq == 0) return ok();
  if ((s = check_batch_ptrs(batch, err_flags)) != MOE_OK) return s;
  if ((s = check_heads("q", q, 16, 8)) != MOE_OK) return s;
  if ((s = check_heads("out", out, 16, 8)) != MOE_OK) return s;
  if (out->p == q->p) return fail(MOE_ERR_INVALID_ARG, "out is q");
  if ((s = check_apart("out", out, batch->T, n_q_heads, cache->D)) != MOE_OK) return s;
  if ((uintptr_t)sinks & 3) return fail(MOE_ERR_INVALID_ARG, "sinks misaligned");
  moe::AttendCall a{};
  const moe::AttendPlan plan = plan_of(cache, batch, n_q_heads, window, keep_first);
  a.splits = plan.splits, a.splits_few = plan.splits_few, a.few = plan.few, a.both = plan.both;
  if (const size_t need = attend_scratch(cache, plan)) {
    CHECK_PTR(scratch);
    if (scratch_bytes < need)
      return fail(MOE_ERR_INVALID_ARG, "scratch holds %zu bytes, %zu needed", scratch_bytes, need);
    const int64_t many = part_rows(plan), few = part_rows_few(plan);
    float* sums = (float*)scratch;
    float* stats = sums + (many + few) * cache->D;
    a.parts = {sums, stats, plan.rows};
    a.parts_few = {sums + many * cache->D, stats + 2 * many, plan.rows_few};
  }
  a.cache = cache_view(cache), a.batch = batch_view(batch);
  a.q = heads_view(q), a.out = heads_view(out);
  a.type = type, a.n_q_heads = n_q_heads, a.group = n_q_heads / cache->n_heads;
  a.group_inv = 0xFFFFFFFFu / (uint32_t)a.group;
  a.scale = scale, a.causal = causal != 0, a.window = window, a.keep_first = keep_first;
  a.sinks = sinks, a.err = err_flags;
  clear_stale_error();
  return hip_status(moe::launch_attend(a, (hipStream_t)stream), "attention");
}

moe_status moe_linear(const void* x, int64_t x_stride, const void* w, int64_t w_stride,
                      int32_t type, int32_t M, int32_t N, int32_t K, const void* bias,
                      int32_t bias_type, int32_t act, const void* resid, int64_t resid_stride,
                      void* out, int32_t out_type, int64_t out_stride, void* stream) {
  moe_status s = check_16bit("x", type);
  if (s != MOE_OK) return s;
  if ((s = check_type("out", out_type, true)) != MOE_OK) return s;
  if (bias != nullptr && (s = check_type("bias", bias_type, true)) != MOE_OK) return s;
  if (act < MOE_ACT_NONE || act > MOE_ACT_SILU)
    return fail(MOE_ERR_UNSUPPORTED, "unknown activation %d", act);
  if (M < 0 || N < 0 || K < 0 || M >= (1 << 30) || N >= (1 << 30) || K >= (1 << 30) || K % 8)
    return fail(MOE_ERR_INVALID_ARG, "M = %d, N = %d, K = %d: below 2^30, K a multiple of 8", M, N, K);
  const int64_t limit = int64_t(1) << 40;
  if ((int64_t)M * N >= limit) return fail(MOE_ERR_INVALID_ARG, "M * N: limit 2^40");
  if (M == 0 || N == 0) return ok();
  if (K > 0) {
    CHECK_PTR(x);
    CHECK_PTR(w);
    if (x_stride < 0 || w_stride < 0 || x_stride % 8 || w_stride % 8 || x_stride >= limit / M ||
        w_stride >= limit / N)
      return fail(MOE_ERR_INVALID_ARG,
                  "x_stride = %lld, w_stride = %lld: not negative, multiples of 8, rows * stride < 2^40",
                  (long long)x_stride, (long long)w_stride);
  }
  const int bytes = type_bytes(out_type);
  if (out == nullptr || ((uintptr_t)out & (bytes - 1)))
    return fail(MOE_ERR_INVALID_ARG, "out is %s", out ? "misaligned" : "NULL");
  if (((uintptr_t)resid & (bytes - 1)) || (bias && ((uintptr_t)bias & (type_bytes(bias_type) - 1))))
    return fail(MOE_ERR_INVALID_ARG, "bias or resid misaligned");
  if (out_stride < N || out_stride >= limit / M)
    return fail(MOE_ERR_INVALID_ARG, "out_stride = %lld: at least N = %d, rows * stride < 2^40",
                (long long)out_stride, N);
  if (resid != nullptr && (resid_stride < 0 || resid_stride >= limit / M))
    return fail(MOE_ERR_INVALID_ARG, "resid_stride = %lld: not negative, rows * stride < 2^40",
                (long long)resid_stride);
  if (resid == out && M > 1 && resid_stride != out_stride)
    return fail(MOE_ERR_INVALID_ARG, "out is resid with another stride");
  if (K > 0 && (out == x || out == w)) return fail(MOE_ERR_INVALID_ARG, "out is x or w");
  moe::LinearCall a{};
  a.x = (const uint16_t*)x, a.w = (const uint16_t*)w;
  a.x_stride = x_stride, a.w_stride = w_stride, a.resid_stride = resid_stride;
  a.out_stride = out_stride;
  a.type = type, a.M = M, a.N = N, a.K = K;
  a.bias = bias, a.bias_type = bias_type, a.act = act;
  a.resid = resid, a.out = out, a.out_type = out_type;
  clear_stale_error();
  return hip_status(moe::launch_linear(a, (hipStream_t)stream), "linear");
}

}  // extern "C"
