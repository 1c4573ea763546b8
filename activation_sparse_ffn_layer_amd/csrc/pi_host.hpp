// Host-side pieces shared by the library's source files: the context, error reporting, kernel
// launches and pointer checks.
#pragma once
#include <hip/hip_runtime.h>
#include <hip/hip_ext.h>

#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <string>
#include <vector>

#include "pi.h"
#include "pi_device.hpp"

using pi::half_t;

struct pi_ctx {
  std::atomic<int> refs{1};  // its creator's until pi_ctx_destroy, and one of each handle
  int device = 0;
  hipStream_t stream = nullptr;
  int max_batch = 0, max_d = 0, max_ffn = 0, max_rank = 0;
  int cus = 256;
  size_t lds_max = 65536;
  uint8_t* ws = nullptr;
  size_t ws_bytes = 0;
  float* z = nullptr;           // [max_batch][max_rank]
  uint64_t* mtok = nullptr;     // [max_batch][max_ffn/64]
  uint64_t* munion = nullptr;   // [max_ffn/64]
  int32_t* idx = nullptr;       // [max_ffn]
  int32_t* nbuf = nullptr;      // [16]
  float* a = nullptr;           // [max_ffn][NB] on the vector path (NB = batch class 1/2/4/8), by neuron id
  float* hp = nullptr;          // slice partials of the column-sliced up GEMV
  int mask_mode = PI_MASK_UNION; // masking of batches (pi_ctx_set_mask_mode)
  int down_g = 8;               // partial sums the last enqueued down projection left in part
  size_t hp_cap = 0;            // floats in hp
  float* part = nullptr;        // [32][max_batch][max_d] down-projection partial sums (groups or K splits)
  float* y = nullptr;           // [max_batch][max_d]
  float* ssq = nullptr;         // [GLUE_SLICES_MAX][2]: k_glue_sum's slice sums of squares
  uint8_t* xbuf[2] = {nullptr, nullptr};  // [max_batch][max_d] fp32-sized
  uint8_t* xstage = nullptr;    // [max_batch][max_d] fp32-sized
  int32_t* nlog = nullptr;      // [NLOG_CAP]
  // batched (matrix-core) path
  float* zpart = nullptr;       // [MM_KS1][max_batch][max_rank]
  half_t* zhi = nullptr;        // [max_batch][max_rank]
  half_t* zlo = nullptr;
  half_t* a16 = nullptr;        // [32 or 64][lda] activations at compacted positions
  int lda = 0;
  int32_t* lin_part = nullptr;  // sums of the 8-bit product's ranges of K (pi_linear_create)
  std::string err;
  // cached graph of one stack step, captured on a private stream (the caller's stream may be
  // the null stream, which cannot be captured) and launched on the caller's stream
  hipStream_t cap_stream = nullptr;
  hipGraphExec_t gexec = nullptr;
  std::vector<uint64_t> g_layers;  // serial numbers of the captured step's layers
  int g_B = 0;
  // per-kernel event timing (pi_stack_profile only)
  bool profiling = false;
  std::vector<hipEvent_t> ev;     // pairs: ev[2i] before, ev[2i+1] after launch i
  std::vector<int> ev_class;
  size_t ev_used = 0;
};

namespace pi {

inline pi_status fail(pi_ctx* ctx, pi_status s, const char* fmt, ...) {
  if (ctx != nullptr) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    ctx->err = buf;
  }
  return s;
}

#define PI_HIP(ctx, call)                                                                        \
  do {                                                                                           \
    hipError_t e_ = (call);                                                                      \
    if (e_ != hipSuccess) return fail((ctx), PI_ERR_HIP, "%s: %s", #call, hipGetErrorString(e_)); \
  } while (0)

// A handle refers to its context until it is destroyed itself, in whatever order: what
// pi_ctx_destroy leaves is an empty context at an address that no other one takes.
inline void ctx_retain(pi_ctx* c) { c->refs.fetch_add(1); }
inline void ctx_release(pi_ctx* c) {
  if (c->refs.fetch_sub(1) == 1) delete c;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The next free pair of profiling events, tagged with a kernel class.
inline void prof_slot(pi_ctx* c, int klass, hipEvent_t* e0, hipEvent_t* e1) {
  if (c->ev_used * 2 + 2 > c->ev.size()) {
    hipEvent_t a = nullptr, b = nullptr;
    if (hipEventCreate(&a) != hipSuccess) return;
    if (hipEventCreate(&b) != hipSuccess) {
      (void)hipEventDestroy(a);
      return;
    }
    c->ev.push_back(a);
    c->ev.push_back(b);
    c->ev_class.push_back(klass);
  }
  const size_t slot = c->ev_used++;
  c->ev_class[slot] = klass;
  *e0 = c->ev[2 * slot];
  *e1 = c->ev[2 * slot + 1];
}

// One kernel launch (`block` threads per workgroup; BLOCK for launch_k) on the context's stream. When profiling,
// the dispatch itself carries a pair of events (hipExtLaunchKernelGGL), so the pair times the
// kernel's execution, not the queueing around it.
template <typename... P, typename... A>
hipError_t launch_kb(pi_ctx* c, int klass, void (*kern)(P...), dim3 grid, int block, size_t lds, A... args) {
  hipEvent_t e0 = nullptr, e1 = nullptr;
  if (c->profiling) prof_slot(c, klass, &e0, &e1);
  if (e0 != nullptr)
    hipExtLaunchKernelGGL(kern, grid, dim3(block), (uint32_t)lds, c->stream, e0, e1, 0u, static_cast<P>(args)...);
  else
    hipLaunchKernelGGL(kern, grid, dim3(block), lds, c->stream, static_cast<P>(args)...);
  return hipGetLastError();
}
template <typename... P, typename... A>
hipError_t launch_k(pi_ctx* c, int klass, void (*kern)(P...), dim3 grid, size_t lds, A... args) {
  return launch_kb(c, klass, kern, grid, BLOCK, lds, args...);
}
template <typename K>
hipError_t allow_lds(K kernel, size_t bytes) {
  if (bytes <= 65536) return hipSuccess;
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                             (int)bytes);
}

inline pi_status check_dev_ptr(pi_ctx* c, const void* p, const char* name, bool nullable = false) {
  if (p == nullptr) return nullable ? PI_OK : fail(c, PI_ERR_INVALID, "%s is NULL", name);
  if (!aligned16(p)) return fail(c, PI_ERR_INVALID, "%s is not 16-byte aligned", name);
  return PI_OK;
}

#define PI_TRY(expr)                 \
  do {                               \
    pi_status s_ = (expr);           \
    if (s_ != PI_OK) return s_;      \
  } while (0)

}  // namespace pi
