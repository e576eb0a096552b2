// api_util.cuh -- host helpers shared by the entry points' source files: error
// codes with their text, pointer checks, and the per-kernel tracing marks.
#pragma once

#include <cmath>
#include <string>

#include "kvc_internal.cuh"

namespace kvc {

inline int fail(kvc_handle* h, int code, const std::string& msg) {
  if (h) h->last_error = msg;
  return code;
}

inline bool aligned16(const void* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

inline int cuda_fail(kvc_handle* h, cudaError_t e, const char* where) {
  return fail(h, KVC_ERR_CUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

inline cudaEvent_t prof_event(kvc_handle* h) {
  auto& P = h->prof;
  if (!P.pool.empty()) {
    cudaEvent_t e = P.pool.back();
    P.pool.pop_back();
    return e;
  }
  cudaEvent_t e = nullptr;
  if (cudaEventCreate(&e) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  return e;
}

// Record the start of one kernel launch (nullptr when tracing is off).
inline cudaEvent_t mark_begin(kvc_handle* h, cudaStream_t s) {
  if (!h->prof.enabled) return nullptr;
  cudaEvent_t e = prof_event(h);
  if (e) cudaEventRecord(e, s);
  return e;
}

inline void mark_end(kvc_handle* h, int kernel, cudaEvent_t begin, cudaStream_t s) {
  if (!begin) return;
  cudaEvent_t e = prof_event(h);
  if (!e) {
    h->prof.pool.push_back(begin);
    return;
  }
  cudaEventRecord(e, s);
  h->prof.pending.push_back({kernel, begin, e});
}

#define KVC_REQUIRE_PTR(p)                                                    \
  do {                                                                        \
    if (!(p)) return fail(h, KVC_ERR_ARG, "null pointer: " #p);               \
    if (!aligned16(p)) return fail(h, KVC_ERR_ALIGN, "not 16-byte aligned: " #p); \
  } while (0)

inline float scale_log2_of(const kvc_config& c) {
  const double s = c.softmax_scale > 0.f ? static_cast<double>(c.softmax_scale)
                                         : 1.0 / std::sqrt(static_cast<double>(c.head_dim));
  return static_cast<float>(s * 1.4426950408889634);
}

}  // namespace kvc
