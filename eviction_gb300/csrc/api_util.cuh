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

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

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

// Strides are multiples of 8 values and not negative.  An output's rows may not share
// memory: each axis has to step over all that the axes of smaller strides span (true of
// any slice or permutation of a dense array).  Strides of axes of size 1 do not matter.
inline int check_rows(kvc_handle* h, const kvc_rows* r, const char* name, bool written, int L, int B,
                      int heads, int n) {
  if (!r || !r->data) return fail(h, KVC_ERR_ARG, std::string("null pointer: ") + name);
  if (!aligned16(r->data)) return fail(h, KVC_ERR_ALIGN, std::string("not 16-byte aligned: ") + name);
  const int64_t stride[4] = {r->layer, r->seq, r->head, r->token};
  const int size[4] = {L, B, heads, n};
  for (int i = 0; i < 4; ++i) {
    if (size[i] > 1 && (stride[i] < 0 || stride[i] % 8))
      return fail(h, KVC_ERR_ALIGN, std::string("strides must be multiples of 8 and >= 0: ") + name);
    if (!written || size[i] == 1) continue;
    __int128 span = h->dims.d;  // values from the first to past the last of the axes below
    for (int k = 0; k < 4; ++k)
      if (size[k] > 1 && (stride[k] < stride[i] || (stride[k] == stride[i] && k < i)))
        span += static_cast<__int128>(stride[k]) * (size[k] - 1);
    if (stride[i] < span) return fail(h, KVC_ERR_ARG, std::string("rows overlap: ") + name);
  }
  return KVC_OK;
}

// The handle's device has to be the current one.
inline int check_device(kvc_handle* h) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(h, e, "current device");
  if (dev != h->device)
    return fail(h, KVC_ERR_DEVICE, "the handle belongs to another device than the current one");
  return KVC_OK;
}

// What an entry point does after its checks: the launch between two tracing marks.
// Nothing thrown (an allocation of the error text or of a mark) leaves the C ABI.
template <class F>
int run(kvc_handle* h, int kernel, const char* name, void* stream, F launch) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaEvent_t b = mark_begin(h, s);
  cudaError_t e = launch(s);
  if (e != cudaSuccess) return cuda_fail(h, e, name);
  mark_end(h, kernel, b, s);
  return KVC_OK;
}
template <class F>
int guarded(F f) {
  try {
    return f();
  } catch (...) {
    return KVC_ERR_NOMEM;
  }
}

#define KVC_TRY(expr)               \
  do {                              \
    if (const int rc_ = (expr)) return rc_; \
  } while (0)

#define KVC_REQUIRE_INTS(p)                                                       \
  do {                                                                            \
    if (!(p)) return fail(h, KVC_ERR_ARG, "null pointer: " #p);                   \
    if (!aligned4(p)) return fail(h, KVC_ERR_ALIGN, "not 4-byte aligned: " #p);   \
  } while (0)

inline float scale_log2_of(const kvc_config& c) {
  const double s = c.softmax_scale > 0.f ? static_cast<double>(c.softmax_scale)
                                         : 1.0 / std::sqrt(static_cast<double>(c.head_dim));
  return static_cast<float>(s * 1.4426950408889634);
}

}  // namespace kvc
