// heaviest.cu -- the tokens that an eviction by gathered weight keeps (kvc_keep_heaviest):
// per unit the last and the first tokens and the heaviest of the others, in order.
//
// The least weight that is kept is found by a radix select over order-preserving 32-bit
// keys, 8 bits a pass (a histogram in shared memory, then the bin that the wanted rank falls
// into).  Tokens above it are kept, and of those equal to it the first ones.
#include "prompt.cuh"

namespace kvc {
namespace prompt {
namespace {

using cache8::before_all;

constexpr int kThreads = 256, kWarps = kThreads / 32;

// Larger weight, larger key; NaN below all, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float w) {
  return w == w ? float_order_key(w + 0.f) : 0u;
}

// What a unit keeps without looking at weights, and how many others.
struct Plan {
  int len, n, head, tail, want;  // tokens < head and >= tail; want others
  bool bad;
};
__device__ __forceinline__ Plan plan_of(const HeaviestArgs& a, int b) {
  Plan p;
  p.len = a.seq_len[b];
  p.bad = p.len < 0 || p.len > a.cap;
  p.n = min(p.len, a.budget);
  const int recent = min(a.n_recent, a.budget);
  p.tail = max(p.len - recent, 0);
  p.head = min(min(a.n_sink, a.budget - recent), p.tail);
  p.want = p.n - p.head - (p.len - p.tail);
  return p;
}

// Exclusive prefix sum over the CTA; *all: the total.  Barriers inside.
__device__ __forceinline__ int prefix(int v, int* s_warp, int* all) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_warp[w];
    total += s_warp[w];
  }
  __syncthreads();
  *all = total;
  return before + incl - v;
}

__global__ void __launch_bounds__(kThreads) heaviest_kernel(HeaviestArgs a) {
  __shared__ int s_hist[256], s_warp[kWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_want;
  before_all();
  const int u = blockIdx.x, b = (u / a.H) % a.B;
  const Plan p = plan_of(a, b);
  if (p.bad) {
    if (threadIdx.x == 0) atomicOr(a.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  const float* w = a.w + static_cast<size_t>(u) * a.cap;
  // ---- the least key that is kept, and how many of those equal to it ----
  uint32_t least = 0;
  int equal = 0;
  if (p.want > 0) {
    if (threadIdx.x == 0) {
      s_prefix = 0;
      s_want = p.want;
    }
    for (int shift = 24; shift >= 0; shift -= 8) {
      s_hist[threadIdx.x] = 0;
      __syncthreads();
      const uint32_t so_far = s_prefix;
      for (int t = p.head + threadIdx.x; t < p.tail; t += kThreads) {
        const uint32_t k = key_of(w[t]);
        if (shift == 24 || (k >> (shift + 8)) == (so_far >> (shift + 8)))
          atomicAdd(&s_hist[(k >> shift) & 255], 1);
      }
      __syncthreads();
      int all;
      const int bin = 255 - threadIdx.x, n = s_hist[bin];  // heaviest first
      const int want = s_want, above = prefix(n, s_warp, &all);
      if (above < want && above + n >= want) {
        s_prefix = so_far | static_cast<uint32_t>(bin) << shift;
        s_want = want - above;
      }
      __syncthreads();
    }
    least = s_prefix;
    equal = s_want;
  }
  // ---- the kept tokens in order (weights_out may be weights: a chunk is read before
  // what it keeps is written, to places that are not behind it) ----
  int32_t* kept = a.kept + static_cast<size_t>(u) * a.budget;
  float* out = a.out + static_cast<size_t>(u) * a.cap;
  int done = 0, equals = 0;
  for (int t0 = 0; t0 < p.len; t0 += kThreads) {
    const int t = t0 + threadIdx.x;
    const float x = t < p.len ? w[t] : 0.f;
    const uint32_t k = key_of(x);
    const bool other = t >= p.head && t < p.tail, same = other && p.want > 0 && k == least;
    int all;
    const int rank = equals + prefix(same, s_warp, &all);
    equals += all;
    const bool keep = t < p.len && (!other || (p.want > 0 && (k > least || (same && rank < equal))));
    const int at = done + prefix(keep, s_warp, &all);
    done += all;
    if (keep) {
      kept[at] = t;
      out[at] = x;
    }
  }
  __syncthreads();
  for (int i = p.n + threadIdx.x; i < a.budget; i += kThreads) kept[i] = -1;
  for (int i = p.n + threadIdx.x; i < a.cap; i += kThreads) out[i] = 0.f;
  if (threadIdx.x == 0) a.n_kept[u] = p.n;
}

}  // namespace

cudaError_t launch_heaviest(const HeaviestArgs& a, cudaStream_t s) {
  return cache8::launch(heaviest_kernel, a.L * a.B * a.H, kThreads, 0, s, a);
}

}  // namespace prompt
}  // namespace kvc
