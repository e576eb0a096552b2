// prompt_attend.cu -- causal attention over whole prompts, one warp a query row.
#include "prompt.cuh"

namespace kvc {
namespace prompt {
namespace {

using cache8::before_all;
using cache8::bf16_hi;
using cache8::bf16_lo;
using cache8::bf16x2;

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) prompt_attend_kernel(AttendArgs a) {
  constexpr int V = D / 64;  // pairs of values a lane
  before_all();
  const int lane = threadIdx.x % 32;
  const long long task = static_cast<long long>(blockIdx.x) * kWarps + threadIdx.x / 32;
  const int hq = static_cast<int>(task % (a.H * a.G));
  const long long t1 = task / (a.H * a.G);
  const int j = static_cast<int>(t1 % a.n), b = static_cast<int>(t1 / a.n);
  if (b >= a.S) return;
  const int m = a.n_tok ? a.n_tok[b] : a.n, first = a.first ? a.first[b] : 0;
  if (m < 0 || first < 0 || m > a.n - first) {
    if (j == 0 && hq == 0 && lane == 0) atomicOr(a.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  if (j >= m) return;
  const int sb = a.first ? 0 : b, h = hq / a.G;
  uint32_t q[V];
  float o[2 * V] = {}, mx = -INFINITY, sum = 0.f;
  for (int x = 0; x < V; ++x)
    q[x] = reinterpret_cast<const uint32_t*>(a.q.at(0, sb, hq, first + j))[lane + 32 * x];
  for (int t = 0; t <= j; ++t) {
    const uint32_t* k = reinterpret_cast<const uint32_t*>(a.k.at(0, sb, h, first + t));
    const uint32_t* v = reinterpret_cast<const uint32_t*>(a.v.at(0, sb, h, first + t));
    float z = 0.f;
#pragma unroll
    for (int x = 0; x < V; ++x)
      z += bf16_lo(q[x]) * bf16_lo(k[lane + 32 * x]) + bf16_hi(q[x]) * bf16_hi(k[lane + 32 * x]);
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) z += __shfl_xor_sync(0xffffffffu, z, i);
    z *= a.scale_log2;
    const float top = fmaxf(mx, z), keep = exp2f(mx - top), p = exp2f(z - top);
    mx = top;
    sum = sum * keep + p;
#pragma unroll
    for (int x = 0; x < V; ++x) {
      o[2 * x] = o[2 * x] * keep + p * bf16_lo(v[lane + 32 * x]);
      o[2 * x + 1] = o[2 * x + 1] * keep + p * bf16_hi(v[lane + 32 * x]);
    }
  }
  uint32_t* out = reinterpret_cast<uint32_t*>(a.out.at(0, sb, hq, first + j));
  for (int x = 0; x < V; ++x) out[lane + 32 * x] = bf16x2(o[2 * x] / sum, o[2 * x + 1] / sum);
  if (a.lse && lane == 0)
    a.lse[(static_cast<size_t>(sb) * a.H * a.G + hq) * a.n + first + j] =
        (mx + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s) {
  const long long tasks = static_cast<long long>(a.S) * a.n * a.H * a.G;
  const dim3 grid(static_cast<unsigned>((tasks + kWarps - 1) / kWarps));
  return a.d == 64 ? cache8::launch(prompt_attend_kernel<64>, grid, 32 * kWarps, 0, s, a)
                   : cache8::launch(prompt_attend_kernel<128>, grid, 32 * kWarps, 0, s, a);
}

}  // namespace prompt
}  // namespace kvc
