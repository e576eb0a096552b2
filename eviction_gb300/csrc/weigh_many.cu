// weigh.cu -- attention weight that the newest tokens' queries give each token of the 8-bit
// paged cache, added to what it has gathered (kvc_cache8_weigh).  One thread a token.
#include "weigh.cuh"

namespace kvc {
namespace prompt {
namespace {

using namespace cache8;

constexpr int kThreads = 128;

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) weigh_many_kernel(Cache c, WeighArgs a) {
  before_all();
  const int per = (a.cap + kThreads - 1) / kThreads;
  const int u = blockIdx.x / per, t = blockIdx.x % per * kThreads + threadIdx.x;
  const int h = u % c.H, b = (u / c.H) % c.B, l = u / (c.H * c.B);
  bool bad = false;
  const int len = length_of(c, b, &bad);
  const int nq = a.n_q ? a.n_q[b] : a.n, first = a.first ? a.first[b] : 0;
  if (bad || len > a.cap || nq < 0 || nq > len || first < 0 || nq > a.n - first) {
    if (threadIdx.x == 0 && t < kThreads) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  if (t >= len) return;
  float* w = a.w + static_cast<size_t>(u) * a.cap + t;
  const float old = a.decay == 0.f ? 0.f : a.decay * *w;
  const int blk = block_at(c, b, t / c.bs);
  if (blk < 0) {
    atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    *w = old;
    return;
  }
  float k[D];
  const uint32_t* codes =
      reinterpret_cast<const uint32_t*>(c.pool[0] + (block_row(c, l, blk, h) + t % c.bs) * D);
#pragma unroll
  for (int i = 0; i < D / 4; ++i) {
    float x[4];
    decode4<FMT>(codes[i], x);
#pragma unroll
    for (int j = 0; j < 4; ++j) k[4 * i + j] = x[j];
  }
  const float f = a.scale_log2 * c.scale[0][scale_at(c, l, blk, h)];
  const int sb = a.first ? 0 : b, S = a.first ? 1 : c.B;
  float sum = 0.f;
  for (int g = 0; g < a.G; ++g) {
    const float* lse = a.lse + ((static_cast<size_t>(l) * S + sb) * c.H * a.G + h * a.G + g) * a.n + first;
    for (int j = max(0, t - (len - nq)); j < nq; ++j) {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(a.q.at(l, sb, h * a.G + g, first + j));
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < D / 2; ++i) z += bf16_lo(q[i]) * k[2 * i] + bf16_hi(q[i]) * k[2 * i + 1];
      const float y = lse[j] == -INFINITY ? INFINITY : lse[j] * 1.4426950408889634f;
      sum += exp2f(z * f - y);
    }
  }
  *w = old + sum;
}

}  // namespace

cudaError_t launch_weigh_many(const Cache& c, int format, const WeighArgs& a, cudaStream_t s) {
  const int grid = c.L * c.B * c.H * ((a.cap + kThreads - 1) / kThreads);
  auto* kernel = c.d == 64 ? (format == KVC_CACHE8_E4M3 ? weigh_many_kernel<64, KVC_CACHE8_E4M3>
                                                        : weigh_many_kernel<64, KVC_CACHE8_INT8>)
                           : (format == KVC_CACHE8_E4M3 ? weigh_many_kernel<128, KVC_CACHE8_E4M3>
                                                        : weigh_many_kernel<128, KVC_CACHE8_INT8>);
  return launch(kernel, grid, kThreads, 0, s, c, a);
}

}  // namespace prompt
}  // namespace kvc
