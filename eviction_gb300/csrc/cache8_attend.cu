// cache8_attend.cu -- attention of the newest tokens' queries over the 8-bit
// paged cache (kvc_cache8_attend).
//
// One warp per query row: each lane holds d/32 values of q and of the output, the
// tokens come one after another, with the running maximum and sum of the softmax.
#include "cache8.cuh"

namespace kvc {

size_t cache8_attend_workspace(int d) { return 0 * d; }

namespace cache8 {
namespace {

constexpr int kWarps = 4;

template <int D, int FMT>
__global__ void __launch_bounds__(32 * kWarps) attend_kernel(Cache c, AttendArgs a) {
  constexpr int PER = D / 32;
  const int lane = threadIdx.x % 32;
  const int Hq = c.H * a.G;
  const long long task = static_cast<long long>(blockIdx.x) * kWarps + threadIdx.x / 32;
  const int j = static_cast<int>(task % a.n);
  const long long t1 = task / a.n;
  const int hq = static_cast<int>(t1 % Hq);
  const long long t2 = t1 / Hq;
  const int b = static_cast<int>(t2 % c.B);
  const int l = static_cast<int>(t2 / c.B);
  if (t2 / c.B >= c.L) return;
  const int h = hq / a.G;
  bool bad = false;
  const int len = length_of(c, b, &bad);
  const int nq = a.n_q ? a.n_q[b] : a.n;
  if (bad || nq < 0 || nq > a.n) {
    if (lane == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  if (j >= nq) return;
  const int end = max(0, len - nq + j + 1);  // tokens this query sees
  const uint16_t* q = a.q.at(l, b, hq, j);
  float qf[PER], o[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    qf[i] = __uint_as_float(static_cast<uint32_t>(q[lane * PER + i]) << 16) * a.scale_log2;
    o[i] = 0.f;
  }
  float m = -INFINITY, sum = 0.f;
  for (int t = 0; t < end; ++t) {
    const int blk = block_at(c, b, t / c.bs);
    if (blk < 0) {
      bad = true;
      continue;
    }
    const size_t row = (block_row(c, l, blk, h) + t % c.bs) * D + lane * PER;
    const size_t sc = scale_at(c, l, blk, h);
    float x[4];
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) codes |= static_cast<uint32_t>(c.pool[0][row + i]) << (8 * i);
    decode4<FMT>(codes, x);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) z = fmaf(qf[i], x[i], z);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
    z *= c.scale[0][sc];
    const float mn = fmaxf(m, z);
    const float keep = mn == m ? 1.f : exp2f(m - mn);
    const float p = z == mn ? 1.f : exp2f(z - mn);
    m = mn;
    sum = sum * keep + p;
    codes = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) codes |= static_cast<uint32_t>(c.pool[1][row + i]) << (8 * i);
    decode4<FMT>(codes, x);
    const float pv = p * c.scale[1][sc];
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = o[i] * keep + pv * x[i];
  }
  const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
  uint16_t* out = a.out.at(l, b, hq, j);
#pragma unroll
  for (int i = 0; i < PER; ++i)
    out[lane * PER + i] = static_cast<uint16_t>(bf16x2(o[i] * inv, 0.f));
  if (a.lse && lane == 0)
    a.lse[(static_cast<size_t>(l) * c.B + b) * Hq * a.n + static_cast<size_t>(hq) * a.n + j] =
        (m + log2f(sum)) * 0.6931471805599453f;
  if (bad && lane == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
}

}  // namespace

cudaError_t launch_attend(const Cache& c, int format, const AttendArgs& a, cudaStream_t s) {
  const long long rows = static_cast<long long>(c.L) * c.B * c.H * a.G * a.n;
  const int grid = static_cast<int>((rows + kWarps - 1) / kWarps);
  auto* kernel = c.d == 64 ? (format == KVC_CACHE8_E4M3 ? attend_kernel<64, KVC_CACHE8_E4M3>
                                                        : attend_kernel<64, KVC_CACHE8_INT8>)
                           : (format == KVC_CACHE8_E4M3 ? attend_kernel<128, KVC_CACHE8_E4M3>
                                                        : attend_kernel<128, KVC_CACHE8_INT8>);
  kernel<<<grid, 32 * kWarps, 0, s>>>(c, a);
  return cudaGetLastError();
}

}  // namespace cache8
}  // namespace kvc
