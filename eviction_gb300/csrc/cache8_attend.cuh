// cache8_attend.cuh -- what the two attention kernels of the 8-bit paged cache
// share: few queries (cache8_attend.cu) and many (cache8_attend_many.cu).
#pragma once

#include <atomic>
#include <cfloat>

#include "cache8.cuh"

namespace kvc {
namespace cache8 {

// Division by the block size: floor(t / bs) = umulhi(t, mul) >> shift for
// 0 <= t < 2^31 (bs > 1).
struct Div {
  uint32_t mul;
  int shift, bs;
  __device__ __forceinline__ int div(int t) const {
    return mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(t), mul) >> shift) : t;
  }
};
inline Div make_div(int bs) {
  if (bs == 1) return {0, 0, 1};
  int s = 0;
  while ((1 << s) < bs) ++s;  // 2^(s-1) < bs <= 2^s
  return {static_cast<uint32_t>((1ull << (31 + s)) / bs + 1), s - 1, bs};
}

constexpr int kCounters = 512;  // at the start of the workspace, zero between calls; parts follow

// Beyond 48 KB of shared memory a kernel has to be told so, once per device.
template <class Kernel>
cudaError_t allow_smem(Kernel* kernel, int smem, std::atomic<uint64_t>& told) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(told.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev < 64) told.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  return e;
}

// Many query rows per head: cache8_attend_many.cu.  (All rows of a call go through
// one of the two kernels.)
cudaError_t launch_attend_many(const Cache& c, int format, const AttendArgs& a, cudaStream_t s);
size_t attend_many_parts_bytes(int d);

__device__ __forceinline__ uint32_t half2_of(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// log2 of the power of two that a query row is divided by: its largest magnitude m goes
// to [1, 4) (a zero or subnormal one below), with room in fp16 for all of bf16's range.
__device__ __forceinline__ int row_exp(float m) {
  return min(max(static_cast<int>(__float_as_uint(m) >> 23) - 127, -126), 126);
}
// What a row's scores are multiplied by; finite, so that a score of 0 stays 0.
__device__ __forceinline__ float finite_factor(float a, float b) { return fminf(a * b, FLT_MAX); }

__device__ __forceinline__ int div_up(int a, int b) { return (a + b - 1) / b; }

// Write kPer values of a row and, with the first ones, its lse.
constexpr int kPer = 8;
__device__ __forceinline__ void write_row(const Cache& c, const AttendArgs& a, int l, int b, int h,
                                          int r, int nq, int d0, const float (&x)[kPer], float m,
                                          float sum) {
  const int hq = h * a.G + r / nq, j = r % nq;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint4*>(a.out.at(l, b, hq, j) + d0) =
      make_uint4(bf16x2(x[0] * inv, x[1] * inv), bf16x2(x[2] * inv, x[3] * inv),
                 bf16x2(x[4] * inv, x[5] * inv), bf16x2(x[6] * inv, x[7] * inv));
  if (a.lse && d0 == 0)
    a.lse[((static_cast<size_t>(l) * c.B + b) * c.H * a.G + hq) * a.n + j] =
        (m + __log2f(sum)) * 0.6931471805599453f;
}

}  // namespace cache8
}  // namespace kvc
