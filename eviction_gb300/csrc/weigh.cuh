// weigh.cuh -- what the two kernels of kvc_cache8_weigh share: few query rows (weigh.cu) and
// many (weigh_many.cu).
#pragma once

#include "cache8_attend.cuh"
#include "prompt.cuh"

namespace kvc {
namespace prompt {

// Queries and tokens of sequence b; none where they are out of range.
struct Lengths {
  int len, nq, first;
};
__device__ __forceinline__ Lengths lengths_of(const cache8::Cache& c, const WeighArgs& a, int b,
                                              bool* bad) {
  Lengths x;
  bool wrong = false;
  x.len = cache8::length_of(c, b, &wrong);
  x.nq = a.n_q ? a.n_q[b] : a.n;
  x.first = a.first ? a.first[b] : 0;
  if (wrong || x.len > a.cap || x.nq < 0 || x.nq > x.len || x.first < 0 || x.nq > a.n - x.first) {
    *bad = true;
    x.len = x.nq = x.first = 0;
  }
  return x;
}

// Many query rows of a head: weigh_many.cu.
cudaError_t launch_weigh_many(const cache8::Cache& c, int format, const WeighArgs& a, cudaStream_t s);

// A query's lse in base 2 as the weights take it: 2^(z - y); no token for one that saw none.
__device__ __forceinline__ bool sees_nothing(float lse) { return fabsf(lse) == INFINITY; }
__device__ __forceinline__ float lse_base2(float lse) {
  return sees_nothing(lse) ? INFINITY : lse * 1.4426950408889634f;
}

}  // namespace prompt
}  // namespace kvc
