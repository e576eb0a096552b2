// rotary.cu -- query and key rows turned by their tokens' positions.
//
// Pair (x, y) of a row goes to (x cos a - y sin a, x sin a + y cos a), a = pos f_i.  The
// frequency is held in turns per token, in 2^-64 of a turn, so that pos * f_i in 64-bit
// integers drops whole turns by itself: the angle is exact at any position, where an fp32
// product is off by 0.06 radians at a million tokens.  The top 32 bits, signed, are the
// angle in half turns, which sincospif takes.
//
// The rows are read and written once, which bounds the call.  A CTA has a few tokens and all
// (or a share) of their heads: it computes their sines and cosines once into shared memory,
// then each thread turns two 16-byte chunks at a time, those that its pairs lie in.
#include "prompt.cuh"

namespace kvc {
namespace prompt {
namespace {

using cache8::before_all;
using cache8::bf16_hi;
using cache8::bf16_lo;
using cache8::bf16x2;

constexpr int kThreads = 256;
constexpr int kTokens = 4;  // of a CTA

__device__ __forceinline__ uint32_t turn_x(uint32_t x, uint32_t y, float2 a, float2 b) {
  return bf16x2(fmaf(bf16_lo(x), a.x, -bf16_lo(y) * a.y), fmaf(bf16_hi(x), b.x, -bf16_hi(y) * b.y));
}
__device__ __forceinline__ uint32_t turn_y(uint32_t x, uint32_t y, float2 a, float2 b) {
  return bf16x2(fmaf(bf16_lo(x), a.y, bf16_lo(y) * a.x), fmaf(bf16_hi(x), b.y, bf16_hi(y) * b.x));
}
__device__ __forceinline__ uint32_t turn_pair(uint32_t xy, float2 a) {
  const float x = bf16_lo(xy), y = bf16_hi(xy);
  return bf16x2(fmaf(x, a.x, -y * a.y), fmaf(x, a.y, y * a.x));
}

// (cos, sin) of a pair at a position, times the magnitude.
__device__ __forceinline__ float2 angle_of(const kvc_rope& r, int i, int pos) {
  const uint64_t a = r.turn[i] * static_cast<uint64_t>(static_cast<int64_t>(pos));
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(a >> 32)) * 0x1p-31f, &s, &c);
  return make_float2(c * r.magnitude, s * r.magnitude);
}

__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a,
                                                          int shares) {
  __shared__ __align__(16) float2 s_cs[kTokens][64];
  __shared__ int s_n[kTokens];  // 1: the token is there
  before_all();
  const long long t0 = static_cast<long long>(blockIdx.x) * kTokens, all = static_cast<long long>(a.S) * a.n;
  const int l = blockIdx.z, pairs = a.rope.dim / 2;
  if (threadIdx.x < kTokens) {
    const long long t = t0 + threadIdx.x;
    int there = t < all;
    if (there && a.n_tok) {
      const int b = static_cast<int>(t / a.n), j = static_cast<int>(t % a.n), m = a.n_tok[b];
      if (m < 0 || m > a.n) {
        there = 0;
        if (j == 0 && l == 0 && blockIdx.y == 0) atomicOr(a.status, KVC_STATUS_BAD_INDEX);
      } else {
        there = j < m;
      }
    }
    s_n[threadIdx.x] = there;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kTokens * pairs; i += kThreads) {
    const int k = i / pairs;
    if (s_n[k]) s_cs[k][i % pairs] = angle_of(a.rope, i % pairs, a.pos[t0 + k]);
  }
  __syncthreads();
  const int units = a.d / 16, turned = a.rope.dim / 16;  // two 16-byte chunks each
  const int heads = a.heads[0] + a.heads[1];
  for (int i = threadIdx.x + blockIdx.y * kThreads; i < kTokens * heads * units;
       i += kThreads * shares) {
    const int u = i % units, row = i / units, head = row % heads, k = row / heads;
    if (!s_n[k]) continue;
    const int w = head < a.heads[0] ? 0 : 1;
    if (u >= turned && a.in_place[w]) continue;
    const long long t = t0 + k;
    const int b = static_cast<int>(t / a.n), j = static_cast<int>(t % a.n);
    const int h = w ? head - a.heads[0] : head;
    // chunks of a turned unit: dim / 2 values apart; of the rest: side by side
    const int c0 = u < turned ? u : 2 * u, c1 = u < turned ? u + turned : 2 * u + 1;
    const uint4* from = reinterpret_cast<const uint4*>(a.in[w].at(l, b, h, j));
    uint4 x = from[c0], y = from[c1];
    if (u < turned) {
      const float4* cs0 = reinterpret_cast<const float4*>(s_cs[k]);
      if (a.rope.interleaved) {
        const float4 p = cs0[2 * c0], q = cs0[2 * c0 + 1], r = cs0[2 * c1], s = cs0[2 * c1 + 1];
        x = make_uint4(turn_pair(x.x, make_float2(p.x, p.y)), turn_pair(x.y, make_float2(p.z, p.w)),
                       turn_pair(x.z, make_float2(q.x, q.y)), turn_pair(x.w, make_float2(q.z, q.w)));
        y = make_uint4(turn_pair(y.x, make_float2(r.x, r.y)), turn_pair(y.y, make_float2(r.z, r.w)),
                       turn_pair(y.z, make_float2(s.x, s.y)), turn_pair(y.w, make_float2(s.z, s.w)));
      } else {
        uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w}, xo[4], yo[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const float4 p = cs0[4 * c0 + z];
          xo[z] = turn_x(xs[z], ys[z], make_float2(p.x, p.y), make_float2(p.z, p.w));
          yo[z] = turn_y(xs[z], ys[z], make_float2(p.x, p.y), make_float2(p.z, p.w));
        }
        x = make_uint4(xo[0], xo[1], xo[2], xo[3]);
        y = make_uint4(yo[0], yo[1], yo[2], yo[3]);
      }
    }
    uint4* to = reinterpret_cast<uint4*>(a.out[w].at(l, b, h, j));
    to[c0] = x;
    to[c1] = y;
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s) {
  const long long groups = (static_cast<long long>(a.S) * a.n + kTokens - 1) / kTokens;
  return cache8::launch(rotary_kernel, dim3(static_cast<unsigned>(groups), 1, a.L), kThreads, 0, s, a,
                        1);
}

}  // namespace prompt
}  // namespace kvc
