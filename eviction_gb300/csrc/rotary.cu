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
// then each thread turns two 16-byte chunks of a row at a time, those that its pairs lie in.
#include "cache8_attend.cuh"
#include "prompt.cuh"

namespace kvc {
namespace prompt {
namespace {

using cache8::before_all;
using cache8::bf16_hi;
using cache8::bf16_lo;
using cache8::bf16x2;

constexpr int kThreads = 256;
constexpr int kTokens = 8;  // of a CTA at most
constexpr int kBatch = 4;   // rows of a thread whose loads are in flight together

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

// Both chunks of a unit turned: pairs of chunk c0's values and chunk c1's, or of side by side values.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn(uint4& x, uint4& y, const float4* cs, int c0, int c1) {
  uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int z = 0; z < 4; z += INTERLEAVED ? 2 : 1) {
    if constexpr (INTERLEAVED) {
      const float4 p = cs[2 * c0 + z / 2], q = cs[2 * c1 + z / 2];
      xs[z] = turn_pair(xs[z], make_float2(p.x, p.y));
      xs[z + 1] = turn_pair(xs[z + 1], make_float2(p.z, p.w));
      ys[z] = turn_pair(ys[z], make_float2(q.x, q.y));
      ys[z + 1] = turn_pair(ys[z + 1], make_float2(q.z, q.w));
    } else {
      const float4 p = cs[4 * c0 + z];
      const float2 a = make_float2(p.x, p.y), b = make_float2(p.z, p.w);
      const uint32_t first = turn_x(xs[z], ys[z], a, b);
      ys[z] = turn_y(xs[z], ys[z], a, b);
      xs[z] = first;
    }
  }
  x = make_uint4(xs[0], xs[1], xs[2], xs[3]);
  y = make_uint4(ys[0], ys[1], ys[2], ys[3]);
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a,
                                                          int tokens, int shares, cache8::Div by_heads) {
  constexpr int kUnits = D / 16;                 // of a row: two 16-byte chunks each
  constexpr int kRows = kThreads / kUnits;       // rows that the CTA's threads take at a time
  __shared__ __align__(16) float2 s_cs[kTokens][64];
  __shared__ long long s_at[4][kTokens];         // a token's place in the rows of in, in, out, out
  __shared__ int s_pos[kTokens], s_there[kTokens];
  before_all();
  const long long t0 = static_cast<long long>(blockIdx.x) * tokens, all = static_cast<long long>(a.S) * a.n;
  const int l = blockIdx.z, pairs = a.rope.dim / 2, turned = a.rope.dim / 16;
  if (threadIdx.x < tokens) {
    const long long t = t0 + threadIdx.x;
    int there = t < all, pos = 0;
    if (there) {
      pos = a.pos[t];
      const int b = static_cast<int>(t / a.n), j = static_cast<int>(t % a.n);
      if (a.n_tok) {
        const int m = a.n_tok[b];
        there = j < m && m <= a.n;
        if ((m < 0 || m > a.n) && j == 0 && l == 0 && blockIdx.y == 0)
          atomicOr(a.status, KVC_STATUS_BAD_INDEX);
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        s_at[w][threadIdx.x] = l * a.in[w].layer + b * a.in[w].seq + j * a.in[w].token;
        s_at[w + 2][threadIdx.x] = l * a.out[w].layer + b * a.out[w].seq + j * a.out[w].token;
      }
    }
    s_there[threadIdx.x] = there;
    s_pos[threadIdx.x] = pos;
  }
  __syncthreads();
  // This thread: unit u of rows (token, head) i, i + kRows, ...; a few rows' loads together, the
  // first ones before the angles.
  const int u = threadIdx.x % kUnits, heads = a.heads[0] + a.heads[1], total = tokens * heads;
  // chunks of a turned unit: dim / 2 values apart; of the rest: side by side
  const int c0 = u < turned ? u : 2 * u, c1 = u < turned ? u + turned : 2 * u + 1;
  uint4 x[kBatch], y[kBatch];
  auto row_of = [&](int i, int* k, int* w) {  // its head among its kind; -1: nothing to do
    if (i >= total) return -1;
    *k = by_heads.div(i);
    const int head = i - *k * heads;
    *w = head >= a.heads[0];
    if (!s_there[*k] || (u >= turned && a.in_place[*w])) return -1;
    return *w ? head - a.heads[0] : head;
  };
  auto load = [&](int i0) {
#pragma unroll
    for (int z = 0; z < kBatch; ++z) {
      int k, w;
      const int h = row_of(i0 + z * kRows, &k, &w);
      if (h < 0) continue;
      const Rows& r = w ? a.in[1] : a.in[0];
      const uint4* from = reinterpret_cast<const uint4*>(r.data + s_at[w][k] + h * r.head);
      x[z] = from[c0];
      y[z] = from[c1];
    }
  };
  const int step = kRows * kBatch * shares;
  int i0 = threadIdx.x / kUnits + blockIdx.y * (kRows * kBatch);
  load(i0);
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int k = i / pairs;
    if (s_there[k]) s_cs[k][i % pairs] = angle_of(a.rope, i % pairs, s_pos[k]);
  }
  __syncthreads();
  for (; i0 < total; i0 += step) {
#pragma unroll
    for (int z = 0; z < kBatch; ++z) {
      int k, w;
      const int h = row_of(i0 + z * kRows, &k, &w);
      if (h < 0) continue;
      if (u < turned) turn<INTERLEAVED>(x[z], y[z], reinterpret_cast<const float4*>(s_cs[k]), c0, c1);
      const Rows& r = w ? a.out[1] : a.out[0];
      uint4* to = reinterpret_cast<uint4*>(r.data + s_at[w + 2][k] + h * r.head);
      to[c0] = x[z];
      to[c1] = y[z];
    }
    if (i0 + step < total) load(i0 + step);
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s) {
  // As many tokens a CTA as give each thread a batch of rows; fewer, and a token's rows over several
  // CTAs, where there are not two CTAs for each SM.
  const long long all = static_cast<long long>(a.S) * a.n;
  const int heads = a.heads[0] + a.heads[1], rows = kThreads / (a.d / 16) * kBatch;
  int tokens = min(max(rows / heads, 1), kTokens);
  while (tokens > 1 && (all + tokens - 1) / tokens * a.L < 2 * a.num_sms) tokens /= 2;
  const long long groups = (all + tokens - 1) / tokens;
  const int batches = (tokens * heads + rows - 1) / rows;
  const int shares = groups * a.L < 2 * a.num_sms ? min(batches, 16) : 1;
  auto* kernel = a.d == 64 ? (a.rope.interleaved ? rotary_kernel<64, true> : rotary_kernel<64, false>)
                           : (a.rope.interleaved ? rotary_kernel<128, true> : rotary_kernel<128, false>);
  return cache8::launch(kernel, dim3(static_cast<unsigned>(groups), shares, a.L), kThreads, 0, s, a,
                        tokens, shares, cache8::make_div(heads));
}

}  // namespace prompt
}  // namespace kvc
