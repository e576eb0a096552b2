// rotary.cu -- query and key rows turned by their tokens' positions.
//
// Pair (x, y) of a row goes to (x cos a - y sin a, x sin a + y cos a), a = pos f_i.  The
// frequency is held in turns per token, in 2^-64 of a turn, so that pos * f_i in 64-bit
// integers drops whole turns by itself, where an fp32 product is off by up to 0.06 radians at a
// million tokens.  The top 32 bits, signed, are the angle in half turns, within one: as a float, which
// sincospif takes, it is rounded by up to 2^-25 of a half turn, 2^-23.3 radians, at any position.
//
// The rows are read and written once, which bounds the call: 8 x 4096 tokens of 32 heads of 128,
// 537 MB, take 79 us, 6.8 TB/s.  A CTA has a few tokens and all of their heads: it computes their
// sines and cosines once into shared memory, then each thread turns two 16-byte chunks of a row at
// a time, those that its pairs lie in, of four heads whose sines and cosines it holds (a head at a
// time, with as many reads of shared memory as of the rows: 94 us).
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
constexpr int kBatch = 4;   // heads of a thread whose loads are in flight together

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

// Both chunks of a unit turned, with its eight pairs' (cos, sin): those of chunk c0's values and
// chunk c1's, or of chunk c0 and then of chunk c1.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn(uint4& x, uint4& y, const float4 (&cs)[4]) {
  uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int z = 0; z < 4; ++z) {
    const float2 a = make_float2(cs[z].x, cs[z].y), b = make_float2(cs[z].z, cs[z].w);
    if constexpr (INTERLEAVED) {
      uint32_t* v = z < 2 ? &xs[2 * z] : &ys[2 * z - 4];
      v[0] = turn_pair(v[0], a);
      v[1] = turn_pair(v[1], b);
    } else {
      const uint32_t first = turn_x(xs[z], ys[z], a, b);
      ys[z] = turn_y(xs[z], ys[z], a, b);
      xs[z] = first;
    }
  }
  x = make_uint4(xs[0], xs[1], xs[2], xs[3]);
  y = make_uint4(ys[0], ys[1], ys[2], ys[3]);
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 4) rotary_kernel(const __grid_constant__ RotaryArgs a,
                                                          int tokens, int slots, cache8::Div by_slots) {
  constexpr int kUnits = D / 16;                 // of a row: two 16-byte chunks each
  constexpr int kRows = kThreads / kUnits;       // rows that the CTA's threads take at a time
  __shared__ __align__(16) float4 s_cs[kTokens][4][kUnits];  // two pairs each, of a unit's eight
  __shared__ long long s_at[4][kTokens];         // a token's place in the rows of in, in, out, out
  __shared__ int s_pos[kTokens], s_there[kTokens];
  before_all();
  const long long t0 = static_cast<long long>(blockIdx.x) * tokens, all = static_cast<long long>(a.S) * a.n;
  const int l = blockIdx.y, pairs = a.rope.dim / 2, turned = a.rope.dim / 16;
  if (threadIdx.x < tokens) {
    const long long t = t0 + threadIdx.x;
    int there = t < all, pos = 0;
    if (there) {
      pos = a.pos[t];
      const int b = static_cast<int>(t / a.n), j = static_cast<int>(t % a.n);
      if (a.n_tok) {
        const int m = a.n_tok[b];
        there = j < m && m <= a.n;
        if ((m < 0 || m > a.n) && j == 0 && l == 0)
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
  // This thread: unit u of a token's heads slot, slot + slots, ...: their sines and cosines are
  // the same.  Their loads go out together, the first ones before the angles.
  const int u = threadIdx.x % kUnits, heads = a.heads[0] + a.heads[1], total = tokens * slots;
  // chunks of a turned unit: dim / 2 values apart; of the rest: side by side
  const int c0 = u < turned ? u : 2 * u, c1 = u < turned ? u + turned : 2 * u + 1;
  uint4 x[kBatch], y[kBatch];
  auto row_at = [&](const Rows (&of)[2], int side, int k, int head) {  // null: nothing to do
    const int w = head >= a.heads[0];
    if (head >= heads || (u >= turned && a.in_place[w])) return static_cast<uint4*>(nullptr);
    return reinterpret_cast<uint4*>((w ? of[1].data : of[0].data) + s_at[2 * side + w][k] +
                                    (w ? (head - a.heads[0]) * of[1].head : head * of[0].head));
  };
  auto load = [&](int s) {
    const int k = by_slots.div(s), slot = s - k * slots;
    if (s >= total || !s_there[k]) return;
#pragma unroll
    for (int z = 0; z < kBatch; ++z) {
      const uint4* from = row_at(a.in, 0, k, slot + z * slots);
      if (!from) continue;
      x[z] = from[c0];
      y[z] = from[c1];
    }
  };
  int s = threadIdx.x / kUnits;
  load(s);
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int k = i / pairs, pair = i % pairs;
    if (!s_there[k]) continue;
    // its unit and place there: units have pairs 8 u .. + 7, or those of their two chunks
    int unit = pair / 8, at = pair % 8;
    if constexpr (INTERLEAVED) {
      const int chunk = pair / 4;
      unit = chunk < turned ? chunk : chunk - turned;
      at = pair % 4 + (chunk < turned ? 0 : 4);
    }
    reinterpret_cast<float2*>(&s_cs[k][at / 2][unit])[at % 2] = angle_of(a.rope, pair, s_pos[k]);
  }
  __syncthreads();
  for (; s < total; s += kRows) {
    const int k = by_slots.div(s), slot = s - k * slots;
    if (s_there[k]) {
      float4 cs[4];
#pragma unroll
      for (int z = 0; z < 4; ++z) cs[z] = s_cs[k][z][u];
#pragma unroll
      for (int z = 0; z < kBatch; ++z) {
        uint4* to = row_at(a.out, 1, k, slot + z * slots);
        if (!to) continue;
        if (u < turned) turn<INTERLEAVED>(x[z], y[z], cs);
        to[c0] = x[z];
        to[c1] = y[z];
      }
    }
    load(s + kRows);
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s) {
  // Slots of kBatch heads each; as many tokens a CTA as its threads have slots for, fewer where
  // there are not two CTAs for each SM (64 tokens of 40 heads: 3.9 us, of 4.1 with four a CTA).
  const long long all = static_cast<long long>(a.S) * a.n;
  const int heads = a.heads[0] + a.heads[1], rows = kThreads / (a.d / 16);
  const int slots = (heads + kBatch - 1) / kBatch;
  int tokens = min(max(rows / slots, 1), kTokens);
  while (tokens > 1 && (all + tokens - 1) / tokens * a.L < 2 * a.num_sms) tokens /= 2;
  const long long groups = (all + tokens - 1) / tokens;
  auto* kernel = a.d == 64 ? (a.rope.interleaved ? rotary_kernel<64, true> : rotary_kernel<64, false>)
                           : (a.rope.interleaved ? rotary_kernel<128, true> : rotary_kernel<128, false>);
  return cache8::launch(kernel, dim3(static_cast<unsigned>(groups), a.L), kThreads, 0, s, a,
                        tokens, slots, cache8::make_div(slots));
}

}  // namespace prompt
}  // namespace kvc
