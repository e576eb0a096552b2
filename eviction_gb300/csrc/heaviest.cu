// heaviest.cu -- the tokens that an eviction by gathered weight keeps (kvc_keep_heaviest):
// per unit the last and the first tokens and the heaviest of the others, in order.
//
// One CTA a unit.  The least weight that is kept is found by a radix select over
// order-preserving 32-bit keys: a histogram of a digit of 11 bits in shared memory, and the bin
// that the wanted rank falls into.  The first digit starts at the highest bit in which the unit's
// keys differ (a minimum and a maximum), so that it tells them apart: with the sign and all of the
// exponent in it most keys of a warp would add to a few bins.  What is left after it, a few percent,
// goes to a list, whose keys are ranked by comparing each with each, or by further digits where
// they are many.  Keys above the least one are kept, and of those equal to it the first ones.
// (For 64 x 8 units of 1112 tokens and 28 x 8 x 4 of 1536, with two more digits over all keys
// instead of the list: 9.6 and 16 us, of 7.0 and 12; with a first digit of 8 bits, which leaves too
// many to rank: 10 and 20.)
//
// The call reads weights once and writes them, and the budget's positions, once; instructions on
// registers and on shared memory bound it, a scan, a digit and a ranking deep.  Measured: 6.0 us for
// 64 x 8 x 1112 -> 512, 8.8 us for 28 x 8 x 4 x 1536 -> 1024, 56 us for 28 x 4 x 4 x 32768 -> 4096
// (125 MB; the choice 17 us of them, places 6, what is kept 5, the zeros behind it 10, by stores or by
// bulk copies).  A CTA that takes units in turns with the next one's weights on their way to shared
// memory took 85 us there.  Kernel, rounds and threads go by cap, which the host knows, not by the
// lengths: 28 x 8 x 4 x 1536 -> 1024 in rows of 8192 takes 24 us, of 32768 92 us.
//
// Weights are read once and stay in registers, as keys: thread i has elements 4 (r NT + i) .. + 3 of
// round r (at 64 registers, for 8 rounds, 28 bytes a thread spill).  Places come from one scan of
// the counts, a byte a round, over the warp and one over the warps.  All of a unit is read before any
// of it is written, so that weights_out may be weights.  Units that registers do not hold (over 32768
// tokens) are read again for each digit, from L2 (16 units of 32768: 42 us, of 65536: 79 us).
#include "prompt.cuh"

namespace kvc {
namespace prompt {
namespace {

using cache8::before_all;

constexpr int kBits = 11, kBins = 1 << kBits;
constexpr int kMaxRounds = 8;
constexpr int kListed = 2048;  // keys that are left after the first digit, in shared memory
constexpr int kRanked = 256;   // of them, that are compared each with each

// Larger weight, larger key; NaN below all, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float w) {
  return w == w ? float_order_key(w + 0.f) : 0u;
}

// The weight of a key (any NaN for a NaN, 0 for -0).
__device__ __forceinline__ float weight_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// Without a branch around them (a branch for each element is as long as what it skips): add to a
// counter in shared memory, store to the places `at` of two arrays.
__device__ __forceinline__ void count_if(bool p, int* counter) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t@p red.shared.add.u32 [%0], 1;\n\t}" ::"r"(
                   smem_u32(counter)),
               "r"(static_cast<int>(p))
               : "memory");
}
__device__ __forceinline__ void list_if(bool p, int* counter, uint32_t* list, uint32_t key) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 n;\n\tsetp.ne.b32 p, %3, 0;\n\t"
      "@p atom.shared.add.u32 n, [%0], 1;\n\t@p mad.lo.u32 n, n, 4, %1;\n\t@p st.shared.b32 [n], %2;\n\t}" ::"r"(
          smem_u32(counter)),
      "r"(smem_u32(list)), "r"(key), "r"(static_cast<int>(p))
      : "memory");
}
__device__ __forceinline__ void store_if(bool p, int32_t* a, int x, float* b, uint32_t y) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "@p st.global.b32 [%0], %1;\n\t@p st.global.b32 [%2], %3;\n\t}" ::"l"(a),
      "r"(x), "l"(b), "r"(y), "r"(static_cast<int>(p))
      : "memory");
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
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  // (every warp sums the others up for itself)
  const int w = lane < warps ? s_warp[lane] : 0;
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
  *all = __reduce_add_sync(0xffffffffu, w);
  __syncthreads();
  return before + incl - v;
}

struct __align__(16) Shared {
  int hist[kBins];
  int warp[32];
  uint32_t low[32], high[32];
  int rounds[kMaxRounds * 32];
  uint32_t list[kListed];
  uint32_t prefix;
  int want, same, listed, ranked_want;
};

// The least and the largest of the CTA's values.  A barrier inside, and one owed before the next call.
__device__ __forceinline__ void range(Shared& s, uint32_t& low, uint32_t& high) {
  const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) s.low[threadIdx.x / 32] = low, s.high[threadIdx.x / 32] = high;
  __syncthreads();
  low = __reduce_min_sync(0xffffffffu, lane < warps ? s.low[lane] : 0xffffffffu);
  high = __reduce_max_sync(0xffffffffu, lane < warps ? s.high[lane] : 0u);
}

// Of the CTA's keys, which each(f) calls f with (and with zeros, which are none), all of them
// between low and high, and with s.hist zero: the want-th largest (want >= 1, there are as many) in
// *least, how many keys equal to it belong to the want largest, and how many there are.
template <class Each>
__device__ __forceinline__ void select(Shared& s, Each each, uint32_t low, uint32_t high, int want,
                                       uint32_t* least, int* equal, int* same) {
  uint32_t so_far = high;             // the bits above `rest` are the least key's
  int rest = 32 - __clz(low ^ high);  // bits that are not known yet
  *same = 0;
  // the bin of the digit at `shift`, of `bits` bits, that the want-th key falls into
  auto settle = [&](int shift, int bits) {
    __syncthreads();
    // thread i: the bins from mask - i per down, heaviest first
    const int mask = (1 << bits) - 1;
    const int per = (mask + blockDim.x) / blockDim.x, first = mask - static_cast<int>(threadIdx.x) * per;
    int mine = 0, all;
    for (int i = 0; i < per && first - i >= 0; ++i) mine += s.hist[first - i];
    int above = prefix(mine, s.warp, &all);
    if (above < want && above + mine >= want) {
      int bin = first;
      while (above + s.hist[bin] < want) above += s.hist[bin--];
      const uint32_t known = shift + bits == 32 ? 0u : so_far >> (shift + bits) << (shift + bits);
      s.prefix = known | static_cast<uint32_t>(bin) << shift;
      s.want = want - above;
      s.same = s.hist[bin];
      s.listed = 0;
    }
    __syncthreads();
    so_far = s.prefix;
    want = s.want;
    *same = s.same;
    rest = shift;
  };
  if (rest > 0) {
    const int bits = min(rest, kBits), shift = rest - bits;
    const uint32_t mask = (1u << bits) - 1;
    each([&](uint32_t k) { count_if(k != 0, &s.hist[(k >> shift) & mask]); });
    settle(shift, bits);
  }
  // What is left is few keys most often: they are listed, and ranked among one another if they
  // are a few for each lane of a warp.
  const bool list = rest > 0 && *same <= kListed;
  const int n = *same;
  if (list) {
    each([&](uint32_t k) { list_if(k >> rest == so_far >> rest && k != 0, &s.listed, s.list, k); });
    __syncthreads();
    if (n <= kRanked) {
      for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const uint32_t k = s.list[i];
        int more = 0, alike = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
          const uint32_t other = s.list[j];
          more += other > k;
          alike += other == k;
        }
        if (more < want && more + alike >= want) {  // (all that are equal to it write the same)
          s.prefix = k;
          s.ranked_want = want - more;
          s.same = alike;
        }
      }
      __syncthreads();
      *least = s.prefix;
      *equal = s.ranked_want;
      *same = s.same;
      return;
    }
  }
  while (rest > 0) {
    for (int i = threadIdx.x; i < kBins; i += blockDim.x) s.hist[i] = 0;
    __syncthreads();
    const int bits = min(rest, kBits), shift = rest - bits;
    const uint32_t mask = (1u << bits) - 1;
    auto count = [&](uint32_t k) {
      count_if((k ^ so_far) >> shift <= mask && k != 0, &s.hist[(k >> shift) & mask]);
    };
    if (list)
      for (int i = threadIdx.x; i < n; i += blockDim.x) count(s.list[i]);
    else
      each(count);
    settle(shift, bits);
  }
  *least = so_far;
  *equal = want;
}

// Zeros behind the kept weights, -1 behind the kept positions, the count.
__device__ __forceinline__ void write_rest(const HeaviestArgs& a, const Plan& p, int u, int32_t* kept,
                                           float* out) {
  for (int i = p.n + threadIdx.x; i < a.budget; i += blockDim.x) kept[i] = -1;
  int i = p.n;
  const int head = static_cast<int>(-(reinterpret_cast<uintptr_t>(out + i) >> 2) & 3);  // to a 16-byte boundary
  const int start = min(i + head, a.cap), wide = (a.cap - start) / 4;
  if (threadIdx.x < start - i) out[i + threadIdx.x] = 0.f;
  for (int k = threadIdx.x; k < wide; k += blockDim.x)
    reinterpret_cast<float4*>(out + start)[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  i = start + 4 * wide + threadIdx.x;
  if (i < a.cap) out[i] = 0.f;
  if (threadIdx.x == 0) a.n_kept[u] = p.n;
}

// Units of at most 4 R blockDim.x tokens.  Keys are above 0; 0 stands for what is kept anyway, or
// not there.  Where no weight is negative or NaN, as sums of softmax weights are, a weight's bits
// are its order and its key is these plus one: nothing to convert.
template <int R, int MaxThreads, int MinCtas>
__global__ void __launch_bounds__(MaxThreads, MinCtas) heaviest_kernel(HeaviestArgs a) {
  __shared__ Shared s;
  before_all();
  const int u = blockIdx.x, b = (u / a.H) % a.B;
  const Plan p = plan_of(a, b);
  if (p.bad) {
    if (threadIdx.x == 0) atomicOr(a.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  const float* w = a.w + static_cast<size_t>(u) * a.cap;
  const int NT = blockDim.x, lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = NT / 32;
  auto index = [&](int r) { return 4 * (r * NT + static_cast<int>(threadIdx.x)); };
  uint32_t x[R][4];  // weights' bits, then keys
  const bool wide = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int t = index(r);
    if (wide && t + 4 <= p.len) {
      const uint4 v = *reinterpret_cast<const uint4*>(w + t);
      x[r][0] = v.x, x[r][1] = v.y, x[r][2] = v.z, x[r][3] = v.w;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[r][c] = t + c < p.len ? __float_as_uint(w[t + c]) : 0u;
    }
  }
  // (what does not depend on the choice is written while the weights are on their way, unless
  // it lies in their place)
  int32_t* kept = a.kept + static_cast<size_t>(u) * a.budget;
  float* out = a.out + static_cast<size_t>(u) * a.cap;
  if (out != w) write_rest(a, p, u, kept, out);
  for (int i = threadIdx.x; i < kBins; i += NT) s.hist[i] = 0;
  auto limits = [&](uint32_t& low, uint32_t& high) {  // of the keys (a zero less one is no minimum)
    low = 0xffffffffu, high = 0;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) low = min(low, x[r][c] - 1), high = max(high, x[r][c]);
    range(s, low, high);
    ++low;
  };
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int t0 = 4 * (r * NT + 32 * warp);  // the warp's elements are 128 from here on
    if (t0 >= p.head && t0 + 128 <= p.tail) {
#pragma unroll
      for (int c = 0; c < 4; ++c) x[r][c] = min(x[r][c], 0xfffffffeu) + 1;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        x[r][c] = index(r) + c >= p.head && index(r) + c < p.tail ? min(x[r][c], 0xfffffffeu) + 1 : 0u;
    }
  }
  uint32_t low, high;
  limits(low, high);
  const bool plain = high <= 0x7f800001u;  // (so for all threads)
  if (!plain) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (x[r][c]) x[r][c] = key_of(__uint_as_float(x[r][c] - 1)) + 1;
    __syncthreads();
    limits(low, high);
  }
  // ---- the least key that is kept (all of them: 1) ----
  uint32_t least = p.want > 0 ? 1u : 0xffffffffu;
  int equal = 0, same = 0;
  if (p.want > 0 && p.want < p.tail - p.head) {
    auto each = [&](auto f) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) f(x[r][c]);
    };
    select(s, each, low, high, p.want, &least, &equal, &same);
    if (same == 0) same = p.tail - p.head;  // (all keys are the same one)
  }
  // Places of flagged elements, a nibble of flags a round: the number of those before a
  // thread's own in round r, for all r.
  uint32_t flags = 0;
  int base[R];
  auto places = [&]() {
    uint64_t counts = 0;
#pragma unroll
    for (int r = 0; r < R; ++r)
      counts |= static_cast<uint64_t>(__popc(flags >> (4 * r) & 15)) << (8 * r);
    uint64_t incl = counts;  // (a warp's count in a round is at most 128: a byte holds it)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) {
#pragma unroll
      for (int r = 0; r < R; ++r) s.rounds[r * warps + warp] = static_cast<int>(incl >> (8 * r) & 255);
    }
    __syncthreads();
    int before = 0;  // rounds before
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int v = lane < warps ? s.rounds[r * warps + lane] : 0;
      base[r] = before + __reduce_add_sync(0xffffffffu, lane < warp ? v : 0) +
                static_cast<int>((incl - counts) >> (8 * r) & 255);
      before += __reduce_add_sync(0xffffffffu, v);
    }
    __syncthreads();
  };
  if (same == equal) {  // all that are equal to the least one
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (x[r][c] >= least) flags |= 1u << (4 * r + c);
  } else {  // the first ones (the same branch for all threads: same and equal are)
    uint32_t more = 0;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (x[r][c] > least) more |= 1u << (4 * r + c);
        if (x[r][c] == least) flags |= 1u << (4 * r + c);
      }
    places();
    const uint32_t ties = flags;
    flags = more;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      int rank = base[r];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t bit = ties & 1u << (4 * r + c);
        if (bit && rank < equal) flags |= bit;
        rank += bit != 0;
      }
    }
  }
  places();  // (all weights of others are read)
  if (!plain) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) x[r][c] = __float_as_uint(weight_of(x[r][c] - 1)) + 1;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    int at = p.head + base[r];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bool keep = flags & 1u << (4 * r + c);
      store_if(keep, kept + at, index(r) + c, out + at, x[r][c] - 1);
      at += keep;
    }
  }
  // The first tokens stay in their places.  The last ones move towards the front, behind the
  // others' places; where weights_out is weights, a chunk is read before it is written.
  for (int t = threadIdx.x; t < p.head; t += NT) {
    kept[t] = t;
    if (out != w) out[t] = w[t];
  }
  const int last = p.len - p.tail;
  for (int t = threadIdx.x; t < last; t += NT) kept[p.n - last + t] = p.tail + t;
  if (out != w) {
    for (int t = threadIdx.x; t < last; t += NT) out[p.n - last + t] = w[p.tail + t];
  } else if (p.n < p.len) {
    for (int t0 = 0; t0 < last; t0 += NT) {
      const int t = t0 + threadIdx.x;
      const float v = t < last ? w[p.tail + t] : 0.f;
      __syncthreads();
      if (t < last) out[p.n - last + t] = v;
    }
    __syncthreads();
  }
  if (out == w) write_rest(a, p, u, kept, out);
}

// Units of any length.
constexpr int kStreamThreads = 1024;
__global__ void __launch_bounds__(kStreamThreads) heaviest_stream_kernel(HeaviestArgs a) {
  __shared__ Shared s;
  before_all();
  const int u = blockIdx.x, b = (u / a.H) % a.B;
  const Plan p = plan_of(a, b);
  if (p.bad) {
    if (threadIdx.x == 0) atomicOr(a.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  const float* w = a.w + static_cast<size_t>(u) * a.cap;
  uint32_t least = 0;
  int equal = 0, same = 0;
  if (p.want > 0) {
    auto each = [&](auto f) {
#pragma unroll 4
      for (int t = p.head + threadIdx.x; t < p.tail; t += kStreamThreads) f(key_of(w[t]) + 1);
    };
    uint32_t low = 0xffffffffu, high = 0;
    each([&](uint32_t k) {
      low = min(low, k);
      high = max(high, k);
    });
    for (int i = threadIdx.x; i < kBins; i += kStreamThreads) s.hist[i] = 0;
    range(s, low, high);
    select(s, each, low, high, p.want, &least, &equal, &same);
  }
  // (where weights_out is weights: a chunk is read before what it keeps is written, to
  // places that are not behind it)
  int32_t* kept = a.kept + static_cast<size_t>(u) * a.budget;
  float* out = a.out + static_cast<size_t>(u) * a.cap;
  int done = 0, equals = 0;
  for (int t0 = 0; t0 < p.len; t0 += kStreamThreads) {
    const int t = t0 + threadIdx.x;
    const float x = t < p.len ? w[t] : 0.f;
    const uint32_t k = key_of(x) + 1;
    const bool other = t >= p.head && t < p.tail, tie = other && p.want > 0 && k == least;
    int all;
    const int rank = equals + prefix(tie, s.warp, &all);
    equals += all;
    const bool keep = t < p.len && (!other || (p.want > 0 && (k > least || (tie && rank < equal))));
    const int at = done + prefix(keep, s.warp, &all);
    done += all;
    if (keep) {
      kept[at] = t;
      out[at] = x;
    }
  }
  __syncthreads();
  write_rest(a, p, u, kept, out);
}

}  // namespace

cudaError_t launch_heaviest(const HeaviestArgs& a, cudaStream_t s) {
  const int grid = a.L * a.B * a.H;
  auto threads = [&](int rounds) {  // 4 tokens a thread and round
    const int n = (a.cap + 4 * rounds - 1) / (4 * rounds);
    return (n + 31) / 32 * 32;
  };
  // Few registers, so that an SM has several units under way (28 x 8 x 4 units of 1536, 4096 and
  // 8192 tokens: 8.8, 15.2 and 25.7 us, of 12.3, 19.6 and 27.4 without a limit to registers).  The
  // stream kernel takes more than twice as long wherever registers hold a unit (16384 tokens: 70 us
  // and 31, 32768: 132 and 56).
  if (a.cap <= 2048) return cache8::launch(heaviest_kernel<2, 256, 5>, grid, threads(2), 0, s, a);
  if (a.cap <= 8192) return cache8::launch(heaviest_kernel<4, 512, 3>, grid, threads(4), 0, s, a);
  if (a.cap <= 32768) return cache8::launch(heaviest_kernel<8, 1024, 1>, grid, threads(8), 0, s, a);
  return cache8::launch(heaviest_stream_kernel, grid, kStreamThreads, 0, s, a);
}

}  // namespace prompt
}  // namespace kvc
