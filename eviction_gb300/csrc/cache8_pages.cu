// cache8_pages.cu -- the block tables of the 8-bit paged cache: reserve blocks
// for new tokens (grow), start sequences from another's cache (fork), give
// sequences up (free).
//
// The tables are a few thousand integers, so their work is latency: one CTA does
// each call, and what counts is how many loads wait for one another.  A thread
// keeps its sequence and its first kKeep table entries in registers from the checks
// to the writes; entries past those (of calls over kKeep * 1024) are read again.  A
// call either does everything or changes nothing, so every index is checked before
// the first write that cannot be taken back.  The order in which blocks leave and
// enter the stack is fixed (list order, then block order), which makes the tables
// reproducible: counts go through atomics, whose order does not matter for
// integers, and places come from prefix sums.
//
// fork copies the rows of the started blocks in a second launch over all layers,
// which skips its work when the first one refused.
//
// Measured: freeing 64 sequences of 100 to 1112 tokens and growing 64 new ones 14 us (39 us
// with a scan and a search for every step over the entries).
#include "cache8.cuh"

namespace kvc {
namespace cache8 {
namespace {

constexpr int kThreads = 1024;
constexpr int kSeqs = kThreads;  // sequences of one pass over the list

// Inclusive scan over the CTA (kThreads threads); every thread gets the total too.
__device__ int block_scan(int v, int* total) {
  __shared__ int sums[kThreads / 32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  if (lane == 31) sums[warp] = v;
  __syncthreads();
  int w = sums[lane];  // kThreads / 32 = 32 warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += t;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, (warp + 31) % 32);
  __syncthreads();
  return v + (warp ? before : 0);
}

// The sequence of the pass that entry e belongs to: the first whose end is past e.
__device__ __forceinline__ int owner(const int* ends, int n, int e) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (ends[mid] > e) hi = mid; else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ int blocks_for(int tokens, int bs) {
  return tokens / bs + (tokens % bs ? 1 : 0);
}

constexpr int kKeep = 4;  // table entries a thread keeps

// Where entry e (of all lists of a pass, one after another) lies: list k of those
// that end at ends[], place col in it.
struct Place {
  int k, col;
};
__device__ __forceinline__ Place place_of(const int* ends, int e) {
  const int k = owner(ends, kSeqs, e);
  return {k, e - (k ? ends[k - 1] : 0)};
}

// ---- grow ----

__global__ void __launch_bounds__(kThreads, 1) grow_kernel(Cache c, const int32_t* n_new) {
  __shared__ int ends[kSeqs], have[kSeqs];
  const int t = threadIdx.x;
  before_all();
  const int top = *c.free_top;
  bool bad = top < 0 || top > c.n_blocks;
  long long need_all = 0;  // of this thread's sequences
  int len = 0, n = 0;      // of its first one
  for (int b = t; b < c.B; b += kThreads) {
    const int bl = length_of(c, b, &bad), bn = n_new[b];
    if (b == t) len = bl, n = bn;
    if (bn < 0 || static_cast<long long>(bl) + bn > static_cast<long long>(c.max_blocks) * c.bs) {
      bad = true;
      continue;
    }
    need_all += blocks_for(bl + bn, c.bs) - blocks_for(bl, c.bs);
    if (bn > 0 && bl % c.bs) {  // the started block has to be this sequence's alone
      const int blk = block_at(c, b, bl / c.bs);
      bad = bad || blk < 0 || c.ref_count[blk] != 1;
    }
  }
  const bool any_bad = __syncthreads_or(bad);
  // a sum of needs can pass 2^31: each capped above the stack's size, then in halves
  const int mine = static_cast<int>(min(need_all, static_cast<long long>(c.n_blocks) + 1));
  int lo_total, hi_total;
  block_scan(mine & 0xffff, &lo_total);
  block_scan(mine >> 16, &hi_total);
  const long long all = (static_cast<long long>(hi_total) << 16) + lo_total;
  if (any_bad || all > top) {
    if (t == 0) atomicOr(c.status, any_bad ? KVC_STATUS_BAD_INDEX : KVC_STATUS_POOL_EXHAUSTED);
    return;  // the same for every thread
  }
  const int base = top - static_cast<int>(all);
  // what the stack gives has to be blocks that nobody holds
  int taken[kKeep];
  bad = false;
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int e = t + i * kThreads;
    taken[i] = e < all ? c.free_list[base + e] : -1;
  }
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    if (t + i * kThreads < all)
      bad = bad || taken[i] < 0 || taken[i] >= c.n_blocks || c.ref_count[taken[i]] != 0;
  }
  for (int e = t + kKeep * kThreads; e < all; e += kThreads) {
    const int blk = c.free_list[base + e];
    bad = bad || blk < 0 || blk >= c.n_blocks || c.ref_count[blk] != 0;
  }
  if (__syncthreads_or(bad)) {
    if (t == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  int from = 0;
  for (int b0 = 0; b0 < c.B; b0 += kSeqs) {
    const int b = b0 + t;
    if (b0 > 0) {
      len = b < c.B ? c.seq_len[b] : 0;
      n = b < c.B ? n_new[b] : 0;
    }
    have[t] = blocks_for(len, c.bs);
    int total;
    ends[t] = block_scan(blocks_for(len + n, c.bs) - have[t], &total);
    if (n) c.seq_len[b] = len + n;
    __syncthreads();
    auto give = [&](int e, int blk) {
      const Place p = place_of(ends, e);
      c.table[static_cast<size_t>(b0 + p.k) * c.max_blocks + have[p.k] + p.col] = blk;
      c.ref_count[blk] = 1;
    };
    if (b0 == 0) {
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if (t + i * kThreads < total) give(t + i * kThreads, taken[i]);
    }
    for (int e = b0 == 0 ? t + kKeep * kThreads : t; e < total; e += kThreads)
      give(e, c.free_list[base + from + e]);
    from += total;
    __syncthreads();
  }
  if (t == 0) *c.free_top = base;
}

// ---- free ----

constexpr int kMarkBits = 1 << 16;  // sequences that the marks in shared memory cover

// Whether a sequence number is listed twice, or is in `others` too (may be null).
// Whole CTA; the numbers are in range.
__device__ bool listed_twice(const Cache& c, int n, const int32_t* seqs, const int32_t* others,
                             uint32_t* marks) {
  bool twice = false;
  for (int base = 0; base < c.B; base += kMarkBits) {
    const int words = (min(c.B - base, kMarkBits) + 31) / 32;
    for (int i = threadIdx.x; i < words; i += kThreads) marks[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const int s = seqs[i] - base;
      if (s >= 0 && s < kMarkBits)
        twice = (atomicOr(&marks[s / 32], 1u << (s % 32)) >> (s % 32) & 1u) || twice;
    }
    __syncthreads();
    for (int i = threadIdx.x; others && i < n; i += kThreads) {
      const int s = others[i] - base;
      if (s >= 0 && s < kMarkBits) twice = (marks[s / 32] >> (s % 32) & 1u) || twice;
    }
    __syncthreads();
  }
  return __syncthreads_or(twice);
}

// Calls f(key, entry) for every table entry of the listed sequences; keys ascend with
// list and block order, and are -1 for a thread without an entry.  Whole CTA; `ends`
// is scratch of kSeqs ints.
template <class F>
__device__ void for_entries(const Cache& c, int n, const int32_t* seqs, int* ends, F f) {
  for (int i0 = 0; i0 < n; i0 += kSeqs) {
    const int i = i0 + threadIdx.x;
    const int held = i < n ? blocks_for(c.seq_len[seqs[i]], c.bs) : 0;
    int total;
    __syncthreads();
    ends[threadIdx.x] = block_scan(held, &total);
    __syncthreads();
    for (int e0 = 0; e0 < total; e0 += kThreads) {
      // (f may hold barriers: every thread calls it, at one place)
      int key = -1;
      int32_t* at = nullptr;
      if (e0 + static_cast<int>(threadIdx.x) < total) {
        const Place p = place_of(ends, e0 + threadIdx.x);
        key = (i0 + p.k) * c.max_blocks + p.col;
        at = c.table + static_cast<size_t>(seqs[i0 + p.k]) * c.max_blocks + p.col;
      }
      f(key, at);
    }
  }
  __syncthreads();
}

// Any number of sequences and entries; the entries are read again in each step.
__device__ __noinline__ void free_many(const Cache& c, int n, const int32_t* seqs, int* ends,
                                       uint32_t* marks) {
  const int t = threadIdx.x;
  const int top = *c.free_top;
  bool bad = top < 0 || top > c.n_blocks;
  for (int i = t; i < n; i += kThreads) {
    const int s = seqs[i];
    if (s < 0 || s >= c.B)
      bad = true;
    else
      length_of(c, s, &bad);
  }
  if (__syncthreads_or(bad) || listed_twice(c, n, seqs, nullptr, marks)) {
    if (t == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
    if (key >= 0) bad = bad || *at < 0 || *at >= c.n_blocks;
  });
  if (__syncthreads_or(bad)) {
    if (t == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
    if (key >= 0) bad = atomicSub(&c.ref_count[*at], 1) < 1 || bad;
  });
  auto put_back = [&] {
    for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
      if (key >= 0) atomicAdd(&c.ref_count[*at], 1);
    });
    if (t == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
  };
  if (__syncthreads_or(bad)) {
    put_back();
    return;
  }
  // a block that nobody holds: its count becomes -1 - (its last key in the list)
  for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
    if (key >= 0 && __ldcg(&c.ref_count[*at]) <= 0) atomicMin(&c.ref_count[*at], -1 - key);
  });
  int mine = 0, all;
  for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
    if (key >= 0) mine += __ldcg(&c.ref_count[*at]) == -1 - key;
  });
  block_scan(mine, &all);
  if (all > c.n_blocks - top) {  // more blocks than there are: the stack was wrong
    for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
      if (key >= 0 && __ldcg(&c.ref_count[*at]) < 0) c.ref_count[*at] = 0;
    });
    put_back();
    return;
  }
  int to = top;
  for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
    const bool push = key >= 0 && __ldcg(&c.ref_count[*at]) == -1 - key;
    int total;
    const int place = to + block_scan(push, &total) - 1;
    if (push) c.free_list[place] = *at;
    to += total;
  });
  for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
    if (key < 0) return;
    if (__ldcg(&c.ref_count[*at]) < 0) c.ref_count[*at] = 0;
    *at = -1;
  });
  for (int i = t; i < n; i += kThreads) c.seq_len[seqs[i]] = 0;
  if (t == 0) *c.free_top = to;
}

__global__ void __launch_bounds__(kThreads, 1) free_kernel(Cache c, int n, const int32_t* seqs) {
  __shared__ int ends[kSeqs], numbers[kSeqs];
  __shared__ uint32_t marks[kMarkBits / 32];
  before_all();
  if (n > kSeqs || c.B > kMarkBits) {
    free_many(c, n, seqs, ends, marks);
    return;
  }
  // one thread, one sequence; then one thread, up to kKeep entries, in registers
  const int t = threadIdx.x;
  const int s = t < n ? seqs[t] : 0;
  const int top = *c.free_top;
  for (int i = t; i < (c.B + 31) / 32; i += kThreads) marks[i] = 0;
  bool bad = top < 0 || top > c.n_blocks || s < 0 || s >= c.B;
  const int len = t < n && !bad ? length_of(c, s, &bad) : 0;
  numbers[t] = s;
  __syncthreads();
  if (t < n && !bad) bad = atomicOr(&marks[s / 32], 1u << (s % 32)) >> (s % 32) & 1u;
  int total;
  ends[t] = block_scan(blocks_for(len, c.bs), &total);
  if (__syncthreads_or(bad)) {
    if (t == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  if (total > kKeep * kThreads) {
    __syncthreads();
    free_many(c, n, seqs, ends, marks);
    return;
  }
  int at[kKeep], key[kKeep], blk[kKeep], was[kKeep];
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    key[i] = -1;
    if (t + i * kThreads < total) {
      const Place p = place_of(ends, t + i * kThreads);
      at[i] = numbers[p.k] * c.max_blocks + p.col;  // below 2^31: checked on the host
      key[i] = p.k * c.max_blocks + p.col;
      blk[i] = c.table[at[i]];
    }
  }
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (key[i] >= 0) bad = bad || blk[i] < 0 || blk[i] >= c.n_blocks;
  if (__syncthreads_or(bad)) {
    if (t == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  // one holder fewer; the count before says whether the block is free now (1), was
  // shared (more), or had more holders than were counted (less)
  bool shared = false;
#pragma unroll
  for (int i = 0; i < kKeep; ++i) was[i] = key[i] >= 0 ? atomicSub(&c.ref_count[blk[i]], 1) : 2;
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    bad = bad || was[i] < 1;
    shared = shared || (key[i] >= 0 && was[i] > 1);
  }
  bad = __syncthreads_or(bad);
  // An entry whose block nobody holds now pushes it: the last one in the list, where
  // several of the list shared it (an entry that saw a count above 1 knows).
  if (!bad && __syncthreads_or(shared)) {
    bool twice = false;
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (key[i] >= 0 && was[i] > 1) twice = twice || __ldcg(&c.ref_count[blk[i]]) == 0;
    if (__syncthreads_or(twice)) {
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if (key[i] >= 0 && __ldcg(&c.ref_count[blk[i]]) <= 0) atomicMin(&c.ref_count[blk[i]], -1 - key[i]);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if (key[i] >= 0) was[i] = __ldcg(&c.ref_count[blk[i]]) == -1 - key[i] ? 1 : 2;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kKeep; ++i)
        if (was[i] == 1) c.ref_count[blk[i]] = 0;
      __syncthreads();
    }
  }
  // places on the stack: entries i * kThreads + t in this order, two counts at a time
  int push[kKeep], place[kKeep], all = 0;
#pragma unroll
  for (int i = 0; i < kKeep; ++i) push[i] = key[i] >= 0 && was[i] == 1;
#pragma unroll
  for (int i = 0; i < kKeep; i += 2) {
    int both;
    const int incl = block_scan(push[i] | push[i + 1] << 16, &both);
    place[i] = all + (incl & 0xffff) - 1;
    all += both & 0xffff;
    place[i + 1] = all + (incl >> 16) - 1;
    all += both >> 16;
  }
  if (bad || all > c.n_blocks - top) {  // a stack with more blocks than there are was wrong
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (key[i] >= 0) atomicAdd(&c.ref_count[blk[i]], 1);
    if (t == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    return;
  }
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    if (push[i]) c.free_list[top + place[i]] = blk[i];
    if (key[i] >= 0) c.table[at[i]] = -1;
  }
  if (t < n) c.seq_len[s] = 0;
  if (t == 0) *c.free_top = top + all;
}

// ---- fork ----

__global__ void __launch_bounds__(kThreads, 1)
    fork_kernel(Cache c, int n, const int32_t* src, const int32_t* dst) {
  __shared__ int ends[kSeqs], part[kSeqs];
  __shared__ uint32_t marks[kMarkBits / 32];
  const int t = threadIdx.x;
  before_all();
  if (t == 0) *c.err = 0;
  const int top = *c.free_top;
  bool bad = top < 0 || top > c.n_blocks;
  int started = 0, first_len = 0;
  for (int i = t; i < n; i += kThreads) {
    const int s = src[i], d = dst[i];
    if (s < 0 || s >= c.B || d < 0 || d >= c.B) {
      bad = true;
      continue;
    }
    const int len = length_of(c, s, &bad);
    if (i == t) first_len = len;
    started += len % c.bs ? 1 : 0;
    bad = bad || c.seq_len[d] != 0;
  }
  int all;
  block_scan(started, &all);
  bool full = false;
  // a new sequence listed twice, or also as a source (which can only be an empty one)
  bad = __syncthreads_or(bad);
  if (!bad) bad = listed_twice(c, n, dst, src, marks);
  int kept[kKeep];  // blocks of this thread's first entries
  if (!bad) {
    full = all > top;
    if (!full) {
      for (int e = t; e < all; e += kThreads) {
        const int blk = c.free_list[top - all + e];
        bad = bad || blk < 0 || blk >= c.n_blocks || c.ref_count[blk] != 0;
      }
    }
    for (int i0 = 0; i0 < n; i0 += kSeqs) {
      const int i = i0 + t;
      const int len = i0 == 0 ? first_len : i < n ? c.seq_len[src[i]] : 0;
      int total;
      ends[t] = block_scan(blocks_for(len, c.bs), &total);
      __syncthreads();
      if (i0 == 0) {
#pragma unroll
        for (int k = 0; k < kKeep; ++k) {
          kept[k] = -1;
          if (t + k * kThreads < total) {
            const Place p = place_of(ends, t + k * kThreads);
            kept[k] = block_at(c, src[p.k], p.col);
            bad = bad || kept[k] < 0;
          }
        }
#pragma unroll
        for (int k = 0; k < kKeep; ++k)
          if (kept[k] >= 0) bad = c.ref_count[kept[k]] < 1 || bad;
      }
      for (int e = i0 == 0 ? t + kKeep * kThreads : t; e < total; e += kThreads) {
        const Place p = place_of(ends, e);
        const int blk = block_at(c, src[i0 + p.k], p.col);
        bad = bad || blk < 0 || c.ref_count[blk] < 1;
      }
      __syncthreads();
    }
    bad = __syncthreads_or(bad);
  }
  if (bad || full) {
    if (t == 0) {
      *c.err = bad ? KVC_STATUS_BAD_INDEX : KVC_STATUS_POOL_EXHAUSTED;
      atomicOr(c.status, *c.err);
    }
    return;  // the same for every thread
  }
  int from = top - all;
  for (int i0 = 0; i0 < n; i0 += kSeqs) {
    const int i = i0 + t;
    const int len = i0 == 0 ? first_len : i < n ? c.seq_len[src[i]] : 0;
    int total, fresh;
    ends[t] = block_scan(blocks_for(len, c.bs), &total);
    const int after = block_scan(len % c.bs ? 1 : 0, &fresh);
    part[t] = len % c.bs ? from + after - 1 : -1;  // where the stack has this one's block
    __syncthreads();
    auto give = [&](int e, int blk) {  // entry e: a source's block, or a new one for its started one
      const Place p = place_of(ends, e);
      if (part[p.k] >= 0 && e == ends[p.k] - 1) {
        blk = c.free_list[part[p.k]];
        c.ref_count[blk] = 1;
      } else {
        if (blk < 0) blk = c.table[static_cast<size_t>(src[i0 + p.k]) * c.max_blocks + p.col];
        atomicAdd(&c.ref_count[blk], 1);
      }
      c.table[static_cast<size_t>(dst[i0 + p.k]) * c.max_blocks + p.col] = blk;
    };
    if (i0 == 0) {
#pragma unroll
      for (int k = 0; k < kKeep; ++k)
        if (t + k * kThreads < total) give(t + k * kThreads, kept[k]);
    }
    for (int e = i0 == 0 ? t + kKeep * kThreads : t; e < total; e += kThreads) give(e, -1);
    if (i < n) c.seq_len[dst[i]] = len;  // a dst is never a src
    from += fresh;
    __syncthreads();
  }
  if (t == 0) *c.free_top = top - all;
}

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kCopyCtas = 6;  // of an SM

// One CTA: the started block of one new sequence in some layers, all heads, keys and
// values.  Finding the blocks takes four loads that wait for one another: each CTA has
// so many layers that all CTAs are resident at once.  (64 sequences, 28 layers, started
// blocks of 32 rows on average, with the two launches before it: 32 us; 38 at 3 CTAs of
// 8 loads a thread, 46 with a CTA for each layer.)
__global__ void __launch_bounds__(kCopyThreads, kCopyCtas)
    fork_copy_kernel(Cache c, int layers, const int32_t* src, const int32_t* dst) {
  before_all();
  const int s = src[blockIdx.x], d = dst[blockIdx.x];
  if (*c.err) return;  // refused: the numbers may be out of range
  const int len = c.seq_len[d];
  const int rows = len % c.bs;
  if (rows == 0) return;
  const int from = block_at(c, s, len / c.bs), to = block_at(c, d, len / c.bs);
  if (from < 0 || to < 0) return;
  const int vec = c.d / 16, head = rows * vec;  // 16-byte vectors of a row, of a head's rows
  const int stride = c.bs * vec;
  const int l0 = blockIdx.y * layers, l1 = min(c.L, l0 + layers);
  for (int l = l0; l < l1; ++l) {
    const size_t x0 = block_row(c, l, from, 0) * vec, y0 = block_row(c, l, to, 0) * vec;
    for (int i = threadIdx.x; i < head; i += kCopyThreads) {
      for (int k0 = 0; k0 < 2 * c.H; k0 += kCopyUnroll) {
        uint4 v[kCopyUnroll];
  #pragma unroll
        for (int k = 0; k < kCopyUnroll; ++k) {
          const int hk = k0 + k, hh = hk < c.H ? hk : hk - c.H;
          const uint4* pool = reinterpret_cast<const uint4*>(hk < c.H ? c.pool[0] : c.pool[1]);
          if (hk < 2 * c.H) v[k] = pool[x0 + hh * stride + i];
        }
  #pragma unroll
        for (int k = 0; k < kCopyUnroll; ++k) {
          const int hk = k0 + k, hh = hk < c.H ? hk : hk - c.H;
          uint4* pool = reinterpret_cast<uint4*>(hk < c.H ? c.pool[0] : c.pool[1]);
          if (hk < 2 * c.H) pool[y0 + hh * stride + i] = v[k];
        }
      }
    }
    for (int i = threadIdx.x; i < 2 * c.H; i += kCopyThreads) {
      float* scale = i < c.H ? c.scale[0] : c.scale[1];
      scale[scale_at(c, l, to, i % c.H)] = scale[scale_at(c, l, from, i % c.H)];
    }
  }
}

}  // namespace

cudaError_t launch_grow(const Cache& c, const int32_t* n_new, cudaStream_t s) {
  return launch(grow_kernel, 1, kThreads, 0, s, c, n_new);
}

cudaError_t launch_free(const Cache& c, int n, const int32_t* seqs, cudaStream_t s) {
  return launch(free_kernel, 1, kThreads, 0, s, c, n, seqs);
}

cudaError_t launch_fork(const Cache& c, int n, const int32_t* src, const int32_t* dst,
                        int num_sms, cudaStream_t s) {
  const cudaError_t e = launch(fork_kernel, 1, kThreads, 0, s, c, n, src, dst);
  if (e != cudaSuccess) return e;
  // as many CTAs as are resident at once, and gridDim.y is at most 65535
  const long long share = static_cast<long long>(n) * c.L / (kCopyCtas * num_sms);
  const int layers = static_cast<int>(max(max(share, static_cast<long long>(c.L) / 65535 + 1), 1ll));
  return launch(fork_copy_kernel, dim3(n, (c.L + layers - 1) / layers), kCopyThreads, 0, s, c, layers,
                src, dst);
}

}  // namespace cache8
}  // namespace kvc
