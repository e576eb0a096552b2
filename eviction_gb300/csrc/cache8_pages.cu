// cache8_pages.cu -- the block tables of the 8-bit paged cache: reserve blocks
// for new tokens (grow), start sequences from another's cache (fork), give
// sequences up (free).
//
// The tables are a few thousand integers, so their work is latency: one CTA does
// each call, with its lists in shared memory.  A call either does everything or
// changes nothing, so every index is checked before the first write.  The order in
// which blocks leave and enter the stack is fixed (list order, then block order),
// which makes the tables reproducible: counts go through atomics, whose order
// does not matter for integers, and places come from prefix sums.
//
// fork copies the rows of the started blocks in a second launch over all layers
// and heads, which skips its work when the first one refused.
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

// ---- grow ----

__global__ void __launch_bounds__(kThreads) grow_kernel(Cache c, const int32_t* n_new) {
  __shared__ int ends[kSeqs], have[kSeqs];
  const int t = threadIdx.x;
  const int top = *c.free_top;
  bool bad = top < 0 || top > c.n_blocks;
  long long need_all = 0;  // of this thread's sequences
  for (int b = t; b < c.B; b += kThreads) {
    const int len = length_of(c, b, &bad), n = n_new[b];
    if (n < 0 || static_cast<long long>(len) + n > static_cast<long long>(c.max_blocks) * c.bs) {
      bad = true;
      continue;
    }
    need_all += blocks_for(len + n, c.bs) - blocks_for(len, c.bs);
    if (n > 0 && len % c.bs) {  // the started block has to be this sequence's alone
      const int blk = block_at(c, b, len / c.bs);
      bad = bad || blk < 0 || c.ref_count[blk] != 1;
    }
  }
  // a thread's own need may be larger than the stack: cap it before the int scan
  int need = 0;
  const int mine = static_cast<int>(min(need_all, static_cast<long long>(c.n_blocks) + 1));
  const bool any_bad = __syncthreads_or(bad);
  // the sum of kThreads capped needs can pass 2^31: scan in 64 bits by halves
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
  bad = false;
  for (int e = t; e < static_cast<int>(all); e += kThreads) {
    const int blk = c.free_list[base + e];
    bad = bad || blk < 0 || blk >= c.n_blocks || c.ref_count[blk] != 0;
  }
  if (__syncthreads_or(bad)) {
    if (t == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  int from = base;
  for (int b0 = 0; b0 < c.B; b0 += kSeqs) {
    const int b = b0 + t;
    need = 0;
    if (b < c.B) {
      const int len = c.seq_len[b], n = n_new[b];
      have[t] = blocks_for(len, c.bs);
      need = blocks_for(len + n, c.bs) - have[t];
      if (n) c.seq_len[b] = len + n;
    }
    int total;
    ends[t] = block_scan(need, &total);
    __syncthreads();
    for (int e = t; e < total; e += kThreads) {
      const int i = owner(ends, kSeqs, e);
      const int k = e - (i ? ends[i - 1] : 0);
      const int blk = c.free_list[from + e];
      c.table[static_cast<size_t>(b0 + i) * c.max_blocks + have[i] + k] = blk;
      c.ref_count[blk] = 1;
    }
    from += total;
    __syncthreads();
  }
  if (t == 0) *c.free_top = base;
}

// ---- free ----

// Calls f(key, block) for every table entry of the listed sequences; keys ascend
// with list and block order (-1 for a thread without an entry).  The sequences
// are checked and marked.  Whole CTA; `ends` is scratch of kSeqs ints.
template <class F>
__device__ void for_entries(const Cache& c, int n, const int32_t* seqs, int* ends, F f) {
  for (int i0 = 0; i0 < n; i0 += kSeqs) {
    const int i = i0 + threadIdx.x;
    const int held = i < n ? blocks_for(c.seq_len[seqs[i]] & 0x7fffffff, c.bs) : 0;
    int total;
    __syncthreads();
    ends[threadIdx.x] = block_scan(held, &total);
    __syncthreads();
    for (int e0 = 0; e0 < total; e0 += kThreads) {
      const int e = e0 + threadIdx.x;
      int k = -1, col = 0;
      if (e < total) {
        k = owner(ends, kSeqs, e);
        col = e - (k ? ends[k - 1] : 0);
      }
      f(k < 0 ? -1 : (i0 + k) * c.max_blocks + col,
        k < 0 ? nullptr : c.table + static_cast<size_t>(seqs[i0 + k]) * c.max_blocks + col);
    }
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads) free_kernel(Cache c, int n, const int32_t* seqs) {
  __shared__ int ends[kSeqs];
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
  if (__syncthreads_or(bad)) {
    if (t == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  // mark the listed sequences (sign bit of the length): one marked twice is listed twice
  for (int i = t; i < n; i += kThreads)
    bad = bad || atomicOr(&c.seq_len[seqs[i]], static_cast<int>(0x80000000u)) < 0;
  if (!__syncthreads_or(bad)) {
    for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
      if (key < 0) return;
      const int blk = *at;
      bad = bad || blk < 0 || blk >= c.n_blocks;
    });
  }
  if (__syncthreads_or(bad)) {
    for (int i = t; i < n; i += kThreads) atomicAnd(&c.seq_len[seqs[i]], 0x7fffffff);
    if (t == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
    if (key >= 0) atomicSub(&c.ref_count[*at], 1);
  });
  // a count below zero: more holders than were counted; put everything back
  for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
    if (key >= 0) bad = bad || c.ref_count[*at] < 0;
  });
  if (__syncthreads_or(bad)) {
    for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
      if (key >= 0) atomicAdd(&c.ref_count[*at], 1);
    });
    for (int i = t; i < n; i += kThreads) atomicAnd(&c.seq_len[seqs[i]], 0x7fffffff);
    if (t == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  // a block that nobody holds: its count becomes -1 - (its last key in the list)
  for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
    if (key >= 0 && c.ref_count[*at] <= 0) atomicMin(&c.ref_count[*at], -1 - key);
  });
  int pushes = 0, all;
  for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
    if (key >= 0) pushes += c.ref_count[*at] == -1 - key;
  });
  block_scan(pushes, &all);
  if (all > c.n_blocks - top) {  // more blocks than there are: the stack was wrong
    for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
      if (key >= 0 && c.ref_count[*at] < 0) c.ref_count[*at] = 0;
    });
    for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
      if (key >= 0) atomicAdd(&c.ref_count[*at], 1);
    });
    for (int i = t; i < n; i += kThreads) atomicAnd(&c.seq_len[seqs[i]], 0x7fffffff);
    if (t == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  int to = top;
  for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
    const int blk = key >= 0 ? *at : 0;
    const bool push = key >= 0 && c.ref_count[blk] == -1 - key;
    int total;
    const int place = to + block_scan(push, &total) - 1;
    if (push) c.free_list[place] = blk;
    to += total;
  });
  for_entries(c, n, seqs, ends, [&](int key, int32_t* at) {
    if (key < 0) return;
    const int blk = *at;
    if (c.ref_count[blk] < 0) c.ref_count[blk] = 0;
    *at = -1;
  });
  for (int i = t; i < n; i += kThreads) c.seq_len[seqs[i]] = 0;
  if (t == 0) *c.free_top = to;
}

// ---- fork ----

__global__ void __launch_bounds__(kThreads)
    fork_kernel(Cache c, int n, const int32_t* src, const int32_t* dst) {
  __shared__ int ends[kSeqs], part[kSeqs];
  const int t = threadIdx.x;
  if (t == 0) *c.err = 0;
  const int top = *c.free_top;
  bool bad = top < 0 || top > c.n_blocks;
  int started = 0;
  for (int i = t; i < n; i += kThreads) {
    const int s = src[i], d = dst[i];
    if (s < 0 || s >= c.B || d < 0 || d >= c.B) {
      bad = true;
      continue;
    }
    const int len = length_of(c, s, &bad);
    started += len % c.bs ? 1 : 0;
    bad = bad || c.seq_len[d] != 0;
  }
  int all;
  block_scan(started, &all);
  bool full = false;
  if (!__syncthreads_or(bad)) {
    // mark the new sequences: one marked twice is listed twice
    for (int i = t; i < n; i += kThreads)
      bad = bad || atomicExch(&c.seq_len[dst[i]], static_cast<int>(0x80000000u)) != 0;
    full = all > top;
    if (!full) {
      for (int e = t; e < all; e += kThreads) {
        const int blk = c.free_list[top - all + e];
        bad = bad || blk < 0 || blk >= c.n_blocks || c.ref_count[blk] != 0;
      }
    }
    __syncthreads();
    for (int i0 = 0; i0 < n; i0 += kSeqs) {
      const int i = i0 + t;
      const int len = i < n ? c.seq_len[src[i]] : 0;
      bad = bad || len < 0;  // marked: a source that is also new
      int total;
      ends[t] = block_scan(blocks_for(max(len, 0), c.bs), &total);
      __syncthreads();
      for (int e = t; e < total; e += kThreads) {
        const int k = owner(ends, kSeqs, e);
        const int blk = block_at(c, src[i0 + k], e - (k ? ends[k - 1] : 0));
        bad = bad || blk < 0 || c.ref_count[blk] < 1;
      }
      __syncthreads();
    }
    bad = __syncthreads_or(bad);
    if (bad || full)
      for (int i = t; i < n; i += kThreads) c.seq_len[dst[i]] = 0;
  } else {
    bad = true;
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
    const int len = i < n ? c.seq_len[src[i]] : 0;
    int total, fresh;
    ends[t] = block_scan(blocks_for(len, c.bs), &total);
    const int after = block_scan(len % c.bs ? 1 : 0, &fresh);
    part[t] = len % c.bs ? from + after - 1 : -1;  // where the stack has this one's block
    __syncthreads();
    for (int e = t; e < total; e += kThreads) {
      const int k = owner(ends, kSeqs, e);
      const int col = e - (k ? ends[k - 1] : 0);
      int blk;
      if (part[k] >= 0 && e == ends[k] - 1) {
        blk = c.free_list[part[k]];
        c.ref_count[blk] = 1;
      } else {
        blk = c.table[static_cast<size_t>(src[i0 + k]) * c.max_blocks + col];
        atomicAdd(&c.ref_count[blk], 1);
      }
      c.table[static_cast<size_t>(dst[i0 + k]) * c.max_blocks + col] = blk;
    }
    from += fresh;
    __syncthreads();
  }
  for (int i = t; i < n; i += kThreads) c.seq_len[dst[i]] = c.seq_len[src[i]];  // src is never a dst
  if (t == 0) *c.free_top = top - all;
}

constexpr int kCopyThreads = 128;

// One CTA: the started block of one new sequence, in one layer and head, of keys
// (blockIdx.z 0) or values.
__global__ void __launch_bounds__(kCopyThreads)
    fork_copy_kernel(Cache c, const int32_t* src, const int32_t* dst) {
  if (*c.err) return;  // refused
  const int h = blockIdx.x % c.H, l = blockIdx.x / c.H;
  const int s = src[blockIdx.y], d = dst[blockIdx.y];
  const int len = c.seq_len[d];
  const int rows = len % c.bs;
  if (rows == 0) return;
  const int from = block_at(c, s, len / c.bs), to = block_at(c, d, len / c.bs);
  if (from < 0 || to < 0) return;
  const int vec = c.d / 16;
  const uint4* x = reinterpret_cast<const uint4*>(c.pool[blockIdx.z]) + block_row(c, l, from, h) * vec;
  uint4* y = reinterpret_cast<uint4*>(c.pool[blockIdx.z]) + block_row(c, l, to, h) * vec;
  for (int i = threadIdx.x; i < rows * vec; i += kCopyThreads) y[i] = x[i];
  if (threadIdx.x == 0)
    c.scale[blockIdx.z][scale_at(c, l, to, h)] = c.scale[blockIdx.z][scale_at(c, l, from, h)];
}

}  // namespace

cudaError_t launch_grow(const Cache& c, const int32_t* n_new, cudaStream_t s) {
  grow_kernel<<<1, kThreads, 0, s>>>(c, n_new);
  return cudaGetLastError();
}

cudaError_t launch_free(const Cache& c, int n, const int32_t* seqs, cudaStream_t s) {
  free_kernel<<<1, kThreads, 0, s>>>(c, n, seqs);
  return cudaGetLastError();
}

cudaError_t launch_fork(const Cache& c, int n, const int32_t* src, const int32_t* dst,
                        cudaStream_t s) {
  fork_kernel<<<1, kThreads, 0, s>>>(c, n, src, dst);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  for (int i = 0; i < n; i += 65535)  // gridDim.y is at most 65535
    fork_copy_kernel<<<dim3(c.L * c.H, min(65535, n - i), 2), kCopyThreads, 0, s>>>(c, src + i,
                                                                                   dst + i);
  return cudaGetLastError();
}

}  // namespace cache8
}  // namespace kvc
