// cache8_rows.cu -- rows into and out of the 8-bit paged cache: quantise new
// tokens (append), make a cache dense for an event (gather), move the rows that
// an event kept into new blocks (compact).
//
// All three are bound by memory: append reads 2 d and writes d bytes per token
// and head, gather reads d and writes 2 d, compact reads and writes d.  A block's
// scale needs all of its rows before the first code can be written, so append and
// compact give one warp a whole block of one head: the warp keeps the rows in
// registers between the two steps (the rows past its registers, of blocks over 16
// tokens of 128 values, are read again, from L2), and the maximum is a warp
// reduction with no shared memory and no barrier.
//
// Measured, of the copy bandwidth of 6.77 TB/s: append of 4000 tokens to 8 sequences of
// 8 heads 33 us, 5.9 TB/s; gather of 28 layers of 8 sequences of 1536 tokens 155 us, 6.8
// TB/s; compact of these to 1024 slots 87 us, 5.5 TB/s.
#include "cache8.cuh"

namespace kvc {
namespace cache8 {
namespace {

constexpr int kWarps = 4;
constexpr int kKeep = 8;  // 16-byte chunks a lane keeps in registers

__device__ __forceinline__ void report(const Cache& c, uint32_t bits) {
  if (bits) atomicOr(c.status, bits);
}

// ---- append ----

// Largest |x| of 8 bf16 values as bf16 bits, folded into both halves of m.
__device__ __forceinline__ uint32_t max_abs8(uint4 v, uint32_t m) {
  m = __vmaxu2(m, v.x & 0x7fff7fffu);
  m = __vmaxu2(m, v.y & 0x7fff7fffu);
  m = __vmaxu2(m, v.z & 0x7fff7fffu);
  return __vmaxu2(m, v.w & 0x7fff7fffu);
}

// The same over the finite values only.
__device__ __forceinline__ uint32_t finite(uint32_t two) {
  two &= 0x7fff7fffu;
  return ((two & 0x7fffu) < 0x7f80u ? two & 0x7fffu : 0u) |
         ((two >> 16) < 0x7f80u ? two & 0x7fff0000u : 0u);
}
__device__ __forceinline__ uint32_t max_abs8_finite(uint4 v, uint32_t m) {
  return max_abs8(make_uint4(finite(v.x), finite(v.y), finite(v.z), finite(v.w)), m);
}

__device__ __forceinline__ uint32_t warp_max_half(uint32_t m) {
  m = max(m & 0xffffu, m >> 16);
  return __reduce_max_sync(0xffffffffu, m);
}

// 8 bf16 values to 8 codes.
template <int FMT, bool NAN_TOO>
__device__ __forceinline__ uint2 encode8(uint4 v, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = encode2<FMT, NAN_TOO>(bf16_lo(w[i]) * inv, bf16_hi(w[i]) * inv);
  return make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// Codes times 2^e, as codes again (the products are at most the largest code, but for
// e4m3's 448 at the largest scale, which int8 does not reach: clamped).  In fp16
// the products are exact wherever they do not round to code 0 (8 significant bits; what
// fp16 cannot hold is far below the smallest code), so that there is one rounding.
// Codes of a block whose scale shrinks by more than 2^15 are too small to be anything
// but 0 and the next few: those go through fp32.
template <int FROM, int TO>
__device__ __forceinline__ uint4 recode16(uint4 v, int e) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if (e <= 15) {
    const uint32_t factor = exp2_half2(e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo, hi;
      halves<FROM>(w[i], lo, hi);
      lo = mul_half2(lo, factor);
      hi = mul_half2(hi, factor);
      if constexpr (FROM == KVC_CACHE8_E4M3 && TO == KVC_CACHE8_INT8) {  // to +-127
        lo = clamp_half2(lo, 0xD7F0D7F0u, 0x57F057F0u);
        hi = clamp_half2(hi, 0xD7F0D7F0u, 0x57F057F0u);
      }
      w[i] = codes_of<TO>(lo, hi);
    }
  } else {
    const float ratio = exp2_int(min(e, 127));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[4];
      decode4<FROM>(w[i], x);
      w[i] = encode2<TO>(x[0] * ratio, x[1] * ratio) | encode2<TO>(x[2] * ratio, x[3] * ratio) << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Exponent of a scale (a power of two).
__device__ __forceinline__ int exp_of(float scale) {
  return static_cast<int>(__float_as_uint(scale) >> 23) - 127;
}

// One warp: one touched block of one head, keys (blockIdx.y 0) or values.  (int8 needs 80
// registers for 6 CTAs on an SM: 4000 tokens to 8 sequences of 8 heads 39 us, 41 with 82.)
template <int D, int FMT>
__global__ void __launch_bounds__(32 * kWarps, 6)
    append_kernel(Cache c, Rows k_new, Rows v_new, int n, int per_seq, const int32_t* row0,
                  const int32_t* n_new) {
  constexpr int CH = D / 8;  // 16-byte chunks of a bf16 row
  before_all();
  const int lane = threadIdx.x % 32;
  const uint32_t task = blockIdx.x * kWarps + threadIdx.x / 32;
  // heads fastest: the rows of a token-major source then lie side by side
  const int h = task % c.H;
  const uint32_t t1 = task / c.H;
  const int ib = t1 % per_seq;
  const uint32_t t2 = t1 / per_seq;
  const int b = t2 % c.B, l = t2 / c.B;
  if (l >= c.L) return;
  const int nn = n_new[b], at = row0 ? row0[b] : 0;  // the sequence's first row
  bool bad = false;
  const int len = length_of(c, b, &bad);
  if (bad || nn < 0 || at < 0 || nn > n - at || nn > len) {
    if (lane == 0) report(c, KVC_STATUS_BAD_INDEX);
    return;
  }
  const int start = len - nn;
  const int i = start / c.bs + ib;
  if (nn == 0 || static_cast<long long>(i) * c.bs >= len) return;
  const int first = i * c.bs;
  const int lo = max(first, start), hi = min(len, first + c.bs);
  const bool values = blockIdx.y != 0;
  const uint16_t* x = values ? v_new.at(l, b, h, at + lo - start) : k_new.at(l, b, h, at + lo - start);
  const long long stride = values ? v_new.token : k_new.token;
  const int total = (hi - lo) * CH;
  auto load = [&](int idx) {
    return *reinterpret_cast<const uint4*>(x + (idx / CH) * stride + (idx % CH) * 8);
  };
  uint4 keep[kKeep];
  uint32_t m = 0;
#pragma unroll
  for (int s = 0; s < kKeep; ++s) {
    const int idx = lane + 32 * s;
    keep[s] = idx < total ? load(idx) : make_uint4(0, 0, 0, 0);
  }
  // (the block and its old scale are looked up while the rows are on their way)
  const int blk = block_at(c, b, i);
  if (blk < 0) {
    if (lane == 0) report(c, KVC_STATUS_BAD_INDEX);
    return;
  }
  const int holders = c.ref_count[blk];
  float* scale_ptr = (values ? c.scale[1] : c.scale[0]) + scale_at(c, l, blk, h);
  const float old = lo > first ? *scale_ptr : 0.f;
#pragma unroll
  for (int s = 0; s < kKeep; ++s) m = max_abs8(keep[s], m);
  for (int idx = lane + 32 * kKeep; idx < total; idx += 32) m = max_abs8(load(idx), m);
  m = warp_max_half(m);
  if (holders != 1) {  // a shared block is never written
    if (lane == 0) report(c, KVC_STATUS_BAD_INDEX);
    return;
  }
  const bool finite_rows = m < 0x7f80u;
  if (!finite_rows) {  // an infinity or a NaN: the finite values alone give the scale
    if (lane == 0) report(c, KVC_STATUS_NONFINITE);
    m = 0;
    for (int idx = lane; idx < total; idx += 32) m = max_abs8_finite(load(idx), m);
    m = warp_max_half(m);
  }
  float scale = exp2_int(scale_exp<FMT>(__uint_as_float(m << 16)));
  uint8_t* rows = (values ? c.pool[1] : c.pool[0]) + block_row(c, l, blk, h) * D;
  if (lo > first) {  // older rows: the scale only grows, and they follow it
    if (old >= scale) {
      scale = old;
    } else {
      const int down = exp_of(old) - exp_of(scale);
      uint4* p = reinterpret_cast<uint4*>(rows);
      for (int idx = lane; idx < (lo - first) * (D / 16); idx += 32)
        p[idx] = recode16<FMT, FMT>(p[idx], down);
    }
    __syncwarp();  // every lane has read the old scale
  }
  const float inv = 1.f / scale;  // exact
  uint2* to = reinterpret_cast<uint2*>(rows + static_cast<size_t>(lo - first) * D);
  if (finite_rows) {
#pragma unroll
    for (int s = 0; s < kKeep; ++s) {
      const int idx = lane + 32 * s;
      if (idx < total) to[idx] = encode8<FMT, false>(keep[s], inv);
    }
    for (int idx = lane + 32 * kKeep; idx < total; idx += 32)
      to[idx] = encode8<FMT, false>(load(idx), inv);
  } else {
    for (int idx = lane; idx < total; idx += 32) to[idx] = encode8<FMT, true>(load(idx), inv);
  }
  if (lane == 0) *scale_ptr = scale;
}

// ---- gather ----

constexpr int kGatherThreads = 256;
constexpr int kGatherUnroll = 4;

// 8 codes to 8 bf16 values (exact: at most 7 significant bits, times a power of two).
template <int FMT>
__device__ __forceinline__ uint4 values8(uint2 v, float scale) {
  float x[4], y[4];
  decode4<FMT>(v.x, x);
  decode4<FMT>(v.y, y);
  return make_uint4(bf16x2(x[0] * scale, x[1] * scale), bf16x2(x[2] * scale, x[3] * scale),
                    bf16x2(y[0] * scale, y[1] * scale), bf16x2(y[2] * scale, y[3] * scale));
}

// One thread: 8 values of kGatherUnroll rows, of keys and values.
template <int D, int FMT>
__global__ void __launch_bounds__(kGatherThreads)
    gather_kernel(Cache c, int T, int ctas_per_unit, uint16_t* k_out, uint16_t* v_out,
                  int32_t* pad_out) {
  constexpr int CH = D / 8;
  before_all();
  const int u = blockIdx.x / ctas_per_unit;
  const int part = blockIdx.x % ctas_per_unit;
  const int h = u % c.H, b = (u / c.H) % c.B, l = u / (c.H * c.B);
  bool bad = false;
  int len = length_of(c, b, &bad);
  if (len > T) {
    bad = true;
    len = 0;
  }
  const int pad = T - len;
  if (l == 0 && h == 0 && part == 0 && threadIdx.x == 0) pad_out[b] = pad;
  const int ch = threadIdx.x % CH;
  const int row0 = part * (kGatherThreads / CH * kGatherUnroll) + threadIdx.x / CH;
  uint2 kc[kGatherUnroll], vc[kGatherUnroll];
  float ks[kGatherUnroll], vs[kGatherUnroll];
#pragma unroll
  for (int i = 0; i < kGatherUnroll; ++i) {
    const int t = row0 + i * (kGatherThreads / CH);
    kc[i] = vc[i] = make_uint2(0, 0);
    ks[i] = vs[i] = 0.f;
    if (t < T && t >= pad) {
      const int pos = t - pad;
      const int blk = block_at(c, b, pos / c.bs);
      if (blk < 0) {
        bad = true;
      } else {
        const size_t at = (block_row(c, l, blk, h) + pos % c.bs) * CH + ch;
        const size_t sc = scale_at(c, l, blk, h);
        kc[i] = reinterpret_cast<const uint2*>(c.pool[0])[at];
        ks[i] = c.scale[0][sc];
        if (v_out) {
          vc[i] = reinterpret_cast<const uint2*>(c.pool[1])[at];
          vs[i] = c.scale[1][sc];
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kGatherUnroll; ++i) {
    const int t = row0 + i * (kGatherThreads / CH);
    if (t < T) {
      const size_t at = (static_cast<size_t>(u) * T + t) * CH + ch;
      reinterpret_cast<uint4*>(k_out)[at] = values8<FMT>(kc[i], ks[i]);
      if (v_out) reinterpret_cast<uint4*>(v_out)[at] = values8<FMT>(vc[i], vs[i]);
    }
  }
  if (bad) report(c, KVC_STATUS_BAD_INDEX);
}

// ---- compact ----

constexpr int kCompactThreads = 256;
constexpr int kKeepRows = 16;     // rows whose codes a warp keeps in registers
constexpr int kLookRows = 1024;   // rows of a CTA at most (the largest block)
constexpr int kMaxBlocks = 16;    // blocks of a CTA at most: two a warp

// Bytes 2 k and 2 k + 1 as two signed 16-bit integers.
template <int K>
__device__ __forceinline__ uint32_t signed_pair(uint32_t four) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(four), "n"(K == 0 ? 0x9180 : 0xb3a2));
  return r;
}

// Largest |code| of 16 finite ones: integers order e4m3 magnitudes as well.
template <int FMT>
__device__ __forceinline__ float max_code16(uint4 v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (FMT == KVC_CACHE8_E4M3) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(__vmaxu2(m, w[i] & 0x007f007fu), (w[i] >> 8) & 0x007f007fu);
    float x[4];
    decode4<FMT>(max(m & 0xffffu, m >> 16), x);
    return x[0];
  } else {
    uint32_t hi = 0, lo = 0;  // pairs of 16 bits: largest and smallest
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = signed_pair<0>(w[i]), b = signed_pair<1>(w[i]);
      hi = __vmaxs2(hi, __vmaxs2(a, b));
      lo = __vmins2(lo, __vmins2(a, b));
    }
    const int most = max(static_cast<int16_t>(hi & 0xffffu), static_cast<int16_t>(hi >> 16));
    const int least = min(static_cast<int16_t>(lo & 0xffffu), static_cast<int16_t>(lo >> 16));
    return static_cast<float>(max(most, -least));
  }
}

// One CTA: some new blocks of one head, keys and values.  Its threads look the rows up
// (kept index, block, scales: three loads that wait for one another, once for all
// blocks), then each warp takes whole blocks, two in turn.  The 28-layer event of 8
// sequences (1536 -> 1024 slots) takes 87 us, 5.5 TB/s; with a warp looking up its own 16
// rows it took 106, with one block a warp 111, at 3 CTAs per SM 95.
template <int D, int FROM, int TO>
__global__ void __launch_bounds__(kCompactThreads, 4)
    compact_kernel(Cache c, Cache to, CompactArgs a, int per_unit, int blocks) {
  constexpr int CH = D / 16;                     // 16-byte chunks of a row
  constexpr int RPI = 32 / CH;                   // rows of one load of a warp
  constexpr int KEEP = kKeepRows / RPI;
  __shared__ int s_row[kLookRows];               // place in the pools (rows of d codes from the
  __shared__ float s_scale[2][kLookRows];        // layer's first, of this head); -1: none
  before_all();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int ch = lane % CH;
  const int u = blockIdx.x / per_unit;
  const int jb0 = blockIdx.x % per_unit * blocks;
  const int h = u % c.H, b = (u / c.H) % c.B, l = u / (c.H * c.B);
  bool bad = false;
  const int len = length_of(c, b, &bad);
  const int nk = a.n_kept[u];
  const int new_len = length_of(to, b, &bad);
  const int pad = a.pad[b];
  if (bad || nk < 0 || nk > a.budget || nk != new_len) {
    if (threadIdx.x == 0) report(c, KVC_STATUS_BAD_INDEX);
    return;
  }
  const int j0 = jb0 * to.bs;
  const size_t scale_base = scale_at(c, l, 0, h);
  for (int r = threadIdx.x; r < blocks * to.bs && j0 + r < a.budget; r += kCompactThreads) {
    const size_t at = static_cast<size_t>(u) * a.budget + j0 + r;
    int row = -1;
    float ks = 0.f, vs = 0.f, credit = 0.f;
    if (j0 + r < nk) {
      const int slot = a.kept[at];
      const long long pos = static_cast<long long>(slot) - pad;
      if (slot >= 0 && slot < a.T && a.credit_out)
        credit = a.credit_post[static_cast<size_t>(u) * a.T + slot];
      const bool in = pos >= 0 && pos < len && slot >= 0 && slot < a.T;
      const int blk = in ? block_at(c, b, static_cast<int>(pos) / c.bs) : -1;
      if (blk < 0) {
        bad = true;
      } else {
        row = blk * c.H * c.bs + static_cast<int>(pos) % c.bs;  // below 2^31: checked on the host
        const size_t sc = scale_base + static_cast<size_t>(blk) * c.H;
        ks = c.scale[0][sc];
        vs = c.scale[1][sc];
      }
    }
    s_row[r] = row;
    s_scale[0][r] = ks;
    s_scale[1][r] = vs;
    if (a.credit_out) a.credit_out[at] = credit;
  }
  __syncthreads();
  const size_t base = block_row(c, l, 0, h);
  for (int jb = warp; jb < blocks; jb += kCompactThreads / 32) {
    const int rows = min(nk - j0 - jb * to.bs, to.bs);
    if (rows <= 0) break;
    const int new_blk = block_at(to, b, jb0 + jb);
    if (new_blk < 0 || to.ref_count[new_blk] != 1) {  // (a shared block is never written)
      bad = true;
      continue;
    }
    const int* my_row = s_row + jb * to.bs;
    const float* my_ks = s_scale[0] + jb * to.bs;
    const float* my_vs = s_scale[1] + jb * to.bs;
    auto load = [&](const uint8_t* pool, int r) {  // chunk ch of row r
      const int from = r < rows ? my_row[r] : -1;
      return from >= 0 ? reinterpret_cast<const uint4*>(pool)[(base + from) * CH + ch]
                       : make_uint4(0, 0, 0, 0);
    };
    uint4 kk[KEEP], kv[KEEP];
#pragma unroll
    for (int i = 0; i < KEEP; ++i) kk[i] = load(c.pool[0], i * RPI + lane / CH);
#pragma unroll
    for (int i = 0; i < KEEP; ++i) kv[i] = load(c.pool[1], i * RPI + lane / CH);
    float km = 0.f, vm = 0.f;
    auto most = [&](int r, uint4 k, uint4 v) {
      if (r >= rows) return;
      km = fmaxf(km, max_code16<FROM>(k) * my_ks[r]);
      vm = fmaxf(vm, max_code16<FROM>(v) * my_vs[r]);
    };
#pragma unroll
    for (int i = 0; i < KEEP; ++i) most(i * RPI + lane / CH, kk[i], kv[i]);
    // (the other rows of larger blocks are read twice, the second time from L2)
    for (int r = kKeepRows + lane / CH; r < rows; r += RPI)
      most(r, load(c.pool[0], r), load(c.pool[1], r));
    const int k_exp = scale_exp<TO>(warp_max(km)), v_exp = scale_exp<TO>(warp_max(vm));
    const size_t out = block_row(to, l, new_blk, h) * CH + ch;
    uint4* ko = reinterpret_cast<uint4*>(to.pool[0]) + out;
    uint4* vo = reinterpret_cast<uint4*>(to.pool[1]) + out;
    auto store = [&](int r, uint4 k, uint4 v) {
      if (r >= rows) return;
      ko[r * CH] = recode16<FROM, TO>(k, exp_of(my_ks[r]) - k_exp);
      vo[r * CH] = recode16<FROM, TO>(v, exp_of(my_vs[r]) - v_exp);
    };
#pragma unroll
    for (int i = 0; i < KEEP; ++i) store(i * RPI + lane / CH, kk[i], kv[i]);
    for (int r = kKeepRows + lane / CH; r < rows; r += RPI)
      store(r, load(c.pool[0], r), load(c.pool[1], r));
    if (lane == 0) {
      const size_t sc = scale_at(to, l, new_blk, h);
      to.scale[0][sc] = exp2_int(k_exp);
      to.scale[1][sc] = exp2_int(v_exp);
    }
  }
  if (bad) report(c, KVC_STATUS_BAD_INDEX);
}

int ctas(long long tasks) { return static_cast<int>((tasks + kWarps - 1) / kWarps); }

}  // namespace

cudaError_t launch_append(const Cache& c, int format, const Rows& k, const Rows& v, int n,
                          const int32_t* row0, const int32_t* n_new, cudaStream_t s) {
  const int most = min(n, c.max_blocks * c.bs);  // a sequence has no more new tokens than that
  const int per_seq = (most - 1 + c.bs - 1) / c.bs + 1;  // blocks that they can touch
  const dim3 grid(ctas(static_cast<long long>(c.L) * c.B * c.H * per_seq), 2);
  auto* kernel = c.d == 64 ? (format == KVC_CACHE8_E4M3 ? append_kernel<64, KVC_CACHE8_E4M3>
                                                        : append_kernel<64, KVC_CACHE8_INT8>)
                           : (format == KVC_CACHE8_E4M3 ? append_kernel<128, KVC_CACHE8_E4M3>
                                                        : append_kernel<128, KVC_CACHE8_INT8>);
  return launch(kernel, grid, 32 * kWarps, 0, s, c, k, v, n, per_seq, row0, n_new);
}

cudaError_t launch_gather(const Cache& c, int format, int T, uint16_t* k_out, uint16_t* v_out,
                          int32_t* pad, cudaStream_t s) {
  const int rows = kGatherThreads / (c.d / 8) * kGatherUnroll;
  const int per_unit = (T + rows - 1) / rows;
  const int grid = c.L * c.B * c.H * per_unit;
  auto* kernel = c.d == 64 ? (format == KVC_CACHE8_E4M3 ? gather_kernel<64, KVC_CACHE8_E4M3>
                                                        : gather_kernel<64, KVC_CACHE8_INT8>)
                           : (format == KVC_CACHE8_E4M3 ? gather_kernel<128, KVC_CACHE8_E4M3>
                                                        : gather_kernel<128, KVC_CACHE8_INT8>);
  return launch(kernel, grid, kGatherThreads, 0, s, c, T, per_unit, k_out, v_out, pad);
}

template <int D>
static cudaError_t launch_compact_d(const Cache& c, int from, const Cache& to, int to_format,
                                    const CompactArgs& a, cudaStream_t s) {
  const int all = (a.budget + to.bs - 1) / to.bs;
  const int blocks = min(min(max(kLookRows / to.bs, 1), kMaxBlocks), all);
  const int per_unit = (all + blocks - 1) / blocks;
  const int grid = c.L * c.B * c.H * per_unit;
  constexpr int E = KVC_CACHE8_E4M3, I = KVC_CACHE8_INT8;
  auto* kernel = from == E ? (to_format == E ? compact_kernel<D, E, E> : compact_kernel<D, E, I>)
                           : (to_format == E ? compact_kernel<D, I, E> : compact_kernel<D, I, I>);
  return launch(kernel, grid, kCompactThreads, 0, s, c, to, a, per_unit, blocks);
}

cudaError_t launch_compact(const Cache& src, int src_format, const Cache& dst, int dst_format,
                           const CompactArgs& a, cudaStream_t s) {
  return src.d == 64 ? launch_compact_d<64>(src, src_format, dst, dst_format, a, s)
                     : launch_compact_d<128>(src, src_format, dst, dst_format, a, s);
}

}  // namespace cache8
}  // namespace kvc
