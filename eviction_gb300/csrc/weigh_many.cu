// weigh_many.cu -- attention weight that many queries (a prompt, or a piece of one) give each
// token of the 8-bit paged cache, on the 5th-generation tensor cores (tcgen05 + TMEM).
//
//   w_t = decay w_t + sum_r 2^(f_t s_rt - y_r),  s = q_r . code_t,  f_t = scale log2(e) scale_t,
//
// y_r the row's log2 normaliser.  Tokens are the rows of S^T = K Q^T (TMEM lanes) and queries its
// columns, so that a token's sum is one thread's, with its key's scale a factor of that thread.
// Keys are codes as bf16, which holds both formats exactly, and queries are what they are in
// memory: nothing is rounded before the product.
//
// A CTA has two tiles of 128 tokens and takes 192 query rows at a time for both:
//   keys (4 warps)    codes of the item's tokens from their blocks to bf16 rows in TMEM, a
//                     thread a token; the next item's are loaded while this one is computed;
//   queries (1 warp)  TMA, through a ring of stages, and the rows' normalisers beside them.  A
//                     group's heads lie side by side (row = token * P + head), so that each
//                     chunk is of few tokens;
//   MMA (1 warp)      128 x 192 products into the tile's columns of TMEM, with the keys read
//                     from there: from shared memory, keys, queries, copies and normalisers
//                     together asked for more than its bandwidth (98 us with 128 columns a
//                     product, 84 us with 256, of 82 then);
//   weights (16 warps)  two warps a lane quarter and tile, a half of the columns each: scale,
//                     exponential, sum.  One tile's exponentials run while the other's
//                     products do.
// Exponentials and products take the same time (512 cycles of an SM for 128 x 128).  Measured, 8
// sequences of 1536 tokens, all queries of 4 x 7 heads of 128: 83 us.  What bounds it are the weight
// warps, busy 85% of the time: 1200 cycles a tile and chunk, for 768 of exponentials alone, go by
// on waits, TMEM loads and normalisers of shared memory.  (A warp of products for each tile 87 us; all
// sixteen weight warps on one tile at a time 88; three buffers of 128 columns for both tiles 101.)  At
// 80 registers up to 20 bytes a thread spill at d 128.
// Chunks that a tile does not see are skipped.
//
// Work: pairs of tiles of all sequences, layers and heads, those with most queries first, dealt
// to one CTA per SM in turns, back and forth.  Where there are few pairs their queries are cut into
// parts, whose sums a second launch adds up in order.  How many goes by the call's sizes (cap,
// table, batch, rows) and the SMs, so that a token's last bits do too, but nothing depends on the
// schedule.  Every wait is bounded.
#include <climits>

#include "weigh.cuh"

namespace kvc {
namespace prompt {
namespace {

using namespace cache8;

constexpr int kTile = 128, kChunk = 192;  // tokens of a tile, query rows of a chunk
constexpr int kHalf = kChunk / 2;         // columns of a weight warp
constexpr uint32_t kKeyCol = 2 * kChunk;  // the keys' first TMEM column, after the products'
constexpr int kWeightWarps = 16, kKeyWarp = 16, kQueryWarp = 20, kMmaWarp = 21, kItemWarp = 22;
constexpr int kThreads = 32 * 23;
// (a warp reads and writes the quarter of TMEM's lanes that its number tells)
static_assert(kWeightWarps == 16 && kKeyWarp % 4 == 0, "groups of four warps");
constexpr int kItems = 4;        // items told ahead
constexpr int kSums = 4;         // chunks whose normalisers are told ahead
constexpr int kReaders = kWeightWarps + 4 + 2;
constexpr int kSorted = 128;     // sequences (or groups of them) in the list of items
constexpr int kPacked = 16;      // heads in a chunk at most

template <bool V>
struct Bool {
  static constexpr bool value = V;
};

struct Params {
  WeighArgs a;
  int P, subs, tok;   // heads in a chunk, such parts of a group, tokens of a chunk
  int parts;          // of an item's queries
  int pairs;          // of tiles that a sequence may have
  float* part;        // [units * B][pairs][parts][2 kTile] sums, where parts > 1; -1: absent
  int q_head, q_seq, q_layer;  // 0 where the axis' stride is 0
};

struct Item {
  int l, b, h;        // of the cache
  int len, nq, first;
  int t0;             // first token of tile 0
  int chunks;         // of a part of the group, from chunk c0 on (before it neither tile is seen)
  int c0;             // first chunk that tile 0 sees
  int c1;             // first chunk that tile 1 sees
  int there;          // 0: no more items
  int part;
};

template <int D>
struct Smem {
  static constexpr int kStage = kChunk * D * 2, kStages = D == 128 ? 4 : 8;
  static constexpr int kRing = 0, kSumsAt = kRing + kStages * kStage,
                       kFactors = kSumsAt + kSums * kChunk * 4,   // [2][2][128] f_t, by item parity
                       kParts = kFactors + 2 * 2 * kTile * 4,     // [2][128] the second halves' sums
                       kBars = kParts + 2 * kTile * 4,
                       kNumBars = 2 * kStages + 2 * kSums + 2 * 6 + 2 * kItems + 2,
                       kItem = (kBars + kNumBars * 8 + 15) & ~15, kMisc = kItem + kItems * 48,
                       kUpTo = kMisc + 16, kCount = kUpTo + (kSorted + 1) * 4,
                       kSeq = kCount + (kSorted + 1) * 4, kBytes = kSeq + kSorted + 1024;
  static_assert(kBytes <= 232448, "shared memory of a block");
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}

// Four codes to four bf16 (exact), without the conversions from fp16, which the exponentials'
// unit does.  e4m3: sign, exponent and mantissa in their places of a bf16 are the value times
// 2^-120 (subnormals too).  Integers: biased to 0..255 they are the last bits of 2^23 + u.
template <int FMT>
__device__ __forceinline__ uint2 bf16_of(uint32_t codes) {
  if constexpr (FMT == KVC_CACHE8_E4M3) {
    uint32_t r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t x = __byte_perm(codes, 0, i ? 0x3424 : 0x1404);  // codes in the high bytes
      const uint32_t bits = (x & 0x80008000u) | ((x >> 4) & 0x07f007f0u);
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r[i]) : "r"(bits), "r"(0x7b807b80u));  // 2^120
    }
    return make_uint2(r[0], r[1]);
  } else {
    const uint32_t u = codes ^ 0x80808080u;
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7440 + i)) - 8388736.f;
    return make_uint2(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]));
  }
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    weigh_many_kernel(const __grid_constant__ CUtensorMap map_q, Cache c, Params p, Div by_bs) {
#if defined(__CUDA_ARCH__) && (__CUDA_ARCH__ >= 1000)
  using Sm = Smem<D>;
  constexpr int DB = D / 64;
  constexpr int NS = Sm::kStages;
  constexpr int kQueryBlock = kChunk * 128;  // bytes of 64 values of all rows
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sm::kBars);
  uint64_t *q_full = bars, *q_empty = bars + NS, *y_full = bars + 2 * NS, *y_empty = y_full + kSums,
           *k_full = y_empty + kSums,
           *k_empty = k_full + 2, *s_full = k_empty + 2, *s_empty = s_full + 2, *part_full = s_empty + 2,
           *part_empty = part_full + 2, *i_full = part_empty + 2, *i_empty = i_full + kItems,
           *done = i_empty + kItems, *odd_full = done + 1;
  static_assert(Sm::kNumBars == 2 * NS + 2 * kSums + 12 + 2 * kItems + 2, "one place for each barrier");
  float* s_sums = reinterpret_cast<float*>(smem + Sm::kSumsAt);      // [kSums][kChunk] -y
  float* s_factors = reinterpret_cast<float*>(smem + Sm::kFactors);  // [2][2][kTile]
  float* s_parts = reinterpret_cast<float*>(smem + Sm::kParts);      // [2][kTile]
  Item* items = reinterpret_cast<Item*>(smem + Sm::kItem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Sm::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + Sm::kMisc + 4);
  int* s_upto = reinterpret_cast<int*>(smem + Sm::kUpTo);
  int* s_count = reinterpret_cast<int*>(smem + Sm::kCount);
  uint8_t* s_seq = smem + Sm::kSeq;
  const WeighArgs& a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    for (int s = 0; s < kSums; ++s) {
      mbar_init(&y_full[s], 1);
      mbar_init(&y_empty[s], kWeightWarps);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&k_full[t], 4);
      mbar_init(&k_empty[t], 1 + 8);
      mbar_init(&s_full[t], 1);
      mbar_init(&s_empty[t], 8);
      mbar_init(&part_full[t], 4);
      mbar_init(&part_empty[t], 4);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&i_full[i], 1);
      mbar_init(&i_empty[i], kReaders);
    }
    mbar_init(done, 1);
    mbar_init(odd_full, 1);
    *abort = 0;
    fence_barrier_init();
    prefetch_tensormap(&map_q);
  }
  // query rows that no copy writes (P does not divide 192) are zeros: their products count nothing
  for (int i = threadIdx.x; i < NS * Sm::kStage / 16; i += kThreads)
    *reinterpret_cast<uint4*>(smem + Sm::kRing + i * 16) = make_uint4(0, 0, 0, 0);
  fence_async_shared();
  before_all();

  // ---- the list of items: groups of `per` sequences (one each, if they are few enough; those
  // with most pairs of tiles first then) ----
  const int units = c.L * c.H * p.parts;  // items of a pair of tiles, over layers and heads
  const int per = div_up(c.B, kSorted), groups = div_up(c.B, per);
  bool bad = false;
  auto pairs_of = [&](int b) { return div_up(lengths_of(c, a, b, &bad).len, 2 * kTile); };
  if (threadIdx.x < kSorted) {
    int n = 0;  // (cap and the sequences' number bound it: checked on the host)
    for (int b = threadIdx.x * per; b < min((static_cast<int>(threadIdx.x) + 1) * per, c.B); ++b)
      n += pairs_of(b);
    s_upto[threadIdx.x] = n;
    if (bad && blockIdx.x == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    bad = false;
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (static_cast<int>(threadIdx.x) < groups) {  // its place: by the count, then by the number
    const int mine = s_upto[threadIdx.x];
    int at = per > 1 ? threadIdx.x : 0;
    if (per == 1)
      for (int g = 0; g < groups; ++g) {
        const int other = s_upto[g];
        at += other > mine || (other == mine && g < static_cast<int>(threadIdx.x));
      }
    s_count[at] = mine;
    s_seq[at] = static_cast<uint8_t>(threadIdx.x);
  }
  if (threadIdx.x == 0) s_count[groups] = 0;
  __syncthreads();
  // s_upto[q]: items of a unit among those of the levels (the x-th pairs from the end of all
  // sequences that have them) that more than q sequences do not reach; or, of groups of several
  // sequences, of groups 0 .. q
  if (warp == kItemWarp) {
    int before = 0;
    for (int q0 = 0; q0 < groups; q0 += 32) {
      const int q = q0 + lane;
      int incl = q < groups ? s_count[q] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      incl += before;
      if (q < groups) s_upto[q] = per > 1 ? incl : incl - (q + 1) * s_count[q + 1];
      before = __shfl_sync(0xffffffffu, incl, 31);
    }
    __syncwarp();
  }

  auto read_item = [&](int i, Item& it) {
    if (!warp_wait(&i_full[i % kItems], (i / kItems) & 1, abort, c.status)) return false;
    it = items[i % kItems];
    return it.there != 0;
  };
  auto leave_item = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&i_empty[i % kItems]);
  };

  if (warp < kWeightWarps) {
    // ------------------------------------------------------------ weights
    // Warp 4 (2 h + t) + q: tile t, half h of the columns, lane quarter q.
    const int t = warp / 4 % 2, half = warp / 8, quarter = warp % 4;
    const int row = quarter * 32 + lane;
    const uint32_t s_tmem = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + t * kChunk + half * kHalf;
    int step = 0;     // products of this tile
    uint32_t use = 0;  // chunks
    Item it;
    for (int i = 0; read_item(i, it); ++i) {
      leave_item(i);
      if (!warp_wait(&k_full[t], i & 1, abort, c.status)) break;  // (the factors come with the keys)
      const float f = s_factors[((i & 1) * 2 + t) * kTile + row];
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_empty[t]);  // (no more than one item ahead of these warps)
      const int token = it.t0 + t * kTile + row;
      const int jmin = token - (it.len - it.nq);   // the first query that sees this token
      const int first_c = t ? it.c1 : it.c0;
      const float2 ff = make_float2(f, f);
      float2 sum = make_float2(0.f, 0.f);
      bool ok = true;
      for (int s = 0; ok && s < p.subs; ++s)
        for (int ch = it.c0; ch < it.chunks; ++ch, ++use) {
          const int st = use % kSums;
          // (also for a chunk that the tile does not see: this warp's arrival counts for its use)
          if (!(ok = warp_wait(&y_full[st], (use / kSums) & 1, abort, c.status))) break;
          if (ch >= first_c) {
            if (!(ok = warp_wait(&s_full[t], step & 1, abort, c.status))) break;
            ++step;
            tc_fence_after();
            const float* y = s_sums + st * kChunk + half * kHalf;
            const int j0 = ch * p.tok;
            // columns of this half that count: [lo, hi)
            const int lo = max(jmin - j0, 0) * p.P - half * kHalf;
            const int hi = min(it.nq - j0, p.tok) * p.P - half * kHalf;
            const bool whole = __all_sync(0xffffffffu, lo <= 0) && hi >= kHalf - (kChunk - p.tok * p.P) * half;
            uint32_t va[32], vb[32], valid = 0;
            auto add = [&](const uint32_t (&v)[32], int col, auto masked) {
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const float4 yy = *reinterpret_cast<const float4*>(y + col + k);
                float2 e0 = fma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), ff,
                                 make_float2(yy.x, yy.y));
                float2 e1 = fma2(make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), ff,
                                 make_float2(yy.z, yy.w));
                e0.x = ex2(e0.x);
                e0.y = ex2(e0.y);
                e1.x = ex2(e1.x);
                e1.y = ex2(e1.y);
                if constexpr (decltype(masked)::value) {
                  e0.x = valid & 1u << k ? e0.x : 0.f;
                  e0.y = valid & 2u << k ? e0.y : 0.f;
                  e1.x = valid & 4u << k ? e1.x : 0.f;
                  e1.y = valid & 8u << k ? e1.y : 0.f;
                }
                sum = add2(sum, add2(e0, e1));
              }
            };
            auto release = [&]() {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&s_empty[t]);
            };
            if (whole) {
              tmem_ld32(s_tmem, va);
              tmem_ld_wait();
              tmem_ld32(s_tmem + 32, vb);
              add(va, 0, Bool<false>{});
              tmem_ld_wait();
              tmem_ld32(s_tmem + 64, va);
              add(vb, 32, Bool<false>{});
              tmem_ld_wait();
              release();
              add(va, 64, Bool<false>{});
            } else {
#pragma unroll 1
              for (int k = 0; k < kHalf / 32; ++k) {
                // this lane's columns of the block that count, a bit each
                const int from = max(lo - 32 * k, 0), to = min(hi - 32 * k, 32);
                valid = from < to ? (0xffffffffu >> (32 - to)) & (0xffffffffu << from) : 0u;
                if (!__any_sync(0xffffffffu, valid)) continue;
                tmem_ld32(s_tmem + 32 * k, va);
                tmem_ld_wait();
                if (__all_sync(0xffffffffu, valid == 0xffffffffu))
                  add(va, 32 * k, Bool<false>{});
                else
                  add(va, 32 * k, Bool<true>{});
              }
              release();
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&y_empty[st]);
        }
      if (!ok) break;
      // the second half's sums to the first half's warps, which write the token
      const float mine = sum.x + sum.y;
      if (half) {
        if (!warp_wait(&part_empty[t], (i & 1) ^ 1, abort, c.status)) break;
        s_parts[t * kTile + row] = mine;
        __syncwarp();
        if (lane == 0) mbar_arrive(&part_full[t]);
      } else {
        float* w = a.w + (static_cast<size_t>(it.l * c.B + it.b) * c.H + it.h) * a.cap + token;
        const bool there = token < it.len;
        const float old = there && a.decay != 0.f && p.parts == 1 ? a.decay * *w : 0.f;
        if (!warp_wait(&part_full[t], i & 1, abort, c.status)) break;
        const float all = mine + s_parts[t * kTile + row];
        __syncwarp();
        if (lane == 0) mbar_arrive(&part_empty[t]);
        if (there && p.parts == 1) *w = f < 0.f ? old : old + all;  // (an absent token)
        if (there && p.parts > 1)
          p.part[((((static_cast<size_t>(it.l) * c.B + it.b) * c.H + it.h) * p.pairs + it.t0 / (2 * kTile)) *
                      p.parts + it.part) * (2 * kTile) + t * kTile + row] = f < 0.f ? -1.f : all;
      }
    }
  } else if (warp < kQueryWarp) {
    // ------------------------------------------------------------ keys
    // This thread: token 32 kw + lane of each tile, a lane of TMEM.
    const int kw = warp - kKeyWarp;
    const uint32_t key_tmem = tmem + (static_cast<uint32_t>(kw * 32) << 16) + kKeyCol;
    Item it;
    for (int i = 0; read_item(i, it); ++i) {
      leave_item(i);
      bool ok = true;
      const int32_t* table = c.table + static_cast<size_t>(it.b) * c.max_blocks;
      int row[2];
      float f[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int own = it.t0 + t * kTile + kw * 32 + lane;
        row[t] = -1;
        f[t] = -1.f;  // absent
        if (own < it.len) {
          const int n = by_bs.div(own), blk = table[n];
          if (static_cast<uint32_t>(blk) < static_cast<uint32_t>(c.n_blocks)) {
            f[t] = finite_factor(a.scale_log2, c.scale[0][scale_at(c, it.l, blk, it.h)]);
            row[t] = blk * c.H * by_bs.bs + (own - n * by_bs.bs);  // < 2^31: checked on the host
          } else {
            bad = true;
          }
        }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (!ok) continue;
        uint4 codes[D / 16];
        const uint4* from = reinterpret_cast<const uint4*>(
            c.pool[0] + (block_row(c, it.l, 0, it.h) + max(row[t], 0)) * D);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) codes[x] = row[t] >= 0 ? from[x] : make_uint4(0, 0, 0, 0);
        // (the last item's products with this tile are done)
        if (!(ok = warp_wait(&k_empty[t], (i & 1) ^ 1, abort, c.status))) continue;
        tc_fence_after();
        s_factors[((i & 1) * 2 + t) * kTile + kw * 32 + lane] = f[t];
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          uint32_t v[16];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t w[4] = {codes[2 * x + k].x, codes[2 * x + k].y, codes[2 * x + k].z, codes[2 * x + k].w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const uint2 y = bf16_of<FMT>(w[z]);
              v[8 * k + 2 * z] = y.x;
              v[8 * k + 2 * z + 1] = y.y;
            }
          }
          tmem_st16(key_tmem + t * (D / 2) + 16 * x, v);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[t]);
      }
      if (!ok) break;
    }
    if (bad) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
  } else if (warp == kQueryWarp) {
    // ------------------------------------------------------------ queries
    // A chunk's rows by TMA, and its rows' normalisers beside them, from this lane's columns
    // lane + 32 k: head g and token j of the chunk.  A query that sees no token may hold anything: where
    // there is one, this warp waits for the copy itself and writes zeros in its place, so that
    // its products are no NaN.
    int j[kChunk / 32], g[kChunk / 32];
#pragma unroll
    for (int k = 0; k < kChunk / 32; ++k) {
      const int col = lane + 32 * k;
      j[k] = col < p.tok * p.P ? col / p.P : INT_MAX / 2;
      g[k] = col % p.P;
    }
    uint32_t use = 0, odd = 0;
    bool ok = true;
    Item it;
    for (int i = 0; ok && read_item(i, it); ++i) {
      leave_item(i);
      const int sb = a.first ? 0 : it.b, S = a.first ? 1 : c.B;
      for (int s = 0; ok && s < p.subs; ++s) {
        const float* lse = a.lse + ((static_cast<size_t>(it.l) * S + sb) * c.H * a.G + it.h * a.G + s * p.P) * a.n +
                           it.first;
        for (int ch = it.c0; ch < it.chunks; ++ch) {
          float y[kChunk / 32];
          const int j0 = ch * p.tok;
#pragma unroll
          for (int k = 0; k < kChunk / 32; ++k)
            y[k] = j[k] < it.nq - j0 ? lse[static_cast<size_t>(g[k]) * a.n + j0 + j[k]] : INFINITY;
          const int st = use % NS, sy = use % kSums;
          auto blind = [&](int k) { return sees_nothing(y[k]) && j[k] < it.nq - j0; };
          bool any = false;
#pragma unroll
          for (int k = 0; k < kChunk / 32; ++k) any = any || blind(k);
          any = __any_sync(0xffffffffu, any);
          if (!(ok = warp_wait(&q_empty[st], ((use / NS) & 1) ^ 1, abort, c.status))) break;
          if (lane == 0) {
            uint64_t* full = any ? odd_full : &q_full[st];
            mbar_arrive_expect_tx(full, DB * p.P * p.tok * 128);
            for (int x = 0; x < DB; ++x)
              tma_load_5d(smem + Sm::kRing + st * Sm::kStage + x * kQueryBlock, &map_q, 64 * x,
                          (it.h * a.G + s * p.P) * p.q_head, it.first + j0, a.first ? 0 : it.b * p.q_seq,
                          it.l * p.q_layer, full);
          }
          __syncwarp();
          if (any) {
            volatile int never = 0;  // (the copy lands before the CTA ends)
            if (!(ok = warp_wait(odd_full, odd++ & 1, &never, c.status))) {
              *abort = 1;
              break;
            }
#pragma unroll
            for (int k = 0; k < kChunk / 32; ++k)
              if (blind(k))
                for (int x = 0; x < DB * 8; ++x)
                  *reinterpret_cast<uint4*>(smem + Sm::kRing + st * Sm::kStage + x / 8 * kQueryBlock +
                                            (lane + 32 * k) * 128 + x % 8 * 16) = make_uint4(0, 0, 0, 0);
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[st]);
          }
          ++use;
          if (!(ok = warp_wait(&y_empty[sy], (((use - 1) / kSums) & 1) ^ 1, abort, c.status))) break;
#pragma unroll
          for (int k = 0; k < kChunk / 32; ++k) s_sums[sy * kChunk + lane + 32 * k] = -lse_base2(y[k]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&y_full[sy]);
        }
      }
    }
    volatile int never = 0;  // every copy has landed before the CTA ends
    for (uint32_t u = use > NS ? use - NS : 0; u < use; ++u)
      mbar_wait(&q_full[u % NS], (u / NS) & 1, &never, c.status);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ products
    // (all lanes run the loop and wait converged)
    const bool lead = lane == 0;
    const uint32_t base = smem_u32(smem);
    uint32_t use = 0;
    int steps[2] = {0, 0};
    bool ok = true;
    Item it;
    for (int i = 0; ok && read_item(i, it); ++i) {
      leave_item(i);
      const int per_sub = it.chunks - it.c0;
      for (int s = 0; ok && s < p.subs; ++s)
        for (int ch = it.c0; ok && ch < it.chunks; ++ch, ++use) {
          const int st = use % NS;
          if (!(ok = warp_wait(&q_full[st], (use / NS) & 1, abort, c.status))) break;
          const bool begins = s == 0 && ch == it.c0, ends = s + 1 == p.subs && ch + 1 == it.chunks;
          const int n = (min(it.nq - ch * p.tok, p.tok) * p.P + 15) & ~15;  // columns
          const uint32_t idesc = idesc_bf16_f32(kTile, n);
          const uint32_t q_low = desc_low(base + Sm::kRing + st * Sm::kStage, 16);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok) continue;
            if (begins && !(ok = warp_wait(&k_full[t], i & 1, abort, c.status))) continue;
            if (t == 0 || ch >= it.c1) {
              if (!(ok = warp_wait(&s_empty[t], (steps[t] & 1) ^ 1, abort, c.status))) continue;
              ++steps[t];
              tc_fence_after();
#pragma unroll
              for (int x = 0; x < D / 16; ++x)
                mma_ts_if(lead, tmem + t * kChunk, tmem + kKeyCol + t * (D / 2) + x * 8,
                          q_low + (((x / 4) * kQueryBlock + (x % 4) * 32) >> 4), idesc, x > 0);
              commit_if(lead, &s_full[t]);
            }
            if (ends) commit_if(lead, &k_empty[t]);
          }
          if (ok) commit_if(lead, &q_empty[st]);
        }
      if (ok && per_sub <= 0) {  // no queries: the keys are done with at once
        for (int t = 0; t < 2; ++t) {
          if (!(ok = warp_wait(&k_full[t], i & 1, abort, c.status))) break;
          if (lane == 0) mbar_arrive(&k_empty[t]);
        }
      }
    }
    if (lane == 0) mma_commit(done);
    __syncwarp();
    volatile int never = 0;  // also after an abort: what was issued ends
    mbar_wait(done, 0, &never, c.status);
  } else {
    // ------------------------------------------------------------ items
    const int total = s_upto[groups - 1] * units;  // below 2^31: checked on the host
    for (int i = 0;; ++i) {
      if (!warp_wait(&i_empty[i % kItems], ((i / kItems) & 1) ^ 1, abort, c.status)) break;
      // rounds go back and forth over the CTAs
      const long long k = static_cast<long long>(i) * gridDim.x +
                          (i & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      Item it = {};
      if (k < total) {
        const int at = static_cast<int>(k / units), unit = static_cast<int>(k % units);
        int q = 0;  // the first place with s_upto[q] > at
        for (int q0 = 0; q0 < groups; q0 += 32) {
          const bool below = q0 + lane < groups && s_upto[q0 + lane] <= at;
          const int n = __popc(__ballot_sync(0xffffffffu, below));
          q += n;
          if (n < 32) break;
        }
        const int in = at - (q ? s_upto[q - 1] : 0);
        int x;  // pairs behind this one
        if (per == 1) {
          x = s_count[q] - 1 - in / (q + 1);
          it.b = s_seq[in % (q + 1)];
        } else {
          it.b = s_seq[q] * per;
          x = in;
          for (int n = pairs_of(it.b); x >= n; n = pairs_of(++it.b)) x -= n;
        }
        const Lengths n = lengths_of(c, a, it.b, &bad);
        it.len = n.len;
        it.nq = n.nq;
        it.first = n.first;
        it.part = unit % p.parts;
        it.l = unit / p.parts / c.H;
        it.h = unit / p.parts % c.H;
        it.t0 = (div_up(n.len, 2 * kTile) - 1 - x) * 2 * kTile;
        it.chunks = div_up(n.nq, p.tok);
        const int start = n.len - n.nq;  // the first query's token
        it.c0 = min(max(it.t0 - start, 0) / p.tok, it.chunks);
        it.c1 = it.t0 + kTile < n.len ? min(max(it.t0 + kTile - start, 0) / p.tok, it.chunks) : it.chunks;
        if (p.parts > 1) {  // this part's share of the chunks
          const int n_ch = it.chunks - it.c0, lo = it.c0;
          it.c0 = lo + n_ch * it.part / p.parts;
          it.chunks = lo + n_ch * (it.part + 1) / p.parts;
        }
        it.there = 1;
      }
      if (lane == 0) {
        items[i % kItems] = it;
        mbar_arrive(&i_full[i % kItems]);
      }
      __syncwarp();
      if (!it.there) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
#endif
}

// Adds the parts of items up, in their order.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) weigh_join_kernel(Cache c, Params p) {
  before_all();
  const WeighArgs& a = p.a;
  const int pair = blockIdx.x % p.pairs, u = blockIdx.x / p.pairs;
  const int b = u / c.H % c.B, token = pair * 2 * kTile + threadIdx.x;
  bool bad = false;
  if (token >= lengths_of(c, a, b, &bad).len) return;
  const float* part = p.part + static_cast<size_t>(blockIdx.x) * p.parts * (2 * kTile) + threadIdx.x;
  float* w = a.w + static_cast<size_t>(u) * a.cap + token;
  const float old = a.decay != 0.f ? a.decay * *w : 0.f;
  float sum = 0.f;
#pragma unroll 4
  for (int s = 0; s < p.parts; ++s) sum += part[s * 2 * kTile];
  *w = sum < 0.f ? old : old + sum;
}
static_assert(kJoinThreads == 2 * kTile, "a thread for each token of a pair of tiles");

template <int D, int FMT>
cudaError_t launch_d(const Cache& c, const WeighArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> told{0};
  cudaError_t e = allow_smem(weigh_many_kernel<D, FMT>, Smem<D>::kBytes, told);
  if (e != cudaSuccess) return e;
  Params p;
  p.a = a;
  p.P = a.G;
  if (a.G > kPacked)
    for (p.P = kPacked; a.G % p.P; --p.P) {
    }
  p.subs = a.G / p.P;
  p.tok = kChunk / p.P;
  // x = 64 values, y = head, z = token, then sequence and layer, in boxes of one block of values
  // by P heads by tok tokens.  An axis whose stride is 0 counts as one.
  EncodeTiledFn enc = tensor_map_encoder(nullptr);
  if (!enc) return cudaErrorNotSupported;
  const int seqs = a.first ? 1 : c.B, heads = c.H * a.G;
  p.q_head = heads > 1;
  p.q_seq = seqs > 1 && a.q.seq > 0;
  p.q_layer = c.L > 1 && a.q.layer > 0;
  auto bytes = [](long long stride, bool used) { return static_cast<cuuint64_t>(used ? stride * 2 : 256); };
  const cuuint64_t dims[5] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(a.n), static_cast<cuuint64_t>(p.q_seq ? seqs : 1),
                              static_cast<cuuint64_t>(p.q_layer ? c.L : 1)};
  const cuuint64_t strides[4] = {bytes(a.q.head, p.q_head), bytes(a.q.token, a.n > 1),
                                 bytes(a.q.seq, p.q_seq), bytes(a.q.layer, p.q_layer)};
  const cuuint32_t box[5] = {64, static_cast<cuuint32_t>(p.P), static_cast<cuuint32_t>(p.tok), 1, 1};
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  CUtensorMap q;
  if (enc(&q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, a.q.data, dims, strides, box, one,
          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  // Where there are few pairs of tiles, their queries are cut into parts of 8 chunks and more, for
  // two items an SM, which a second launch adds up.  Both numbers are upper bounds, since the lengths are
  // on the device: pairs from the room of cap and table, chunks from all rows of a packed call, whose
  // sequences may have fewer (parts may be empty then).  Prompts of 1536 tokens, whole and cut: 24
  // pairs 82 and 24 us, 96 pairs 82 and 48, 192 pairs 85 and 82, but 288 pairs 105 and 113; and
  // parts of less cost more than they save (64 queries, 192 pairs: 18 and 22 us).  With more room than
  // tokens there are fewer parts (1 x 1536 tokens, 24 pairs: 24 us with cap 1536, 38 with 8192, 83 with
  // 32768).
  const int tokens = min(a.cap, c.max_blocks * c.bs);
  p.pairs = (tokens + 2 * kTile - 1) / (2 * kTile);
  const long long most = static_cast<long long>(c.L) * c.B * c.H * p.pairs;
  const int chunks = (a.n + p.tok - 1) / p.tok;
  p.parts = 1;
  if (2 * most < 3ll * a.num_sms)
    p.parts = static_cast<int>(max(1ll, min(2ll * a.num_sms / most + 1, min(chunks / 8ll, 16ll))));
  p.part = static_cast<float*>(a.workspace);
  const long long items = most * p.parts;
  const int grid = static_cast<int>(items < a.num_sms ? items : a.num_sms);
  e = launch(weigh_many_kernel<D, FMT>, grid, kThreads, Smem<D>::kBytes, s, q, c, p, make_div(c.bs));
  if (e != cudaSuccess || p.parts == 1) return e;
  return launch(weigh_join_kernel, static_cast<int>(most), kJoinThreads, 0, s, c, p);
}

}  // namespace

cudaError_t launch_weigh_many(const Cache& c, int format, const WeighArgs& a, cudaStream_t s) {
  if (c.d == 64)
    return format == KVC_CACHE8_E4M3 ? launch_d<64, KVC_CACHE8_E4M3>(c, a, s)
                                     : launch_d<64, KVC_CACHE8_INT8>(c, a, s);
  return format == KVC_CACHE8_E4M3 ? launch_d<128, KVC_CACHE8_E4M3>(c, a, s)
                                   : launch_d<128, KVC_CACHE8_INT8>(c, a, s);
}

}  // namespace prompt
}  // namespace kvc
