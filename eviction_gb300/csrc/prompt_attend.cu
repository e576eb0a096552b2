// prompt_attend.cu -- causal attention over whole prompts (kvc_prompt_attend), on the
// 5th-generation tensor cores (tcgen05 + TMEM) with TMA-staged operands.
//
//   out_j = sum_t w_jt v_t / sum_t w_jt,  w_jt = exp(scale q_j . k_t), t <= j
//
// The heads of a group share their keys and values: a tile of 128 rows is up to 16 heads
// by the tokens that fit beside them (row = token * P + head), so that short prompts fill
// it and a group's keys are read once.  A CTA has two such tiles, of consecutive tokens,
// and takes 128 keys and values at a time for both:
//   load (1 warp)     Q, K and V by TMA, keys and values through a ring of stages;
//   MMA (2 warps)     a warp a tile: S = Q K^T (128 x 128, in TMEM), then O += P V with P read
//                     from TMEM, where it has taken the place of S; the tiles take turns, so
//                     that one tile's products run during the other's softmax;
//   softmax (4 + 4 warps)  one thread a row: weights, their sum in fp32, P to TMEM as bf16,
//                     and at the end the row's result;
//   items (1 warp)    which tiles come next, a few ahead of the others.
// P is rounded to bf16 because V is bf16 (both operands of a product have one type): half
// a step of 2^-8 a weight, less than that in their sum, which is taken before rounding.
// bf16 has fp32's exponents: a weight may lie above 1, so that the reference m of a row,
// its first tile's largest logit, moves only when a later one passes it by 14 in base 2 (and O is
// scaled then, by the softmax warps themselves).  O holds sums of weights times values before they
// are divided: what weights may grow by is missing there (at 2^32 values of 8e28 were too large).
// Less room costs more moves: 16384 tokens with keys and queries of uneven length 1282 us with 20
// or 32, 1298 with 14, 1340 with 8.  The maximum comes with the TMEM load.
//
// The arithmetic bounds this: 4 d operations a pair of tokens and head.  Measured, d = 128: one
// sequence of 16384 tokens, 28 heads, 1.31 ms in a row (1470 TFLOP/s; power holds the clocks down) and
// 1.21 ms in runs of a few (1590; a step of both tiles 3000 cycles, its 32 products alone 2048:
// S = Q K^T reads both operands at all of shared memory's bandwidth, beside the copies); 16 sequences
// of 612 to 1112 tokens, 32 heads, 108 us back to back in a graph, 113 as calls, a quarter of it the
// changes of items (a result written beside the next item's products slows those more than it hides: 111
// us, of 106 then).  The last tile of keys is cut to the columns (steps of 16) that some row of the tile
// sees, in both products.
// Rows of V behind a sequence's end are zeroed in shared memory first (their weights are
// 0, and what stands there need not be finite).
//
// Work: pairs of tiles of all sequences and KV heads, those with most keys first, dealt to
// one CTA per SM in turns (back and forth), which leaves the CTAs' shares within about
// one small item of one another.  Every wait is bounded.
#include <atomic>
#include <climits>

#include "cache8_attend.cuh"
#include "prompt.cuh"

namespace kvc {
namespace prompt {
namespace {

using cache8::before_all;
using cache8::bf16x2;
using cache8::div_up;

constexpr int kRows = 128, kTokens = 128;  // rows of a tile, keys of a step
constexpr int kSoftmaxWarps = 8;           // 4 a tile
constexpr int kMmaWarp = 8, kLoadWarp = 10, kItemWarp = 11;  // (two warps issue products)
constexpr int kThreads = 32 * 12;
constexpr int kItems = 4;        // items told ahead
constexpr int kReaders = kSoftmaxWarps + 3;
constexpr int kSorted = 128;     // sequences (or groups of them) in the list of items
constexpr int kPacked = 16;      // heads in a tile at most
constexpr float kRoom = 14.f;    // log2 of the largest weight
// A row's weights are 2^(s f - r), r = m f rounded, m the largest score so far: all of them are off by
// the factor that r is rounded by, which the sum takes out again, but from |r| = 2^30 on it is
// infinite or zero.  From 2^29 on f is a power of two instead: r is exact then, and scores
// that are not the same are 64 apart in base 2, 42 with that f, so that weights are 1 or nothing.
constexpr float kExactRef = 536870912.f;
// Registers: 168 a thread at launch, moved to where a row of S is held.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "more registers than the block has");

struct Params {
  AttendArgs a;
  int P, subs, tok;            // heads in a tile, such tiles of a group, tokens of a tile
  int k_head, v_head, q_head;  // 0 where all heads are one (stride 0)
  int k_seq, v_seq, q_seq;
};

struct Item {
  int row0, sb;     // the sequence's first row; its index where rows have one
  int h, hq;        // KV head, first query head
  int len, t0;      // tokens of the sequence, first token of tile 0
  int steps[2];     // of 128 keys, of each tile; 0: no more items
  __device__ __forceinline__ int of(int t) const { return t ? steps[1] : steps[0]; }
};

template <int D>
struct Smem {
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kQ = 0, kRing = 2 * kTile, kOut = kRing + kStages * kTile,
                       kBars = kOut + kSoftmaxWarps * 4096,
                       kNumBars = 2 * kStages + 12 + 2 * kItems + 1,
                       kItem = (kBars + kNumBars * 8 + 15) & ~15, kMisc = kItem + kItems * 32,
                       kUpTo = kMisc + 16, kCount = kUpTo + (kSorted + 1) * 4,
                       kSeq = kCount + (kSorted + 1) * 4, kBytes = kSeq + kSorted + 1024;
  static_assert(kBytes <= 232448, "shared memory of a block");
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}

// Tokens of sequence b, 0 where it does not lie within its rows.
__device__ __forceinline__ int length_of(const AttendArgs& a, int b, bool* bad) {
  const int m = a.n_tok ? a.n_tok[b] : a.n, first = a.first ? a.first[b] : 0;
  if (m < 0 || first < 0 || m > a.n - first) {
    *bad = true;
    return 0;
  }
  return m;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attend_kernel(const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, Params p) {
#if defined(__CUDA_ARCH__) && (__CUDA_ARCH__ >= 1000)
  using Sm = Smem<D>;
  constexpr int DB = D / 64;             // 64-value blocks (128 bytes) of a row
  constexpr int kBlock = 128 * 128;      // bytes of one block of all rows
  constexpr int NS = Sm::kStages;
  constexpr uint32_t kOutCol = 256;      // O's first TMEM columns, after the two of S
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sm::kBars);
  uint64_t *kv_full = bars, *kv_empty = bars + NS, *q_full = bars + 2 * NS, *q_empty = q_full + 2,
           *s_full = q_empty + 2, *p_full = s_full + 2, *o_full = p_full + 2, *turn = o_full + 2, *i_full = turn + 2,
           *i_empty = i_full + kItems, *done = bars + Sm::kNumBars - 1;
  Item* items = reinterpret_cast<Item*>(smem + Sm::kItem);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Sm::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + Sm::kMisc + 4);
  int* s_upto = reinterpret_cast<int*>(smem + Sm::kUpTo);
  int* s_count = reinterpret_cast<int*>(smem + Sm::kCount);
  uint8_t* s_seq = smem + Sm::kSeq;
  const AttendArgs& a = p.a;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_empty[t], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_full[t], 1);
      mbar_init(&turn[t], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&i_full[i], 1);
      mbar_init(&i_empty[i], kReaders);
    }
    mbar_init(done, 2);
    *abort = 0;
    fence_barrier_init();
    prefetch_tensormap(&map_q);
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
  }
  before_all();

  // ---- the list of items: groups of `per` sequences (one each, if they are few enough;
  // those with most pairs of tiles first then) ----
  const int Hv = a.H * p.subs;  // (KV head, part of its group)
  const int per = div_up(a.S, kSorted), groups = div_up(a.S, per);
  bool bad = false;
  auto pairs_of = [&](int b) { return div_up(length_of(a, b, &bad), 2 * p.tok); };
  if (threadIdx.x < kSorted) {
    long long n = 0;
    for (int b = threadIdx.x * per; b < min((static_cast<int>(threadIdx.x) + 1) * per, a.S); ++b)
      n += pairs_of(b);
    s_upto[threadIdx.x] = static_cast<int>(min(n, 1ll << 30));
    if (bad && blockIdx.x == 0) atomicOr(a.status, KVC_STATUS_BAD_INDEX);
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (threadIdx.x < groups) {  // its place: by the count, then by the number
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
  // s_upto[q]: items of a head among those of the levels (tile pairs x, x + 1, ... of all
  // sequences that have them) that more than q sequences do not reach; or, of groups
  // of several sequences, of groups 0 .. q
  if (warp == kItemWarp) {
    long long before = 0;
    for (int q0 = 0; q0 < groups; q0 += 32) {
      const int q = q0 + lane;
      long long incl = q < groups ? s_count[q] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      incl += before;
      if (q < groups)
        s_upto[q] = static_cast<int>(per > 1 ? incl : incl - (q + 1ll) * s_count[q + 1]);
      before = __shfl_sync(0xffffffffu, incl, 31);
    }
    // (sequences that overlap may claim more rows than there are: nothing is done then)
    if (before > INT_MAX / Hv) {
      if (lane == 0 && blockIdx.x == 0) atomicOr(a.status, KVC_STATUS_BAD_INDEX);
      if (lane == 0) s_upto[groups - 1] = 0;
    }
    __syncwarp();
  }

  // Item i of this CTA, as the item warp tells it; steps[1] = 0: there is none.
  auto read_item = [&](int i, Item& it) {
    if (!warp_wait(&i_full[i % kItems], (i / kItems) & 1, abort, a.status)) return false;
    it = items[i % kItems];
    return true;
  };
  auto leave_item = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&i_empty[i % kItems]);
  };

  if (warp < kSoftmaxWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------------------ softmax
    const int t = warp / 4;  // tile
    const int row = threadIdx.x % 128;
    const int row_token = row / p.P, row_head = row - row_token * p.P;
    const int warp_token0 = __shfl_sync(0xffffffffu, row_token, 0),
              warp_token1 = __shfl_sync(0xffffffffu, row_token, 31);  // of the warp's rows
    const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16;
    const uint32_t s_tmem = tmem + lanes + t * 128, o_tmem = tmem + lanes + kOutCol + t * D;
    const float f = a.scale_log2;  // and the power of two next to it
    const float near_f = __uint_as_float((__float_as_uint(f) + 0x400000u) & 0x7f800000u);
    int step = 0;  // of all items
    Item it;
    for (int i = 0; read_item(i, it) && it.steps[1] > 0; ++i) {
      leave_item(i);
      const int n_steps = it.of(t), t0 = it.t0 + t * p.tok;
      const int token = t0 + row_token;     // this row's token, and the last that it sees
      const int first_token = t0 + warp_token0, last_token = t0 + warp_token1;
      float m = -INFINITY, sum = 0.f;       // score that the weights refer to, their sum
      float own_f = f;
      bool ok = true;
      for (int j = 0; j < n_steps; ++j, ++step) {
        if (!warp_wait(&s_full[t], step & 1, abort, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t v[4][32];
        float mx[4];
        const int c0 = j * kTokens;
        if (c0 + kTokens - 1 <= first_token) {  // all rows of the warp see all of it
#pragma unroll
          for (int k = 0; k < 4; ++k) tmem_ld32_max(s_tmem + 32 * k, v[k], mx[k]);
          tmem_ld_wait();
        } else {
          const int seen = token - c0 + 1;  // columns that this row sees
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            mx[k] = -INFINITY;
            if (c0 + 32 * k + 31 <= first_token) {
              tmem_ld32_max(s_tmem + 32 * k, v[k], mx[k]);
              tmem_ld_wait();
            } else if (c0 + 32 * k <= last_token) {
              tmem_ld32(s_tmem + 32 * k, v[k]);
              tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 32; ++x) {
                if (32 * k + x >= seen) v[k][x] = 0xff800000u;  // -inf
                mx[k] = fmaxf(mx[k], __uint_as_float(v[k][x]));
              }
            } else {  // none of them
#pragma unroll
              for (int x = 0; x < 32; ++x) v[k][x] = 0xff800000u;
            }
          }
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const bool raise = (top - m) * f > kRoom;
        if (__any_sync(0xffffffffu, raise)) {
          const float keep = raise ? ex2((m - top) * f) : 1.f;
          if (raise) {
            m = top;
            own_f = fabsf(top * f) < kExactRef ? f : near_f;
          }
          sum *= keep;
          if (j > 0) {  // what is there is scaled to the new references (the last step's product
                        // was issued before these scores: it is done)
#pragma unroll 1
            for (int k = 0; k < D / 16; ++k) {
              uint32_t o[16];
              tmem_ld16(o_tmem + k * 16, o);
              tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * keep);
              tmem_st16(o_tmem + k * 16, o);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : __fmul_rn(m, own_f);
        const float2 ff = make_float2(own_f, own_f), off = make_float2(-ref, -ref);
        float2 part = make_float2(0.f, 0.f);
        uint32_t w[4][16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float2 z = fma2(make_float2(__uint_as_float(v[k][2 * x]), __uint_as_float(v[k][2 * x + 1])),
                            ff, off);
            z.x = ex2(z.x);
            z.y = ex2(z.y);
            part = add2(part, z);
            w[k][x] = bf16x2(z.x, z.y);
          }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_st16(s_tmem + 16 * k, w[k]);
        sum += part.x + part.y;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      if (!ok) break;
      // ---- the result ----
      if (!warp_wait(&o_full[t], i & 1, abort, a.status)) break;
      tc_fence_after();
      const bool there = row_token < p.tok && token < it.len;
      const float inv = 1.f / sum;
      // 64 values of the warp's rows at a time through shared memory, so that a store
      // writes whole lines of 4 rows (each thread its own row, 16 bytes of 32 rows a store:
      // 6000 cycles a tile)
      const uint64_t out = there ? reinterpret_cast<uint64_t>(
                                       a.out.at(0, it.sb, it.hq + row_head, it.row0 + token))
                                 : 0;
      uint8_t* stage = smem + Sm::kOut + warp * 4096;
      uint32_t o[DB][2][32];
#pragma unroll
      for (int h = 0; h < DB; ++h)
#pragma unroll
        for (int k = 0; k < 2; ++k) tmem_ld32(o_tmem + 64 * h + 32 * k, o[h][k]);
      tmem_ld_wait();
#pragma unroll
      for (int h = 0; h < DB; ++h) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            float y[8];
#pragma unroll
            for (int z = 0; z < 8; ++z) y[z] = __uint_as_float(o[h][k][8 * x + z]) * inv;
            *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * k + x) ^ (lane & 7)) << 4)) =
                make_uint4(bf16x2(y[0], y[1]), bf16x2(y[2], y[3]), bf16x2(y[4], y[5]), bf16x2(y[6], y[7]));
          }
        __syncwarp();
        uint4 y[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int r = 4 * x + lane / 8;
          y[x] = *reinterpret_cast<const uint4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const uint64_t to = __shfl_sync(0xffffffffu, out, 4 * x + lane / 8);
          if (to) reinterpret_cast<uint4*>(to)[8 * h + (lane & 7)] = y[x];
        }
        __syncwarp();
      }
      if (there && a.lse)
        a.lse[(static_cast<size_t>(it.sb) * a.H * a.G + it.hq + row_head) * a.n + it.row0 + token] =
            (__fmul_rn(m, f) + __log2f(sum)) * 0.6931471805599453f;
      tc_fence_before();  // (the next item's P is told after this: O may be written again then)
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == kMmaWarp || warp == kMmaWarp + 1) {
      // ------------------------------------------------------------ products
      // A warp for each tile: the tensor pipe takes a product only when the one ahead of it
      // has begun, so that a single warp's waits (100 cycles each) left it idle.  The tiles
      // take turns, a step's products and the next one's scores at a time: where both issued
      // as they liked, they fell into step, products of both, then softmax of both (3780
      // cycles a step of both tiles; the products alone are 2048).  All that a turn needs is
      // waited for before it, and it is passed on a few products before its end.
      // (All lanes run the loop and wait converged.)
      const int t = warp - kMmaWarp;
      const uint32_t base = smem_u32(smem);
      const bool lead = lane == 0;
      const uint32_t s_tmem = tmem + t * 128, o_tmem = tmem + kOutCol + t * D;
      const uint32_t q_low = desc_low(base + Sm::kQ + t * Sm::kTile, 16);
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_test(bar, parity)) || warp_wait(bar, parity, abort, a.status);
      };
      // 16s of columns that some row of the tile sees in a step
      auto cols_of = [&](const Item& it, int j) {
        if (j + 1 < it.of(t)) return kTokens / 16;
        const int end = min(it.t0 + (t + 1) * p.tok, it.len) - j * kTokens;
        return (end + 15) >> 4;
      };
      int st = 0;            // the next stage, and its uses' parity
      uint32_t st_parity = 0;
      auto take = [&](int* stage) {
        const bool ok = wait(&kv_full[st], st_parity);
        *stage = st;
        if (++st == NS) st = 0, st_parity ^= 1;
        return ok;
      };
      auto scores = [&](int stage, int n, bool end) {  // S = Q K^T
        const uint32_t idesc = idesc_bf16_f32(kRows, 0) | static_cast<uint32_t>(n) << 18;
        const uint32_t k = desc_low(base + Sm::kRing + stage * Sm::kTile, 16);
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const uint32_t off = ((x / 4) * kBlock + (x % 4) * 32) >> 4;
          mma_ss_if(lead, s_tmem, q_low + off, k + off, idesc, x > 0);
          if (x == D / 16 - 3 && lead) mbar_arrive(&turn[t ^ 1]);
        }
        commit_if(lead, &s_full[t]);
        commit_if(lead, &kv_empty[stage]);
        if (end) commit_if(lead, &q_empty[t]);
      };
      uint32_t p_parity = 0, turn_parity = t ^ 1;
      auto my_turn = [&]() {
        const bool ok = wait(&turn[t], turn_parity);
        turn_parity ^= 1;
        tc_fence_after();
        return ok;
      };
      Item it, next;
      int ks, vs;  // stages of keys, of values
      bool ok = read_item(0, it) && it.steps[1] > 0 && wait(&q_full[t], 0) && take(&ks) && my_turn();
      if (ok) scores(ks, cols_of(it, 0), it.of(t) == 1);
      for (int i = 0; ok; ++i) {
        const int steps = it.of(t);
        for (int j = 0; ok && j < it.steps[1]; ++j) {
          const bool last = j + 1 == it.steps[1], own_last = j + 1 == steps;
          if (last) {
            ok = read_item(i + 1, next);
            leave_item(i);
            if (!ok) break;
          }
          const bool more = !last || next.steps[1] > 0;
          // all that this turn needs
          ok = take(&vs);
          const int n = cols_of(it, j), rows = it.len - j * kTokens;
          if (ok && j < steps && rows < 16 * n) {
            // rows of V behind the sequence, up to the last step of 16, are zeroed (by both warps)
            uint8_t* v = smem + Sm::kRing + vs * Sm::kTile;
            for (int x = lane; x < (16 * n - rows) * (D / 8); x += 32)
              *reinterpret_cast<uint4*>(v + (x % (D / 8) / 8) * kBlock + (rows + x / (D / 8)) * 128 +
                                        x % 8 * 16) = make_uint4(0, 0, 0, 0);
            fence_async_shared();
            __syncwarp();
          }
          ok = ok && (!more || take(&ks)) && (!(last && more) || wait(&q_full[t], (i + 1) & 1));
          if (ok && j < steps) {
            ok = wait(&p_full[t], p_parity);
            p_parity ^= 1;
          }
          if (!ok || !my_turn()) {
            ok = false;
            break;
          }
          if (j < steps) {  // O += P V
            constexpr uint32_t idesc = idesc_bf16_f32(kRows, D) | 1u << 16;
            const uint32_t v = desc_low(base + Sm::kRing + vs * Sm::kTile, kBlock);
#pragma unroll
            for (int x = 0; x < kTokens / 16; ++x)
              mma_ts_if(lead && x < n, o_tmem, s_tmem + x * 8, v + x * (2048 >> 4), idesc, j > 0 || x > 0);
            commit_if(lead, &kv_empty[vs]);
            if (own_last) commit_if(lead, &o_full[t]);
          } else if (lead) {
            mbar_arrive(&kv_empty[vs]);
          }
          if (j + 1 < steps) {
            scores(ks, cols_of(it, j + 1), j + 2 == steps);
          } else if (last && more) {
            scores(ks, cols_of(next, 0), next.of(t) == 1);
          } else if (lead) {  // no scores in this turn
            mbar_arrive(&turn[t ^ 1]);
            if (more) mbar_arrive(&kv_empty[ks]);
          }
        }
        if (!ok || next.steps[1] == 0) break;
        it = next;
      }
      if (lane == 0) mma_commit(done);
      __syncwarp();
      volatile int never = 0;  // also after an abort: what was issued ends
      mbar_wait(done, 0, &never, a.status);
    } else if (warp == kLoadWarp) {
      // ------------------------------------------------------------ loads
      int use = 0, n_q = 0;
      bool ok = true;
      Item it;
      for (int i = 0; ok && read_item(i, it) && it.steps[1] > 0; ++i) {
        leave_item(i);
        auto load = [&](const CUtensorMap* map, int j, int head, int seq) {
          const int s = use % NS;
          if (!warp_wait(&kv_empty[s], ((use / NS) & 1) ^ 1, abort, a.status)) return false;
          ++use;
          if (lane == 0) {
            mbar_arrive_expect_tx(&kv_full[s], Sm::kTile);
            tma_load_5d(smem + Sm::kRing + s * Sm::kTile, map, 0, it.row0 + j * kTokens, 0, head, seq,
                        &kv_full[s]);
          }
          __syncwarp();
          return true;
        };
        for (int j = 0; ok && j < it.steps[1]; ++j) {
          ok = load(&map_k, j, it.h * p.k_head, it.sb * p.k_seq);
          if (ok && j == 0) {
            for (int t = 0; ok && t < 2; ++t) {
              ok = warp_wait(&q_empty[t], (n_q & 1) ^ 1, abort, a.status);
              if (ok && lane == 0) {
                mbar_arrive_expect_tx(&q_full[t], DB * p.P * p.tok * 128);
                for (int x = 0; x < DB; ++x)
                  tma_load_5d(smem + Sm::kQ + t * Sm::kTile + x * kBlock, &map_q, 64 * x,
                              it.hq * p.q_head, it.row0 + it.t0 + t * p.tok, it.sb * p.q_seq, 0, &q_full[t]);
              }
              __syncwarp();
              if (!ok && t == 1) {  // tile 0's is on its way
                volatile int never = 0;
                mbar_wait(&q_full[0], n_q & 1, &never, a.status);
              }
            }
            if (ok) ++n_q;
          }
          if (ok) ok = load(&map_v, j, it.h * p.v_head, it.sb * p.v_seq);
        }
      }
      // every copy has landed before the CTA ends
      volatile int never = 0;
      for (int u = max(use - NS, 0); u < use; ++u)
        mbar_wait(&kv_full[u % NS], (u / NS) & 1, &never, a.status);
      for (int t = 0; t < 2; ++t)
        if (n_q > 0) mbar_wait(&q_full[t], (n_q - 1) & 1, &never, a.status);
    } else if (warp == kItemWarp) {
      // ------------------------------------------------------------ items
      const int total = s_upto[groups - 1] * Hv;
      for (int i = 0;; ++i) {
        if (!warp_wait(&i_empty[i % kItems], ((i / kItems) & 1) ^ 1, abort, a.status)) break;
        // rounds go back and forth over the CTAs
        const long long k = static_cast<long long>(i) * gridDim.x +
                            (i & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        Item it = {};
        if (k < total) {
          const int at = static_cast<int>(k / Hv), hv = static_cast<int>(k % Hv);
          int q = 0;  // the first place with s_upto[q] > at
          for (int q0 = 0; q0 < groups; q0 += 32) {
            const bool below = q0 + lane < groups && s_upto[q0 + lane] <= at;
            const int n = __popc(__ballot_sync(0xffffffffu, below));
            q += n;
            if (n < 32) break;
          }
          const int in = at - (q ? s_upto[q - 1] : 0);
          int b, x;
          if (per == 1) {  // levels of q + 1 sequences, from the highest
            x = s_count[q] - 1 - in / (q + 1);
            b = s_seq[in % (q + 1)];
          } else {
            b = s_seq[q] * per;
            x = in;
            for (int n = pairs_of(b); x >= n; n = pairs_of(++b)) x -= n;
          }
          it.len = length_of(a, b, &bad);
          it.row0 = a.first ? a.first[b] : 0;
          it.sb = a.first ? 0 : b;
          it.h = hv / p.subs;
          it.hq = it.h * a.G + hv % p.subs * p.P;
          it.t0 = x * 2 * p.tok;
          const int last0 = min(it.t0 + p.tok, it.len) - 1, last1 = min(it.t0 + 2 * p.tok, it.len) - 1;
          it.steps[0] = last0 / kTokens + 1;
          it.steps[1] = last1 / kTokens + 1;
        }
        if (lane == 0) {
          items[i % kItems] = it;
          mbar_arrive(&i_full[i % kItems]);
        }
        __syncwarp();
        if (it.steps[1] == 0) break;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
#endif
}

// Rows of 64-value blocks as TMA reads them.  Keys and values: x = 64 values, y = token,
// z = block, then head and sequence, in boxes of 128 tokens and all blocks.  Queries: x = values,
// y = head, z = token, then sequence, in boxes of one block of `heads` by `tokens` rows.
// An axis whose stride is 0 counts as one.
bool make_map(CUtensorMap* m, const Rows& r, bool queries, int d, int heads_all, int n, int seqs,
              int heads, int tokens, int* head_mul, int* seq_mul) {
  EncodeTiledFn enc = tensor_map_encoder(nullptr);
  if (!enc) return false;
  *head_mul = heads_all > 1 && r.head > 0;
  *seq_mul = seqs > 1 && r.seq > 0;
  const cuuint64_t H = *head_mul ? heads_all : 1, S = *seq_mul ? seqs : 1;
  auto bytes = [](long long stride, bool used) {
    return static_cast<cuuint64_t>(used ? stride * 2 : 256);
  };
  const cuuint64_t head = bytes(r.head, *head_mul), seq = bytes(r.seq, *seq_mul),
                   token = bytes(r.token, n > 1), N = n;
  cuuint64_t dims[5] = {64, N, static_cast<cuuint64_t>(d / 64), H, S}, strides[4] = {token, 128, head, seq};
  cuuint32_t box[5] = {64, 128, static_cast<cuuint32_t>(d / 64), 1, 1}, one[5] = {1, 1, 1, 1, 1};
  if (queries) {
    dims[0] = d, dims[1] = H, dims[2] = N, dims[3] = S, dims[4] = 1;
    strides[0] = head, strides[1] = token, strides[2] = seq, strides[3] = 256;
    box[1] = heads, box[2] = tokens, box[3] = 1;
  }
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, r.data, dims, strides, box, one,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_d(const AttendArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> told{0};
  if (!told.load(std::memory_order_relaxed)) {  // the registers that the warps share out have to be there
    cudaFuncAttributes has;
    const cudaError_t e = cudaFuncGetAttributes(&has, prompt_attend_kernel<D>);
    if (e != cudaSuccess) return e;
    if (has.numRegs * kThreads < 256 * kSoftmaxRegs + 128 * kOtherRegs) return cudaErrorLaunchOutOfResources;
  }
  const cudaError_t e = cache8::allow_smem(prompt_attend_kernel<D>, Smem<D>::kBytes, told);
  if (e != cudaSuccess) return e;
  Params p;
  p.a = a;
  p.P = a.G;
  if (a.G > kPacked)
    for (p.P = kPacked; a.G % p.P; --p.P) {
    }
  p.subs = a.G / p.P;
  p.tok = kRows / p.P;
  const int seqs = a.first ? 1 : a.S;
  CUtensorMap q, k, v;
  if (!make_map(&q, a.q, true, D, a.H * a.G, a.n, seqs, p.P, p.tok, &p.q_head, &p.q_seq) ||
      !make_map(&k, a.k, false, D, a.H, a.n, seqs, 0, 0, &p.k_head, &p.k_seq) ||
      !make_map(&v, a.v, false, D, a.H, a.n, seqs, 0, 0, &p.v_head, &p.v_seq))
    return cudaErrorInvalidValue;
  // pairs of tiles at most, over all sequences
  const long long rows = a.first ? a.n : static_cast<long long>(a.n) * a.S;
  const long long most = (rows / (2 * p.tok) + a.S) * a.H * p.subs;
  const int grid = static_cast<int>(most < a.num_sms ? most : a.num_sms);
  return cache8::launch(prompt_attend_kernel<D>, grid, kThreads, Smem<D>::kBytes, s, q, k, v, p);
}

}  // namespace

cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace prompt
}  // namespace kvc
