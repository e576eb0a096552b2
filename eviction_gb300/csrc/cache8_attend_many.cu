// cache8_attend_many.cu -- attention over the 8-bit paged cache for many queries
// (a prompt in pieces, the window of an event): 128 query rows a CTA on the
// 5th-generation tensor cores (tcgen05 + TMEM).
//
//   out_r = sum_t w_rt v_t / sum_t w_rt,  w_rt = exp(scale q_r . k_t)
//
// Row r of a KV head is query r % nq of its group's head r / nq.  Per 128 tokens:
//   converters (4 warps)  codes from global memory to fp16 tiles in shared memory, in
//                         the swizzled layout of the MMA operands, one tile ahead.
//                         Keys and values carry their block's scale relative to the
//                         tile's largest (powers of two, and exact: see below);
//   MMA (1 thread)        S = Q K^T (128 x 128, in TMEM), then O += P V with P read
//                         from TMEM, where it takes the place of S;
//   softmax (4 warps)     one thread a row: the weights, their sum in fp32, P to TMEM
//                         as fp16.  The first of these warps also issues the MMAs: it
//                         would wait for them anyway.
// A weight carries its token's value scale 2^e: w = 2^(x - m), x = z + e, and O is the
// sum of w times the code, so that fp16 weights stay near 1 whatever the blocks' scales
// are; the sum of the softmax takes 2^-e w.  Where the value scales of a tile are at
// most 2^8 below its largest, 2^v, the values are codes times 2^(e - v) instead and the
// weights 2^(z + v - m): no scale for each column, and the sum is scaled once a tile.
// Keys are codes times 2^(their scale - the tile's largest), which fp16 holds exactly
// where that is at most 2^15 down.  A tile whose scales are further apart than either
// has bare codes for both, and its logits get their scales and e column by column.
// That path takes absent tokens as well (e = -inf).
// The reference m of a row lies below its largest x: weights may reach 2^15 (fp16 has
// the room) before m moves, and a new m leaves them at 2^8.  Only what a row sees moves
// it (but for v, at most 2^8): not a block of large values that has no weight or that a
// mask hides.  The maximum comes with the TMEM load (tcgen05.ld.red).  Half of a row
// stays in registers between the maximum and the exponentials, the other half is loaded
// again.
//
// The arithmetic bounds this: 4 R d operations a token, 1024 cycles of the tensor
// pipe per 128 x 128 tile of d = 128.  S and P share columns, so that one CTA's
// softmax and MMAs take turns; two CTAs on an SM (half of TMEM and shared memory
// each) fill each other's gaps, and a CTA's beginning and end as well.
//
// Measured: 128 new tokens on 32 sequences of 1024 to 1536, 4 KV heads of 7 (71 GFLOP)
// 154 us, 22% of the tensor pipe.  By clock stamps in an instrumented copy a tile takes
// 3.3 us: 1.7 in the softmax (half of that exponentials, at the rate of their unit), the
// rest from one product's end to the next one's beginning and in waiting for the other
// CTA's.  128 registers a thread do not hold it all: 160 bytes spill at d 128, 84 at 64.
//
// Heads and row tiles that do not fill the GPU have their tokens cut into parts, which
// a second launch joins in order.  Every wait is bounded.
#include "cache8_attend.cuh"

namespace kvc {
namespace cache8 {
namespace {

constexpr int kRows = 128, kTokens = 128;
constexpr int kSoftmaxWarps = 4, kConvertWarps = 4;
constexpr int kThreads = 32 * (kSoftmaxWarps + kConvertWarps);
constexpr int kInfos = 4;         // tiles whose scales are told ahead
constexpr int kTmemCols = 256;    // S / P: 128, O: up to 128
constexpr int kMaxParts = 320;    // CTAs of a call that cuts heads
constexpr float kRoom = 15.f, kStart = 8.f;  // log2 of the weights' limit and of a new m's
// From references of this size on the logits are rounded (as in the reference) before m is
// taken off them, column by column: one rounding of the difference would leave weights
// off by up to half a step of the logits, 2^-3 here.
constexpr float kExactRef = 1048576.f;
// log2 of how far below the tile's largest scale a plain tile's scales lie at most.  Keys:
// e4m3's last step is 2^-9, fp16's 2^-24.
constexpr int kSpread = 8, kKeySpread = 15;

struct Parts {
  int per_tile;   // CTAs of a row tile
  int row_tiles;  // of a head
  float* part;    // [kMaxParts][D + 2][kRows]: reference, sum, values
};

template <int D>
struct Smem {
  static constexpr int kTile = kTokens * D * 2;
  static constexpr int kV = 0, kK = kTile, kQ = 2 * kTile, kMeta = 3 * kTile;
  static constexpr int kE = kMeta, kBack = kE + kInfos * kTokens * 4,
                       kInfo = kBack + kInfos * kTokens * 4,
                       kTok = kInfo + kInfos * 16, kRed = kTok + 2 * kTokens * 8,
                       kBars = kRed + 2 * kConvertWarps * 16, kMisc = kBars + 24 * 8;
  static constexpr int kBytes = kMisc + 32 + 1024;  // and 1024 for the alignment
};

template <bool V>
struct Bool {
  static constexpr bool value = V;
};

// What a tile's converters tell the softmax warps.
struct TileInfo {
  float k_ref;   // the scale that the tile's keys are relative to, if plain; else 1
  int plain;     // no token is absent and no scale is 2^kSpread / 2^kKeySpread below the largest
  float v_ref;   // log2 of the scale that the values are relative to, if plain; else 0
  float v_back;  // 2^-v_ref
};

__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Instruction descriptor, kind::f16: A = B = fp16, D = fp32; B with N contiguous
// (bit 16) where mn_major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool mn_major) {
  return (1u << 4) | (mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// B operand with N contiguous: rows (K) of 128 bytes = 64 values of N, swizzled in
// groups of 8 rows 1024 bytes apart; the next 64 values of N `block` bytes on.
__device__ __forceinline__ uint64_t sw128_desc_mn(uint32_t addr, uint32_t block) {
  uint64_t desc = sw128_desc(addr);
  desc &= ~(static_cast<uint64_t>(0x3FFF) << 16);
  return desc | static_cast<uint64_t>(block >> 4) << 16;
}

// D += A B with A in tensor memory.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// All lanes wait converged and agree on the outcome.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}

// All lanes' shared-memory writes, then one arrival for the warp.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if (threadIdx.x % 32 == 0) mbar_arrive(bar);
}

// One row tile of one head, and how its tokens are cut.
struct RowTile {
  int l, b, h, r0, rows, nq, len, tiles, per, parts;
  bool bad;
};
__device__ __forceinline__ RowTile row_tile(const Cache& c, const AttendArgs& a, const Parts& sp,
                                            int ur) {
  RowTile w;
  const int u = ur / sp.row_tiles;
  w.h = u % c.H;
  w.b = (u / c.H) % c.B;
  w.l = u / (c.H * c.B);
  w.bad = false;
  w.len = length_of(c, w.b, &w.bad);
  w.nq = a.n_q ? a.n_q[w.b] : a.n;
  if (w.nq < 0 || w.nq > a.n) w.bad = true;
  w.r0 = (ur % sp.row_tiles) * kRows;
  w.rows = w.bad ? 0 : min(a.G * w.nq - w.r0, kRows);
  w.tiles = w.per = w.parts = 0;
  if (w.rows <= 0) return w;
  // the last token that one of the rows sees
  const int r1 = w.r0 + w.rows - 1;
  const int last_q = w.r0 / w.nq == r1 / w.nq ? r1 % w.nq : w.nq - 1;
  w.tiles = div_up(max(w.len - w.nq + last_q + 1, 0), kTokens);
  w.per = max(div_up(w.tiles, sp.per_tile), 2);
  w.parts = max(div_up(w.tiles, w.per), 1);
  return w;
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 2)
    attend_many_kernel(Cache c, AttendArgs a, Parts sp, Div by_bs) {
#if defined(__CUDA_ARCH__) && (__CUDA_ARCH__ >= 1000)
  using Sm = Smem<D>;
  constexpr int DB = D / 64;  // 64-value blocks (128 bytes) of a row
  constexpr int kBlock = kTokens * 128;  // bytes of one block of all rows
  constexpr uint32_t kOutCol = 128;      // O's first TMEM column
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* s_e = reinterpret_cast<float*>(smem + Sm::kE);        // [kInfos][kTokens]
  // [kInfos][kTokens] 2^-e and the key's scale, as two bf16
  uint32_t* s_back = reinterpret_cast<uint32_t*>(smem + Sm::kBack);
  TileInfo* s_info = reinterpret_cast<TileInfo*>(smem + Sm::kInfo);
  int2* s_tok = reinterpret_cast<int2*>(smem + Sm::kTok);  // [2][kTokens] row, exponents
  int4* s_red = reinterpret_cast<int4*>(smem + Sm::kRed);  // [2][kConvertWarps]
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sm::kBars);
  uint64_t *q_full = bars, *k_full = bars + 1, *k_empty = bars + 2, *v_full = bars + 3,
           *v_empty = bars + 4, *s_full = bars + 5, *p_full = bars + 6, *o_full = bars + 7,
           *r_full = bars + 8, *done = bars + 9, *m_full = bars + 10,
           *m_empty = bars + 10 + kInfos;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Sm::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + Sm::kMisc + 4);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  before_all();

  // ---- this CTA's row tile and tokens ----
  const int part = blockIdx.x % sp.per_tile;
  const RowTile w = row_tile(c, a, sp, blockIdx.x / sp.per_tile);
  if (w.bad && threadIdx.x == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
  if (w.rows <= 0 || part >= w.parts) return;
  const int l = w.l, b = w.b, h = w.h, r0 = w.r0, rows = w.rows, nq = w.nq, len = w.len,
            parts = w.parts;
  const int tile0 = part * w.per, n_tiles = min(w.per, w.tiles - tile0);
  bool bad = false;

  if (threadIdx.x == 0) {
    mbar_init(q_full, kSoftmaxWarps);
    mbar_init(k_full, kConvertWarps);
    mbar_init(k_empty, 1);
    mbar_init(v_full, kConvertWarps);
    mbar_init(v_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(p_full, kSoftmaxWarps);
    mbar_init(o_full, 1);
    mbar_init(r_full, kConvertWarps);
    for (int i = 0; i < kInfos; ++i) {
      mbar_init(&m_full[i], kConvertWarps);
      mbar_init(&m_empty[i], kSoftmaxWarps);
    }
    mbar_init(done, 1);
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(tmem_slot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < kSoftmaxWarps) {
    // ------------------------------------------------------------ softmax
    const int row = threadIdx.x, r = r0 + row;
    const bool there = row < rows;
    const int hq = h * a.G + (there ? r / nq : 0), j = there ? r % nq : 0;
    const uint32_t my_tmem = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    // the query row as fp16, times a power of two
    float qf;
    {
      const uint4* q = reinterpret_cast<const uint4*>(a.q.at(l, b, hq, j));
      uint4 v[D / 8];
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) v[i] = there ? q[i] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint32_t x[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(x[k])), fabsf(bf16_hi(x[k]))));
      }
      const int e = row_exp(mx);
      const float down = exp2_int(-e);
      qf = finite_factor(a.scale_log2, exp2_int(e));
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<uint4*>(smem + Sm::kQ + (i / 8) * kBlock + row * 128 +
                                  (((i % 8) ^ (row % 8)) << 4)) =
            make_uint4(half2_of(bf16_lo(v[i].x) * down, bf16_hi(v[i].x) * down),
                       half2_of(bf16_lo(v[i].y) * down, bf16_hi(v[i].y) * down),
                       half2_of(bf16_lo(v[i].z) * down, bf16_hi(v[i].z) * down),
                       half2_of(bf16_lo(v[i].w) * down, bf16_hi(v[i].w) * down));
      fence_async_shared();
      warp_arrive(q_full);
    }
    // the first warp issues the products (all lanes wait converged, lane 0 issues)
    const uint32_t base = smem_u32(smem);
    auto issue_scores = [&](int i) {  // S = Q K^T of tile i
      // (S takes P's columns: the last product has to be done with them)
      if (!warp_wait(k_full, i & 1, abort, c.status) ||
          (i > 0 && !warp_wait(o_full, (i - 1) & 1, abort, c.status)))
        return false;
      tc_fence_after();
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_f16(kRows, kTokens, false);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k / 4) * kBlock + (k % 4) * 32;
          mma_bf16(tmem, sw128_desc(base + Sm::kQ + off), sw128_desc(base + Sm::kK + off), idesc,
                   k > 0 ? 1u : 0u);
        }
        mma_commit(k_empty);
        mma_commit(s_full);
      }
      __syncwarp();
      return true;
    };
    auto issue_output = [&](int i) {  // O += P V of tile i
      if (!warp_wait(v_full, i & 1, abort, c.status) || !warp_wait(p_full, i & 1, abort, c.status))
        return false;
      tc_fence_after();
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_f16(kRows, D, true);
#pragma unroll
        for (int k = 0; k < kTokens / 16; ++k)
          mma_f16_ts(tmem + kOutCol, tmem + k * 8,
                     sw128_desc_mn(base + Sm::kV + k * 2048, kBlock), idesc,
                     i > 0 || k > 0 ? 1u : 0u);
        mma_commit(v_empty);
        mma_commit(o_full);
      }
      __syncwarp();
      return true;
    };
    const int limit = len - nq + j;     // last token that this row sees
    float m = -INFINITY, sum = 0.f;     // reference of the weights, their sum
    bool ok = true;
    if (warp == 0 && n_tiles > 0)
      ok = warp_wait(q_full, 0, abort, c.status) && issue_scores(0);
    for (int i = 0; ok && i < n_tiles; ++i) {
      const int t0 = (tile0 + i) * kTokens, st = i % kInfos;
      if (!warp_wait(&m_full[st], (i / kInfos) & 1, abort, c.status) ||
          !warp_wait(s_full, i & 1, abort, c.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const TileInfo info = s_info[st];
      const float* e_col = s_e + st * kTokens;
      const uint32_t* back_col = s_back + st * kTokens;
      const float f = finite_factor(qf, info.k_ref);
      const bool whole = t0 + kTokens <= len - nq + 1;  // seen by all rows
      const int seen = limit - t0 + 1;                  // columns that this row sees
      uint32_t va[32], vb[32];
      float top;
      if (info.plain && whole) {
        float m0, m1;
        tmem_ld32_max(my_tmem + 64, va, m0);
        tmem_ld32_max(my_tmem + 96, vb, m1);
        tmem_ld_wait();
        top = fmaxf(m0, m1);
        tmem_ld32_max(my_tmem, va, m0);
        tmem_ld32_max(my_tmem + 32, vb, m1);
        tmem_ld_wait();
        top = fmaf(fmaxf(top, fmaxf(m0, m1)), f, info.v_ref);
      } else if (info.plain) {
        auto most = [&](const uint32_t (&v)[32], int first, float so_far) {
#pragma unroll
          for (int x = 0; x < 32; ++x)
            so_far = first + x < seen ? fmaxf(so_far, __uint_as_float(v[x])) : so_far;
          return so_far;
        };
        tmem_ld32(my_tmem + 64, va);
        tmem_ld32(my_tmem + 96, vb);
        tmem_ld_wait();
        top = most(vb, 96, most(va, 64, -INFINITY));
        tmem_ld32(my_tmem, va);
        tmem_ld32(my_tmem + 32, vb);
        tmem_ld_wait();
        top = fmaf(most(vb, 32, most(va, 0, top)), f, info.v_ref);
      } else {
        top = -INFINITY;
#pragma unroll 1
        for (int k = 0; k < kTokens / 32; ++k) {
          tmem_ld32(my_tmem + k * 32, va);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            const float z =
                fmaf(__uint_as_float(va[x]) * bf16_lo(back_col[k * 32 + x]), f, e_col[k * 32 + x]);
            if (k * 32 + x < seen) top = fmaxf(top, z);
          }
        }
      }
      // ---- new references: what is there is scaled to them ----
      const bool raise = top - m > kRoom;  // (not top > m + kRoom: that sum may round)
      if (__any_sync(0xffffffffu, raise)) {
        // (where top's own steps are 16, top - kStart may round to top - 16)
        const float next = !raise ? m : top - (top - kStart) > kRoom ? top : top - kStart;
        const float keep = raise ? ex2(m - next) : 1.f;
        m = next;
        sum *= keep;
        if (i > 0) {
          if (!warp_wait(o_full, (i - 1) & 1, abort, c.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint32_t v[16];
#pragma unroll 1
          for (int k = 0; k < D / 16; ++k) {
            tmem_ld16(my_tmem + kOutCol + k * 16, v);
            tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 16; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) * keep);
            tmem_st16(my_tmem + kOutCol + k * 16, v);
          }
          tmem_st_wait();
        }
      }
      // ---- weights: S's columns become P's ----
      const float ref = m == -INFINITY ? 0.f : m;
      const float add = info.v_ref - ref;
      const float2 ff = make_float2(f, f), off = make_float2(add, add), back = make_float2(-ref, -ref);
      float2 part_sum = make_float2(0.f, 0.f);
      if (info.plain && __all_sync(0xffffffffu, fabsf(ref) < kExactRef)) {
        auto weights = [&](const uint32_t (&v)[32], int first, auto masked) {
          uint32_t p[16];
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float2 z = fma2(make_float2(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1])),
                            ff, off);
            if constexpr (decltype(masked)::value) {
              z.x = first + 2 * x < seen ? z.x : -INFINITY;
              z.y = first + 2 * x + 1 < seen ? z.y : -INFINITY;
            }
            z.x = ex2(z.x);
            z.y = ex2(z.y);
            part_sum = add2(part_sum, z);
            p[x] = half2_of(z.x, z.y);
          }
          tmem_st16(my_tmem + first / 2, p);
        };
        // columns 0-63 are in registers, and P takes no others before 64-127 are read
        auto all = [&](auto masked) {
          weights(va, 0, masked);
          tmem_ld32(my_tmem + 64, va);
          weights(vb, 32, masked);
          tmem_ld32(my_tmem + 96, vb);
          tmem_ld_wait();
          weights(va, 64, masked);
          weights(vb, 96, masked);
        };
        if (whole)
          all(Bool<false>{});
        else
          all(Bool<true>{});
      } else {
#pragma unroll 1
        for (int k = 0; k < kTokens / 32; ++k) {
          uint32_t p[16];
          tmem_ld32(my_tmem + k * 32, va);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 16; x += 2) {
            const float4 e4 = *reinterpret_cast<const float4*>(e_col + k * 32 + 2 * x);
            const uint4 b4 = *reinterpret_cast<const uint4*>(back_col + k * 32 + 2 * x);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int at = 2 * (x + y);
              float2 z = make_float2(__uint_as_float(va[at]) * bf16_lo(y ? b4.z : b4.x),
                                     __uint_as_float(va[at + 1]) * bf16_lo(y ? b4.w : b4.y));
              z = fma2(z, ff, y ? make_float2(e4.z, e4.w) : make_float2(e4.x, e4.y));
              z = add2(z, back);
              z.x = k * 32 + at < seen ? ex2(z.x) : 0.f;
              z.y = k * 32 + at + 1 < seen ? ex2(z.y) : 0.f;
              part_sum = fma2(z, make_float2(bf16_hi(y ? b4.z : b4.x), bf16_hi(y ? b4.w : b4.y)),
                              part_sum);
              p[x + y] = half2_of(z.x, z.y);
            }
          }
          tmem_st16(my_tmem + k * 16, p);
        }
      }
      sum = fmaf(part_sum.x + part_sum.y, info.v_back, sum);
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(p_full);
      if (lane == 0) mbar_arrive(&m_empty[st]);
      if (warp == 0) ok = issue_output(i) && (i + 1 == n_tiles || issue_scores(i + 1));
    }
    if (warp == 0) {
      if (lane == 0) mma_commit(done);
      __syncwarp();
      volatile int never = 0;  // also after an abort: what was issued ends
      mbar_wait(done, 0, &never, c.status);
    }
    // ---- the result ----
    if (ok && n_tiles > 0) ok = warp_wait(o_full, (n_tiles - 1) & 1, abort, c.status);
    if (ok) {
      tc_fence_after();
      float* slot = sp.part + static_cast<size_t>(blockIdx.x) * ((D + 2) * kRows) + row;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 1
      for (int k = 0; k < D / 32; ++k) {
        uint32_t v[32];
        if (n_tiles > 0) {
          tmem_ld32(my_tmem + kOutCol + k * 32, v);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) v[x] = 0;
        }
        if (there && parts == 1) {
          uint4* out = reinterpret_cast<uint4*>(a.out.at(l, b, hq, j) + k * 32);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            float y[8];
#pragma unroll
            for (int z = 0; z < 8; ++z) y[z] = __uint_as_float(v[8 * x + z]) * inv;
            out[x] = make_uint4(bf16x2(y[0], y[1]), bf16x2(y[2], y[3]), bf16x2(y[4], y[5]),
                                bf16x2(y[6], y[7]));
          }
        } else if (there) {
#pragma unroll
          for (int x = 0; x < 32; ++x) slot[(2 + k * 32 + x) * kRows] = __uint_as_float(v[x]);
        }
        __syncwarp();
      }
      if (there && parts == 1 && a.lse)
        a.lse[((static_cast<size_t>(l) * c.B + b) * c.H * a.G + hq) * a.n + j] =
            (m + __log2f(sum)) * 0.6931471805599453f;
      if (there && parts > 1) {
        slot[0] = m;
        slot[kRows] = sum;
      }
    }
  } else {
    // ------------------------------------------------------------ converters
    // This lane: rows (tokens) row_in + 32 i, 16-byte chunks q4 + 4 j of them.
    const int cw = warp - kSoftmaxWarps, q4 = lane % 4;
    const int row_in = cw * 8 + lane / 4;
    const uint8_t* kp = c.pool[0] + block_row(c, l, 0, h) * D;
    const uint8_t* vp = c.pool[1] + block_row(c, l, 0, h) * D;
    const float* ksp = c.scale[0] + scale_at(c, l, 0, h);
    const float* vsp = c.scale[1] + scale_at(c, l, 0, h);
    const int32_t* table = c.table + static_cast<size_t>(b) * c.max_blocks;
    // This lane looks up token 32 cw + lane of a tile; the warps exchange what they find.
    const int own = cw * 32 + lane;
    int own_blk, own_row;
    uint32_t own_ks, own_vs;  // scales as they are in memory
    int row[4];               // of the tokens row_in + 32 k
    uint4 kc[4][DB], vc[4][DB];
    auto lookup = [&](int i) {  // the tile's blocks
      const int t = (tile0 + i) * kTokens + own;
      const bool in = i < n_tiles && t < len;
      own_blk = table[in ? by_bs.div(t) : 0];
      if (!in) own_blk = -1;
    };
    auto resolve = [&](int i) {  // rows and scales of the tile whose blocks are known
      const int t = (tile0 + i) * kTokens + own;
      const bool in = i < n_tiles && t < len;
      const bool found = in && static_cast<uint32_t>(own_blk) < static_cast<uint32_t>(c.n_blocks);
      bad = bad || (in && !found);
      const size_t sc = found ? static_cast<size_t>(own_blk) * c.H : 0;
      own_ks = __float_as_uint(ksp[sc]);
      own_vs = __float_as_uint(vsp[sc]);
      own_row = found ? own_blk * c.H * by_bs.bs + (t - by_bs.div(t) * by_bs.bs) : -1;
    };
    auto load_codes = [&](const uint8_t* pool, uint4 (&to)[4][DB]) {
      bool all = true;
#pragma unroll
      for (int k = 0; k < 4; ++k) all = all && row[k] >= 0;
      if (__all_sync(0xffffffffu, all)) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int x = 0; x < DB; ++x)
            to[k][x] = *reinterpret_cast<const uint4*>(pool + static_cast<size_t>(row[k]) * D +
                                                       (q4 + 4 * x) * 16);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int x = 0; x < DB; ++x)
            to[k][x] = row[k] >= 0 ? *reinterpret_cast<const uint4*>(
                                         pool + static_cast<size_t>(row[k]) * D + (q4 + 4 * x) * 16)
                                   : make_uint4(0, 0, 0, 0);
      }
    };
    // 16 codes each of this lane's rows, times their factors, to their places in a tile
    // (the two 16-byte places of a chunk are the same in all rows: row_in + 32 k)
    uint8_t* const place0 = smem + row_in * 128 + (((2 * q4) ^ (row_in % 8)) << 4);
    uint8_t* const place1 = smem + row_in * 128 + (((2 * q4 + 1) ^ (row_in % 8)) << 4);
    constexpr uint32_t kOne = 0x3C003C00u;
    auto store = [&](int tile, const uint4 (&codes)[4][DB], const uint32_t (&factor)[4]) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool scaled = __any_sync(0xffffffffu, factor[k] != kOne);
#pragma unroll
        for (int x = 0; x < DB; ++x) {
          const uint32_t w[4] = {codes[k][x].x, codes[k][x].y, codes[k][x].z, codes[k][x].w};
          uint32_t o[8];
#pragma unroll
          for (int y = 0; y < 4; ++y) halves<FMT>(w[y], o[2 * y], o[2 * y + 1]);
          if (scaled) {
#pragma unroll
            for (int y = 0; y < 8; ++y) o[y] = mul_half2(o[y], factor[k]);
          }
          const int at = tile + x * kBlock + k * 32 * 128;
          *reinterpret_cast<uint4*>(place0 + at) = make_uint4(o[0], o[1], o[2], o[3]);
          *reinterpret_cast<uint4*>(place1 + at) = make_uint4(o[4], o[5], o[6], o[7]);
        }
      }
    };
    // A tile's rows and scales: this lane's rows and factors; the softmax warps are told.
    uint32_t k_factor[4], v_factor[4], v_next[4];
    auto announce = [&](int i) {
      const int st = i % kInfos, ex = i & 1;
      const bool there = own_row >= 0;
      const int ke = static_cast<int>(own_ks >> 23) - 127, ve = static_cast<int>(own_vs >> 23) - 127;
      // (an absent token's minima leave no tile plain)
      int k_max = __reduce_max_sync(0xffffffffu, there ? ke : -1000);
      int k_min = __reduce_min_sync(0xffffffffu, there ? ke : -1000);
      int v_max = __reduce_max_sync(0xffffffffu, there ? ve : -1000);
      int v_min = __reduce_min_sync(0xffffffffu, there ? ve : -1000);
      // (two buffers: a warp writes one again after all have read the other)
      s_tok[ex * kTokens + own] = make_int2(own_row, (ke & 0xffff) | ve << 16);
      if (lane == 0) s_red[ex * kConvertWarps + cw] = make_int4(k_max, k_min, v_max, v_min);
      warp_arrive(r_full);
      if (!warp_wait(&m_empty[st], ((i / kInfos) & 1) ^ 1, abort, c.status) ||
          !warp_wait(r_full, i & 1, abort, c.status))
        return false;
      k_max = v_max = -126;
#pragma unroll
      for (int k = 0; k < kConvertWarps; ++k) {
        const int4 o = s_red[ex * kConvertWarps + k];
        k_max = max(k_max, o.x);
        k_min = min(k_min, o.y);
        v_max = max(v_max, o.z);
        v_min = min(v_min, o.w);
      }
      const bool plain = v_max - v_min <= kSpread && k_max - k_min <= kKeySpread;
      // (a plain tile's scales are in its references)
      s_e[st * kTokens + own] = plain ? static_cast<float>(v_max)
                                      : there ? static_cast<float>(ve) : -INFINITY;
      s_back[st * kTokens + own] =
          plain ? 0x3f803f80u : there ? __float_as_uint(exp2_int(-ve)) | own_ks >> 16 : 0x3f80u;
      if (lane == 0 && cw == 0) {
        TileInfo info;
        info.k_ref = plain ? exp2_int(k_max) : 1.f;
        info.plain = plain;
        info.v_ref = plain ? static_cast<float>(v_max) : 0.f;
        info.v_back = plain ? exp2_int(-v_max) : 1.f;
        s_info[st] = info;
      }
      warp_arrive(&m_full[st]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int2 tok = s_tok[ex * kTokens + row_in + 32 * k];
        row[k] = tok.x;
        const int e = static_cast<int16_t>(tok.y & 0xffff), f = tok.y >> 16;
        k_factor[k] = plain ? exp2_half2(e - k_max) : kOne;
        v_next[k] = plain ? exp2_half2(f - v_max) : kOne;
      }
      return true;
    };
    // A tile's keys can be stored once the last one's scores are done, its values once
    // the last one's output is.  Between the two stores of one turn of the loop, which
    // the products wait for, there are only the next values' loads.  Codes are on their
    // way one tile ahead, scales two, blocks three.
    lookup(0);
    resolve(0);
    lookup(1);
    bool go = n_tiles > 0 && announce(0);
    if (go) {
      load_codes(kp, kc);
      load_codes(vp, vc);
      resolve(1);
      lookup(2);
      store(Sm::kK, kc, k_factor);
      fence_async_shared();
      warp_arrive(k_full);
#pragma unroll
      for (int k = 0; k < 4; ++k) v_factor[k] = v_next[k];
      if (n_tiles > 1) {
        go = announce(1);
        load_codes(kp, kc);
        resolve(2);
        lookup(3);
      }
    }
    for (int i = 0; go && i < n_tiles; ++i) {
      if (!warp_wait(v_empty, (i & 1) ^ 1, abort, c.status)) break;
      store(Sm::kV, vc, v_factor);
      fence_async_shared();
      warp_arrive(v_full);
      if (i + 1 == n_tiles) break;
      load_codes(vp, vc);
      if (!warp_wait(k_empty, i & 1, abort, c.status)) break;
      store(Sm::kK, kc, k_factor);
      fence_async_shared();
      warp_arrive(k_full);
#pragma unroll
      for (int k = 0; k < 4; ++k) v_factor[k] = v_next[k];
      if (i + 2 == n_tiles) continue;
      if (!announce(i + 2)) break;
      load_codes(kp, kc);
      resolve(i + 3);
      lookup(i + 4);
    }
    if (bad) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
#endif
}

// Joins the parts of a row tile, in their order: 128 rows x kJoin values of a CTA, so
// that many SMs read the parts.  (One CTA alone took longer for it than the parts'
// own work on 16 heads of 16384 tokens.)
constexpr int kJoin = 8;
template <int D>
__global__ void __launch_bounds__(kRows) attend_many_join_kernel(Cache c, AttendArgs a, Parts sp) {
  static_assert(kJoin == kPer, "write_row takes kPer values");
  before_all();
  const RowTile w = row_tile(c, a, sp, blockIdx.x);
  const int row = threadIdx.x, d0 = blockIdx.y * kJoin;
  if (w.parts <= 1 || row >= w.rows) return;
  constexpr size_t kSlot = (D + 2) * kRows;
  const float* from = sp.part + static_cast<size_t>(blockIdx.x) * sp.per_tile * kSlot + row;
  float m = -INFINITY, sum = 0.f, y[kJoin];
#pragma unroll 8
  for (int k = 0; k < w.parts; ++k) m = fmaxf(m, from[k * kSlot]);
  const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int x = 0; x < kJoin; ++x) y[x] = 0.f;
#pragma unroll 4
  for (int k = 0; k < w.parts; ++k) {
    const float* p = from + k * kSlot;
    const float f = ex2(p[0] - ref);
    sum += f * p[kRows];
#pragma unroll
    for (int x = 0; x < kJoin; ++x) y[x] += f * p[(2 + d0 + x) * kRows];
  }
  write_row(c, a, w.l, w.b, w.h, w.r0 + row, w.nq, d0, y, m, sum);
}

template <int D, int FMT>
cudaError_t launch_many(const Cache& c, const AttendArgs& a, cudaStream_t s) {
  auto* kernel = attend_many_kernel<D, FMT>;
  static std::atomic<uint64_t> told{0};
  cudaError_t e = allow_smem(kernel, Smem<D>::kBytes, told);
  if (e != cudaSuccess) return e;
  Parts sp;
  sp.row_tiles = (a.G * a.n + kRows - 1) / kRows;
  sp.part = reinterpret_cast<float*>(static_cast<int*>(a.workspace) + kCounters);
  const long long tiles = static_cast<long long>(c.L) * c.B * c.H * sp.row_tiles;
  long long per = min(2 * a.num_sms, kMaxParts) / tiles;
  sp.per_tile = static_cast<int>(per < 1 ? 1 : per);
  e = launch(kernel, static_cast<int>(tiles * sp.per_tile), kThreads, Smem<D>::kBytes, s, c, a, sp,
             make_div(c.bs));
  if (e != cudaSuccess || sp.per_tile == 1) return e;
  return launch(attend_many_join_kernel<D>, dim3(static_cast<int>(tiles), D / kJoin), kRows, 0, s, c,
                a, sp);
}

}  // namespace

cudaError_t launch_attend_many(const Cache& c, int format, const AttendArgs& a, cudaStream_t s) {
  if (c.d == 64)
    return format == KVC_CACHE8_E4M3 ? launch_many<64, KVC_CACHE8_E4M3>(c, a, s)
                                     : launch_many<64, KVC_CACHE8_INT8>(c, a, s);
  return format == KVC_CACHE8_E4M3 ? launch_many<128, KVC_CACHE8_E4M3>(c, a, s)
                                   : launch_many<128, KVC_CACHE8_INT8>(c, a, s);
}

size_t attend_many_parts_bytes(int d) {
  return kMaxParts * static_cast<size_t>(d + 2) * kRows * sizeof(float);
}

}  // namespace cache8
}  // namespace kvc
