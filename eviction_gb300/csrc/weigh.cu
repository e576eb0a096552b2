// weigh.cu -- attention weight that the newest tokens' queries give each token of the 8-bit
// paged cache, added to what it has gathered (kvc_cache8_weigh), for few queries: decode steps.
//
//   w_t = decay w_t + sum_r 2^(z_rt - y_r),  z = scale log2(e) q_r . k_t,  y = lse_r log2(e)
//
// over the R = G n query rows of a KV head that see t.  The rows' normalisers are known, so
// that a token's sum needs nothing of other tokens: every warp takes steps of 32 tokens by
// itself, with nothing to join.  A token is d bytes of keys and 8 of weights, read and written
// once, and 2 R d operations: the call is bound by memory.
//
// The list of all heads' steps is cut into equal stretches, one a warp, whatever the lengths
// are.  A warp has a ring of stages in shared memory, filled by bulk copies of the rows that
// lie side by side in a block, two steps ahead; blocks are looked up a step ahead of the
// copies, and a next head's queries are on their way one step before they are needed.  Per 16
// tokens a warp computes S^T = K Q^T (m16n8k16, tokens on the M axis, 8 NT query rows), with
// the codes converted to fp16, which holds both formats exactly, and a query row divided by a
// power of two that its largest magnitude brings to [1, 4).
//
// Measured: 64 sequences of 612 to 1112 tokens, 8 heads of 128 (e4m3, 61 MB) 15.5 us, 4 of 32768,
// 4 heads (int8, 71 MB) 16 us, of which launch, the first copies' latency and the last stretch's end
// are 6 us.  Up to 32 query rows of a KV head (packed calls: of all sequences together, which is all that
// the host knows): on the former batch 15.5 us for 8 rows, 19 for 12 and 16, 28 for 24 and 32, where the
// other kernel takes 54; 36 to 64 rows take 55 there, 128 62, 188 65.
#include "weigh.cuh"

namespace kvc {
namespace prompt {
namespace {

using namespace cache8;

constexpr int kTile = 32;    // tokens of a step
constexpr int kWarps = 4;    // of a CTA
constexpr int kStages = 3;

// Bulk copy global -> shared (16-byte aligned, a multiple of 16 bytes), counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t to, const void* from, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(to),
      "l"(reinterpret_cast<uint64_t>(from)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A place in the list of steps: step of head h of sequence b in layer l.
struct Cursor {
  int l, b, h, step, steps;
  Lengths n;
};

__device__ __forceinline__ int steps_of(const Lengths& n) { return (n.len + kTile - 1) / kTile; }

__device__ __forceinline__ void advance(const Cache& c, const WeighArgs& a, Cursor& x) {
  bool unused = false;
  if (++x.step < x.steps) return;
  x.step = 0;
  if (++x.h < c.H) return;
  x.h = 0;
  do {
    if (++x.b == c.B) {
      x.b = 0;
      ++x.l;
    }
    x.n = lengths_of(c, a, x.b, &unused);
    x.steps = steps_of(x.n);
  } while (x.steps == 0);
}

template <int D, int FMT, int NT>
__global__ void __launch_bounds__(32 * kWarps) weigh_few_kernel(Cache c, WeighArgs a, Div by_bs) {
  constexpr int KV = D / 64;  // 16-byte loads of a key row per lane
  extern __shared__ __align__(128) uint8_t smem[];  // [kWarps][kStages][kTile][D] codes
  __shared__ uint64_t s_full[kWarps][kStages];
  __shared__ int s_abort;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, q4 = lane % 4;
  bool bad = false, unused = false;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&s_full[warp][i], 1);
    if (warp == 0) s_abort = 0;
    fence_barrier_init();
  }
  __syncthreads();

  before_all();

  // ---- this warp's stretch of the list ----
  // (every warp computes it for itself; the counts are below 2^31: checked on the host)
  int all = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32)
    all += b0 + lane < c.B ? steps_of(lengths_of(c, a, b0 + lane, &bad)) : 0;
  all = __reduce_add_sync(0xffffffffu, all);
  if (blockIdx.x == 0 && warp == 0 && bad) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
  bad = false;
  const int heads = c.H * c.L, total = all * heads, warps = gridDim.x * kWarps;
  // equal shares, the first ones a step larger where they do not come out even
  // (where there is a step for some warps only, a warp of each CTA first: 2 sequences of 1112 tokens, 8
  // heads, 4.4 us, of 5.4 with all warps of few CTAs; side by side in a CTA otherwise: 4 x 32768
  // tokens 16.1 us, of 16.5 so)
  const int share = total / warps, more = total % warps;
  const int w = share ? blockIdx.x * kWarps + warp : warp * gridDim.x + blockIdx.x;
  const int begin = w * share + min(w, more), count = share + (w < more);
  if (count == 0) return;
  Cursor at;
  at.l = begin / (all * c.H);
  {
    int in = begin % (all * c.H), before = 0;  // within the layer
    for (int b0 = 0;; b0 += 32) {
      const int own = b0 + lane < c.B ? steps_of(lengths_of(c, a, b0 + lane, &unused)) * c.H : 0;
      int incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, in < before + incl);
      if (past) {
        const int place_in = __ffs(past) - 1;
        in -= before + __shfl_sync(0xffffffffu, incl - own, place_in);
        at.b = b0 + place_in;
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    at.n = lengths_of(c, a, at.b, &unused);
    at.steps = steps_of(at.n);
    at.h = in / at.steps;
    at.step = in % at.steps;
  }

  const uint8_t* own_ring = smem + warp * (kStages * kTile * D);
  const uint32_t ring = smem_u32(own_ring);
  uint64_t* full = s_full[warp];
  // Lane i looks after token i of a step: its block, and the copy of its row with those behind
  // it in the same block.
  auto block_of = [&](const Cursor& x) {
    const int t = x.step * kTile + lane;
    return t < x.n.len ? c.table[static_cast<size_t>(x.b) * c.max_blocks + by_bs.div(t)] : -1;
  };
  // start a step's copies; the lane's token's scale (0: there is none)
  auto fetch = [&](const Cursor& x, int blk, int stage) {
    const int t = x.step * kTile + lane, in = t - by_bs.div(t) * by_bs.bs;
    const bool there = t < x.n.len && static_cast<uint32_t>(blk) < static_cast<uint32_t>(c.n_blocks);
    bad = bad || (t < x.n.len && !there);
    const uint32_t rows = __popc(__ballot_sync(0xffffffffu, there));
    if (lane == 0) mbar_arrive_expect_tx(&full[stage], rows * D);
    __syncwarp();
    if (!there) return 0.f;
    const size_t head = block_row(c, x.l, blk, x.h);
    if (lane == 0 || in == 0)
      bulk_load(ring + stage * (kTile * D) + lane * D, c.pool[0] + (head + in) * D,
                min(min(by_bs.bs - in, kTile - lane), x.n.len - t) * D, &full[stage]);
    return c.scale[0][scale_at(c, x.l, blk, x.h)];
  };
  // (after the sums over the lanes a lane has those of token own)
  const int own = g + 8 * q4;
  auto weight_at = [&](const Cursor& x) {
    const size_t u = (static_cast<size_t>(x.l) * c.B + x.b) * c.H + x.h;
    return a.w + u * a.cap + x.step * kTile + own;
  };
  auto old_weight = [&](const Cursor& x) {
    return a.decay != 0.f && x.step * kTile + own < x.n.len ? *weight_at(x) : 0.f;
  };
  // a head's query rows g + 8 nt as they are in memory, and the lse of rows 2 q4, 2 q4 + 1
  uint4 raw[NT][KV][2];
  float raw_lse[NT][2];
  auto load_queries = [&](const Cursor& x) {
    const int rows = a.G * x.n.nq, sb = a.first ? 0 : x.b, S = a.first ? 1 : c.B;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;
      const bool there = r < rows;
      const uint16_t* qp = a.q.at(x.l, sb, x.h * a.G + (there ? r / x.n.nq : 0),
                                  there ? x.n.first + r % x.n.nq : 0);
#pragma unroll
      for (int k = 0; k < KV; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          raw[nt][k][i] = there ? *reinterpret_cast<const uint4*>(qp + (k * 4 + q4) * 16 + i * 8)
                                : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int s = nt * 8 + 2 * q4 + i;
        raw_lse[nt][i] = s < rows ? a.lse[((static_cast<size_t>(x.l) * S + sb) * c.H * a.G + x.h * a.G +
                                           s / x.n.nq) * a.n + x.n.first + s % x.n.nq]
                                  : INFINITY;
      }
    }
  };

  // ---- the pipeline: step i is computed, i + 1 and i + 2 are being copied, i + 3 is looked up ----
  Cursor far = at;
  load_queries(at);
  float scales[3], olds[3];  // of steps i, i + 1, i + 2
  bool begins[3];            // a head: its queries are new
  int blk = block_of(far), stage = 0;
  uint32_t parity = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    scales[i] = olds[i] = 0.f;
    begins[i] = i == 0 || far.step == 0;
    if (i < count) {
      olds[i] = old_weight(far);
      scales[i] = fetch(far, blk, i);
      if (i + 1 < count) {
        advance(c, a, far);
        blk = block_of(far);
      }
    }
  }
  uint32_t qf[NT][KV * 4][2];
  float qscale[NT][2], y[NT][2];
  int limit[NT][2];
  for (int i = 0; i < count; ++i) {
    scales[2] = olds[2] = 0.f;
    begins[2] = far.step == 0;
    if (i + 2 < count) {
      olds[2] = old_weight(far);
      scales[2] = fetch(far, blk, stage == 0 ? kStages - 1 : stage - 1);
      if (i + 3 < count) {
        advance(c, a, far);
        blk = block_of(far);
      }
    }
    const bool fresh = begins[0];
    if (fresh) {  // queries as fp16, in the order of the key reads
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        auto& v = raw[nt];
        // a row that sees no token may hold anything: zeros, so that its scores are no NaN (the lse of
        // row g is with the lanes whose q4 is g / 2)
        const float lse0 = __shfl_sync(0xffffffffu, raw_lse[nt][0], g / 2);
        const float lse1 = __shfl_sync(0xffffffffu, raw_lse[nt][1], g / 2);
        if (sees_nothing(g % 2 ? lse1 : lse0)) {
#pragma unroll
          for (int k = 0; k < KV; ++k) v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);
        }
        float mx = 0.f;
#pragma unroll
        for (int k = 0; k < KV; ++k)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint32_t x[4] = {v[k][z].x, v[k][z].y, v[k][z].z, v[k][z].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(x[j])), fabsf(bf16_hi(x[j]))));
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int e = row_exp(mx);
        const float down = exp2_int(-e);
#pragma unroll
        for (int k = 0; k < KV; ++k)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint32_t x[4] = {v[k][z].x, v[k][z].y, v[k][z].z, v[k][z].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              qf[nt][k * 4 + z * 2 + j / 2][j % 2] =
                  half2_of(bf16_lo(x[j]) * down, bf16_hi(x[j]) * down);
          }
        const float up = finite_factor(a.scale_log2, exp2_int(e));
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int r = nt * 8 + 2 * q4 + z;
          qscale[nt][z] = __shfl_sync(0xffffffffu, up, (2 * q4 + z) * 4);
          y[nt][z] = lse_base2(raw_lse[nt][z]);
          limit[nt][z] = at.n.nq > 0 ? at.n.len - at.n.nq + r % at.n.nq : -1;
        }
      }
    }
    if (i + 1 < count && begins[1]) {
      Cursor next = at;
      advance(c, a, next);
      load_queries(next);
    }
    if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], parity, &s_abort, c.status))) {
      volatile int never = 0;  // what is on its way lands before the warp ends
      for (int k = 1; k < kStages && i + k < count; ++k) {
        if (++stage == kStages) stage = 0, parity ^= 1;
        mbar_wait(&full[stage], parity, &never, c.status);
      }
      break;
    }
    const uint8_t* keys = own_ring + stage * (kTile * D);

    // ---- S^T = K Q^T ----
    float z[2][NT][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) z[mt][nt][j] = 0.f;
#pragma unroll
    for (int k = 0; k < KV; ++k)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const uint4 k0 = *reinterpret_cast<const uint4*>(keys + (mt * 16 + g) * D + (k * 4 + q4) * 16);
        const uint4 k1 = *reinterpret_cast<const uint4*>(keys + (mt * 16 + g + 8) * D + (k * 4 + q4) * 16);
        const uint32_t xa[4] = {k0.x, k0.y, k0.z, k0.w};
        const uint32_t xb[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a0, a1, a2, a3;
          halves<FMT>(xa[j], a0, a2);
          halves<FMT>(xb[j], a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma(z[mt][nt], a0, a1, a2, a3, qf[nt][k * 4 + j][0], qf[nt][k * 4 + j][1]);
        }
      }

    // ---- this lane's rows' weights of tokens g + 8 m, then over the four lanes of a token ----
    const int t0 = at.step * kTile;
    const bool masked = t0 + kTile > at.n.len - at.n.nq + 1;  // not every query sees all of the step
    float sum[4], own_scale = 0.f;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float ks = __shfl_sync(0xffffffffu, scales[0], g + 8 * m);
      if (m == q4) own_scale = ks;
      sum[m] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float p = ex2(fmaf(z[m / 2][nt][(m % 2) * 2 + j], finite_factor(ks, qscale[nt][j]), -y[nt][j]));
          sum[m] += masked && t0 + g + 8 * m > limit[nt][j] ? 0.f : p;
        }
    }
    // half of the sums to the lane two on, half of these to the next one
    const bool up = q4 & 2, odd = q4 & 1;
    float s0 = up ? sum[2] : sum[0], s1 = up ? sum[3] : sum[1];
    s0 += __shfl_xor_sync(0xffffffffu, up ? sum[0] : sum[2], 2);
    s1 += __shfl_xor_sync(0xffffffffu, up ? sum[1] : sum[3], 2);
    const float mine = (odd ? s1 : s0) + __shfl_xor_sync(0xffffffffu, odd ? s0 : s1, 1);
    if (t0 + own < at.n.len)  // (a token that is absent has whatever the stage held)
      *weight_at(at) = (a.decay != 0.f ? a.decay * olds[0] : 0.f) + (own_scale == 0.f ? 0.f : mine);
    __syncwarp();  // every lane has read the stage before it is filled again

    // ---- on to the next step ----
    if (i + 1 < count) advance(c, a, at);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      scales[k] = scales[k + 1];
      olds[k] = olds[k + 1];
      begins[k] = begins[k + 1];
    }
    if (++stage == kStages) stage = 0, parity ^= 1;
  }
  if (bad) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
}

template <int D, int FMT, int NT>
cudaError_t launch_few(const Cache& c, const WeighArgs& a, cudaStream_t s) {
  constexpr int kSmem = kWarps * kStages * kTile * D;
  static std::atomic<uint64_t> told{0};
  static std::atomic<int> per_sm{0};
  cudaError_t e = allow_smem(weigh_few_kernel<D, FMT, NT>, kSmem, told);
  if (e != cudaSuccess) return e;
  int ctas = per_sm.load(std::memory_order_relaxed);
  if (ctas == 0) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&ctas, weigh_few_kernel<D, FMT, NT>, 32 * kWarps,
                                                      kSmem);
    if (e != cudaSuccess) return e;
    if (ctas < 1) return cudaErrorLaunchOutOfResources;
    per_sm.store(ctas, std::memory_order_relaxed);
  }
  // no more CTAs than steps that the tables have room for
  const long long most = static_cast<long long>(c.L) * c.B * c.H *
                         ((min(a.cap, c.max_blocks * c.bs) + kTile - 1) / kTile);
  const int grid = static_cast<int>(min(most, static_cast<long long>(a.num_sms) * ctas));
  return launch(weigh_few_kernel<D, FMT, NT>, grid, 32 * kWarps, kSmem, s, c, a, make_div(c.bs));
}

template <int D, int FMT>
cudaError_t launch_rows(const Cache& c, const WeighArgs& a, cudaStream_t s) {
  const long long R = static_cast<long long>(a.G) * a.n;
  if (R <= 8) return launch_few<D, FMT, 1>(c, a, s);
  if (R <= 16) return launch_few<D, FMT, 2>(c, a, s);
  if (R <= 32) return launch_few<D, FMT, 4>(c, a, s);
  return launch_weigh_many(c, FMT, a, s);
}

}  // namespace

cudaError_t launch_weigh(const Cache& c, int format, const WeighArgs& a, cudaStream_t s) {
  if (c.d == 64)
    return format == KVC_CACHE8_E4M3 ? launch_rows<64, KVC_CACHE8_E4M3>(c, a, s)
                                     : launch_rows<64, KVC_CACHE8_INT8>(c, a, s);
  return format == KVC_CACHE8_E4M3 ? launch_rows<128, KVC_CACHE8_E4M3>(c, a, s)
                                   : launch_rows<128, KVC_CACHE8_INT8>(c, a, s);
}

}  // namespace prompt
}  // namespace kvc
