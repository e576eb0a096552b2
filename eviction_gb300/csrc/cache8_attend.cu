// cache8_attend.cu -- attention of the newest tokens' queries over the 8-bit
// paged cache (kvc_cache8_attend), for few queries: decode steps.
//
//   out_r = sum_t w_rt v_t / sum_t w_rt,  w_rt = exp(scale q_r . k_t)
//
// for the R = G n query rows of a KV head.  Every key and value is read once for
// all rows, 2 d bytes a token, and the arithmetic on it is 4 R d operations: the
// kernel is bound by memory as long as the instructions around the loads keep up.
// Each warp has tokens and a ring of stages in shared memory of its own: 32 tokens'
// keys, values and scales a stage, filled by asynchronous 16-byte copies (absent
// tokens are filled with zeros), so that the loop has no barrier and enough bytes
// in flight to cover the latency of HBM.
//
// Per 16 tokens a warp computes S^T = K Q^T (m16n8k16, tokens on the M axis) and
// O^T += V^T P^T (values on the M axis), so that the 8 columns are query rows and
// nothing is wasted on a 16-row query tile that has 7 rows.  The order of d inside
// the products is free: 16 bytes of a key row are four k-slices' worth of a lane's A
// fragment as they stand, with Q loaded in the same order; 16 bytes of 4 tokens'
// values become A fragments by two byte permutes for each pair of tokens.  The
// 16-byte chunks of a row are swizzled so that both reads are free of bank
// conflicts (of 128 values; 64 have one on the values).  Codes are converted to
// fp16, which holds both formats exactly; q is scaled by a power of two per row so
// that fp16 holds it as well.
//
// The softmax is kept in base 2 with a running maximum.  The value scale 2^e of a
// token's block joins its logit (x = z + e) instead of its weight, so that the
// fp16 weights of the second product stay near 1 whatever the blocks' scales are;
// the sum uses 2^-e again, in fp32.  The maximum is only raised when a logit
// passes it by 2^8 (fp16 has the room), which turns the reduction over lanes into
// one vote per 32 tokens.
//
// Work is the list of all heads' steps of 32 tokens, one after another.  Many heads:
// small CTAs, three on an SM, take equal stretches of the list, whatever the lengths
// are, and walk the heads that they meet (a head counts as a few steps more than it has,
// what it takes to begin and end it).  Few heads: one large CTA per SM takes a
// part of one head.  A head within one CTA is finished there; the parts of one that
// is not go to the workspace, and the last CTA of it to finish joins them in order
// (the result does not depend on which one that is).
//
// Measured: 64 sequences of 612 to 1112 tokens, 8 KV heads of 4 (114 MB) 26.9 us, 4.2
// TB/s; 4 sequences of 32768, 4 heads of 7, int8 (134 MB) 30 us, 4.5 TB/s; one head of
// 768 tokens 7.7 us.  Loads straight into registers, one step ahead, took 37 and 52 us.
#include "cache8_attend.cuh"

namespace kvc {
namespace cache8 {
namespace {

constexpr int kTile = 32;        // tokens of one step of a warp
constexpr int kRowTile = 16;     // query rows of a stretch at most
constexpr int kStages = 2;
constexpr int kSmWarps = 12;     // warps of an SM, by registers and shared memory
constexpr int kMaxCtas = kCounters;  // CTAs of a call
constexpr float kSlack = 8.f;    // log2 of how far a weight may pass 1
// Steps that beginning and ending a head costs a small CTA.  In us at 0 / 4 / 8 / 12 / 16:
//   512 heads of 4 rows, 612-1112 tokens       28.6 / 27.7 / 26.8 / 27.2 / 27.5
//   1024 heads of 4 rows, 40-300 tokens        28.7 / 23.5 / 22.9 / 23.1 / 23.2
//   256 heads of 8 rows, 500-4000, d 64        23.2 / 22.2 / 21.7 / 21.5 / 21.8
//   256 heads of 16 rows, 1000-3000            42.7 / 42.0 / 40.7 / 41.4 / 41.6
//   192 heads of 5 rows, all 2048, int8        26.6 / 26.0 / 25.4 / 24.9 / 25.7
//   256 heads of 7 rows, 64-8000               54.2 / 52.3 / 50.9 / 50.7 / 51.0
//   128 heads of 28 rows, 1000-1536            33.9 / 32.7 / 32.6 / 32.7 / 31.8
constexpr int kHeadCost = 8;
constexpr int kMinRounds = 3;    // steps of a CTA's warps at least, before a head is cut

struct Split {
  int row_tiles;  // of a head
  float* part;    // [2 kMaxCtas][kRowTile][D + 2]: maximum, sum, values
  int* arrived;   // [kMaxCtas] zero between calls
};

// Asynchronous copies global -> shared; where `there` is false, zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from),
               "r"(there ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A stage of a warp's ring: kTile rows of keys, as many of values, their scales.
template <int D>
struct Stage {
  static constexpr int kKeys = 0, kValues = kTile * D, kKeyScales = 2 * kTile * D,
                       kValueScales = kKeyScales + kTile * 4, kBytes = kValueScales + kTile * 4;
  // place of 16-byte chunk ch of row r
  static __device__ __forceinline__ int at(int r, int ch) {
    const int f = D == 128 ? ((((r >> 1) & 3) << 1) ^ ((r & 1) << 2)) : ((r >> 1) & 3);
    return r * D + ((ch ^ f) << 4);
  }
};

// Values in the order of the second product's A operand: from four codes of each of
// two tokens, pairs (token x, token y) of codes 0 and 1 (HIGH: 2 and 3).  (int8 codes
// left biased, with the bias taken off the sums, saved a tenth of the instructions
// and lost columns much smaller than their block's largest value.)
template <int FMT, bool HIGH>
__device__ __forceinline__ void value_pairs(uint32_t x, uint32_t y, uint32_t& even, uint32_t& odd) {
  halves<FMT>(__byte_perm(x, y, HIGH ? 0x7362 : 0x5140), even, odd);
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <int D, int NT, int W>
constexpr int smem_bytes() {
  const int ring = W * kStages * Stage<D>::kBytes, parts = W * 8 * NT * (D + 4) * 4;
  return ring > parts ? ring : parts;
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xffffffffu, v); }

// Steps of one head of sequence b; 0 for one that has no queries or is refused.
__device__ __forceinline__ int steps_of(const Cache& c, const AttendArgs& a, int b, bool* bad) {
  bool wrong = false;
  const int len = length_of(c, b, &wrong);
  const int nq = a.n_q ? a.n_q[b] : a.n;
  if (wrong || nq < 0 || nq > a.n) {
    *bad = true;
    return 0;
  }
  return nq == 0 ? 0 : max((len + kTile - 1) / kTile, 1);
}

template <int D, int FMT, int NT, int W>
__global__ void __launch_bounds__(32 * W, kSmWarps / W)
    attend_few_kernel(Cache c, AttendArgs a, Split sp, Div by_bs) {
  constexpr int KV = D / 64;   // 16-byte loads of a key row per lane
  constexpr int MT = D / 16;   // 16-value tiles of the output
  constexpr int Q = 8 * NT;    // query rows
  constexpr int OS = D + 4;    // row stride of the parts in shared memory
  constexpr int TPR = D / kPer;
  constexpr int kThreads = 32 * W;
  using St = Stage<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  auto s_o = reinterpret_cast<float(*)[Q][OS]>(smem);  // after a head's loop, the warps' parts
  __shared__ float s_m[W][Q], s_l[W][Q];
  __shared__ int s_last;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, q4 = lane % 4;
  bool bad = false, unused = false;

  before_all();

  // ---- this CTA's work: steps [begin, ...) of a head, `left` steps in all ----
  // (every warp computes it for itself; all counts are below 2^31, checked on the host)
  const int heads = c.H * sp.row_tiles;  // of one sequence and layer
  int own_steps[2] = {0, 0};             // of the first 64 sequences, by lane
  int all = 0, most = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    const int n = b0 + lane < c.B ? steps_of(c, a, b0 + lane, &bad) : 0;
    if (b0 == 0) own_steps[0] = n;
    if (b0 == 32) own_steps[1] = n;
    all += n;
    most = max(most, n);
  }
  all = warp_sum(all);
  if (blockIdx.x == 0 && bad) atomicOr(c.status, KVC_STATUS_BAD_INDEX);  // one report is enough
  bad = false;
  // the sum over sequences of f(steps)
  auto steps_at = [&](int b0) {
    return b0 == 0 ? own_steps[0] : b0 == 32 ? own_steps[1]
           : b0 + lane < c.B ? steps_of(c, a, b0 + lane, &unused) : 0;
  };
  auto sum_over = [&](auto f) {
    int v = 0;
    for (int b0 = 0; b0 < c.B; b0 += 32) v += f(steps_at(b0));
    return warp_sum(v);
  };
  // the sequence in which place `at` of the sum over sequences of heads * f(steps)
  // lies, the place within it and the sequence's steps
  auto find = [&](int at, auto f, int* in, int* steps) {
    int before = 0;
    for (int b0 = 0;; b0 += 32) {
      const int own = steps_at(b0), n = heads * f(own);
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      const int chunk = __shfl_sync(0xffffffffu, incl, 31);
      if (at < before + chunk || b0 + 32 >= c.B) {
        const int place = __ffs(__ballot_sync(0xffffffffu, at < before + incl)) - 1;
        *in = at - before - __shfl_sync(0xffffffffu, incl - n, place);
        *steps = __shfl_sync(0xffffffffu, own, place);
        return b0 + place;
      }
      before += chunk;
    }
  };
  // (in the list, each head of a small CTA's kernel has kHeadCost places before its steps)
  constexpr int kCost = W == kSmWarps ? 0 : kHeadCost;
  auto places = [](int n) { return n > 0 ? n + kCost : 0; };
  if (kCost > 0) all += kCost * sum_over([](int n) { return n > 0; });
  const int n_cta = gridDim.x, total = all * heads * c.L;
  if (total == 0) return;
  int chunk = max(div_up(total, n_cta), kMinRounds * W);
  int l, b, head, begin, left, steps;  // (steps of a head of sequence b)
  if constexpr (W == kSmWarps) {
    // parts of at most `chunk` steps, so many that the grid has a CTA for each: with
    // n_cta / (heads in all) parts of the longest head that is so; where lengths
    // differ, the even share and one in between may do and are tried first
    most = __reduce_max_sync(0xffffffffu, most);
    const int seqs = sum_over([](int n) { return n > 0; }) * heads * c.L;
    const int safe = max(div_up(most, max(n_cta / seqs, 1)), kMinRounds * W);
    if (seqs * most == total) chunk = safe;
    int parts_all = 0;  // of a layer
    for (int i = 0; i < 3; ++i) {
      parts_all = heads * sum_over([&](int n) { return div_up(n, chunk); });
      if (parts_all * c.L <= n_cta) break;
      chunk = i == 0 ? (chunk + safe + 1) / 2 : safe;
    }
    if (static_cast<int>(blockIdx.x) >= parts_all * c.L) return;
    l = blockIdx.x / parts_all;
    int in;
    b = find(blockIdx.x % parts_all, [&](int n) { return div_up(n, chunk); }, &in, &steps);
    const int parts = div_up(steps, chunk);
    head = in / parts;
    begin = in % parts * chunk;
    left = min(chunk, steps - begin);
  } else {
    const int lo = blockIdx.x * chunk;
    if (static_cast<long long>(blockIdx.x) * chunk >= total) return;
    l = lo / (all * heads);
    int in;
    b = find(lo % (all * heads), places, &in, &steps);
    head = in / (steps + kCost);
    begin = in % (steps + kCost) - kCost;  // below 0: before the head's first step
    left = min(chunk, total - lo);
  }

  uint8_t* ring = smem + warp * (kStages * St::kBytes);
  const uint32_t ring_addr = smem_u32(ring);

  int at = blockIdx.x * chunk;  // place in the list, of step `begin`
  for (;;) {
    if (begin < 0) {  // on to the first step, if it is this CTA's
      left += begin;
      at -= begin;
      begin = 0;
      if (left <= 0) break;
    }
    const int h = head / sp.row_tiles, rt = head % sp.row_tiles;
    const int end = min(steps, begin + left);
    const int len = c.seq_len[b];
    const int nq = a.n_q ? a.n_q[b] : a.n;
    const int rows = min(a.G * nq - rt * Q, Q);  // of this tile: r = rt * Q + 0..rows-1
    const int32_t* table = c.table + static_cast<size_t>(b) * c.max_blocks;
    const uint8_t* kp = c.pool[0] + block_row(c, l, 0, h) * D;
    const uint8_t* vp = c.pool[1] + block_row(c, l, 0, h) * D;
    const float* ksp = c.scale[0] + scale_at(c, l, 0, h);
    const float* vsp = c.scale[1] + scale_at(c, l, 0, h);

    // Lane i looks after token i of a step.
    auto block_of = [&](int step) {
      const int t = step * kTile + lane;
      return step < end && t < len ? table[by_bs.div(t)] : -1;
    };
    // start the copies of a step, whose tokens lie in the lanes' blocks `blk`
    auto fetch = [&](int step, int blk, int stage) {
      const uint32_t to = ring_addr + stage * St::kBytes;
      if (step < end) {
        const int t = step * kTile + lane;
        int row = -1;
        if (t < len) {
          if (blk < 0 || blk >= c.n_blocks)
            bad = true;
          else
            row = blk * c.H * by_bs.bs + (t - by_bs.div(t) * by_bs.bs);  // < 2^31: checked on the host
        }
        const size_t sc = row < 0 ? 0 : static_cast<size_t>(blk) * c.H;
        copy4(to + St::kKeyScales + lane * 4, ksp + sc, row >= 0);
        copy4(to + St::kValueScales + lane * 4, vsp + sc, row >= 0);
        constexpr int CH = D / 16, RPI = 32 / CH;  // chunks of a row, rows of one copy
#pragma unroll
        for (int i = 0; i < kTile / RPI; ++i) {
          const int r = lane / CH + i * RPI, ch = lane % CH;
          const int from = __shfl_sync(0xffffffffu, row, r);
          const size_t off = static_cast<size_t>(max(from, 0)) * D + ch * 16;
          copy16(to + St::kKeys + St::at(r, ch), kp + off, from >= 0);
          copy16(to + St::kValues + St::at(r, ch), vp + off, from >= 0);
        }
      }
      copies_commit();
    };

    // ---- queries: row g of each 8-row tile, in the order of the key reads ----
    // row r is head r / nq of the group, query r % nq; the loads start before the first
    // step's, which wait for the table
    int step = rows > 0 ? begin + warp : end;
    int blk = block_of(step);
    int next = block_of(step + W);
    uint4 raw[NT][KV][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = rt * Q + nt * 8 + g;
      const bool there = nt * 8 + g < rows;
      const uint16_t* qp = a.q.at(l, b, h * a.G + (there ? r / nq : 0), there ? r % nq : 0);
#pragma unroll
      for (int k = 0; k < KV; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          raw[nt][k][i] = there ? *reinterpret_cast<const uint4*>(qp + (k * 4 + q4) * 16 + i * 8)
                                : make_uint4(0, 0, 0, 0);
    }
    fetch(step, blk, 0);
    int stage = 0;
    uint32_t qf[NT][KV * 4][2];
    float qscale[NT][2];  // of rows 2 q4, 2 q4 + 1: scale log2(e) 2^e
    int limit[NT][2];     // last token that they see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const auto& w = raw[nt];
      float mx = 0.f;
#pragma unroll
      for (int k = 0; k < KV; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t x[4] = {w[k][i].x, w[k][i].y, w[k][i].z, w[k][i].w};
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
        for (int i = 0; i < 2; ++i) {
          const uint32_t x[4] = {w[k][i].x, w[k][i].y, w[k][i].z, w[k][i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            qf[nt][k * 4 + i * 2 + j / 2][j % 2] =
                half2_of(bf16_lo(x[j]) * down, bf16_hi(x[j]) * down);
        }
      const float up = finite_factor(a.scale_log2, exp2_int(e));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        qscale[nt][i] = __shfl_sync(0xffffffffu, up, (2 * q4 + i) * 4);
        limit[nt][i] = len - nq + (rt * Q + nt * 8 + 2 * q4 + i) % nq;
      }
    }

    float o[NT][MT][4];
    float m[NT][2], sum[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[nt][i][j] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      sum[nt][0] = sum[nt][1] = 0.f;
    }

    for (; step < end; step += W) {
      const int t0 = step * kTile;
      fetch(step + W, next, stage ^ 1);
      next = block_of(step + 2 * W);
      copies_wait<1>();
      __syncwarp();  // all lanes' copies of this step are there
      const uint8_t* st = ring + stage * St::kBytes;
      stage ^= 1;

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
          const uint8_t* keys = st + St::kKeys;
          const uint4 k0 = *reinterpret_cast<const uint4*>(keys + St::at(mt * 16 + g, k * 4 + q4));
          const uint4 k1 =
              *reinterpret_cast<const uint4*>(keys + St::at(mt * 16 + g + 8, k * 4 + q4));
          const uint32_t x[4] = {k0.x, k0.y, k0.z, k0.w};
          const uint32_t y[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a0, a1, a2, a3;
            halves<FMT>(x[j], a0, a2);
            halves<FMT>(y[j], a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma(z[mt][nt], a0, a1, a2, a3, qf[nt][k * 4 + j][0], qf[nt][k * 4 + j][1]);
          }
        }

      // ---- weights: this lane's tokens are g + 8 i ----
      const float* k_scales = reinterpret_cast<const float*>(st + St::kKeyScales);
      const float* v_scales = reinterpret_cast<const float*>(st + St::kValueScales);
      float back[4];  // 2^-e, 0 for an absent token
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float ks = k_scales[g + 8 * i], vs = v_scales[g + 8 * i];
        const int e = static_cast<int>(__float_as_uint(vs) >> 23) - 127;
        // (an absent token has zeros for key and scales: its logit becomes -inf)
        const float ef = vs == 0.f ? -INFINITY : static_cast<float>(e);
        back[i] = vs == 0.f ? 0.f : exp2_int(-e);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float& x = z[i / 2][nt][(i % 2) * 2 + j];
            x = fmaf(x, finite_factor(ks, qscale[nt][j]), ef);
          }
      }
      if (t0 + kTile > len - nq + 1) {  // not every query sees all of the step
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (t0 + g + 8 * i > limit[nt][j]) z[i / 2][nt][(i % 2) * 2 + j] = -INFINITY;
      }
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float x = fmaxf(fmaxf(z[0][nt][j], z[0][nt][2 + j]), fmaxf(z[1][nt][j], z[1][nt][2 + j]));
          up = up || x - m[nt][j] > kSlack;  // (not x > m + kSlack: that sum may round)
        }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = fmaxf(fmaxf(z[0][nt][j], z[0][nt][2 + j]), fmaxf(z[1][nt][j], z[1][nt][2 + j]));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            x = fmaxf(x, m[nt][j]);
            const float f = x > m[nt][j] ? ex2(m[nt][j] - x) : 1.f;
            m[nt][j] = x;
            sum[nt][j] *= f;
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              o[nt][t][j] *= f;
              o[nt][t][2 + j] *= f;
            }
          }
      }
      uint32_t p[2][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
        const float m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float w0 = ex2(z[i / 2][nt][(i % 2) * 2] - m0);
          const float w1 = ex2(z[i / 2][nt][(i % 2) * 2 + 1] - m1);
          sum[nt][0] = fmaf(w0, back[i], sum[nt][0]);
          sum[nt][1] = fmaf(w1, back[i], sum[nt][1]);
          p[i / 2][nt][i % 2] = transpose8x8(half2_of(w0, w1));
        }
      }

      // ---- O^T += V^T P^T ----
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        uint32_t vr[4][MT / 2];  // 2 MT codes of the tokens 2 q4, 2 q4 + 1, 2 q4 + 8, 2 q4 + 9
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = kt * 16 + 2 * q4 + (i & 1) + 8 * (i >> 1);
          const uint8_t* from = st + St::kValues + St::at(r, g * MT / 8) + (g * 2 * MT) % 16;
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(from);
            vr[i][0] = v.x, vr[i][1] = v.y, vr[i][2] = v.z, vr[i][3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(from);
            vr[i][0] = v.x, vr[i][1] = v.y;
          }
        }
#pragma unroll
        for (int j = 0; j < MT / 2; ++j) {
          uint32_t a0, a1, a2, a3;
          value_pairs<FMT, false>(vr[0][j], vr[1][j], a0, a1);
          value_pairs<FMT, false>(vr[2][j], vr[3][j], a2, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma(o[nt][2 * j], a0, a1, a2, a3, p[kt][nt][0], p[kt][nt][1]);
          value_pairs<FMT, true>(vr[0][j], vr[1][j], a0, a1);
          value_pairs<FMT, true>(vr[2][j], vr[3][j], a2, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma(o[nt][2 * j + 1], a0, a1, a2, a3, p[kt][nt][0], p[kt][nt][1]);
        }
      }
      __syncwarp();  // every lane has read the stage before it is filled again
    }

    // ---- join the warps ----
    copies_wait<0>();
    __syncthreads();  // the rings become the parts
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float s = sum[nt][i];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        const int r = nt * 8 + 2 * q4 + i;
        if (g == 0) {
          s_m[warp][r] = m[nt][i];
          s_l[warp][r] = s;
        }
        // this lane's values: tile t has d = 2 (g MT + t) in c0/c1 and one more in c2/c3
#pragma unroll
        for (int t = 0; t < MT; t += 2)
          *reinterpret_cast<float4*>(&s_o[warp][r][2 * (g * MT + t)]) =
              make_float4(o[nt][t][i], o[nt][t][2 + i], o[nt][t + 1][i], o[nt][t + 1][2 + i]);
      }
    __syncthreads();
    constexpr size_t kSlot = static_cast<size_t>(kRowTile) * (D + 2);
    const bool whole_head = begin == 0 && end == steps;
    float* slot = sp.part + (2 * static_cast<size_t>(blockIdx.x) + (begin == 0 ? 1 : 0)) * kSlot;
    for (int i = threadIdx.x; i < Q * TPR; i += kThreads) {
      const int r = i / TPR, d0 = (i % TPR) * kPer;
      if (r >= rows) continue;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) mm = fmaxf(mm, s_m[w][r]);
      const float ref = mm == -INFINITY ? 0.f : mm;
      float x[kPer], s = 0.f;
#pragma unroll
      for (int k = 0; k < kPer; ++k) x[k] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = ex2(s_m[w][r] - ref);
        s += f * s_l[w][r];
#pragma unroll
        for (int k = 0; k < kPer; ++k) x[k] += f * s_o[w][r][d0 + k];
      }
      if (whole_head) {
        write_row(c, a, l, b, h, rt * Q + r, nq, d0, x, mm, s);
      } else {
        float* to = slot + r * (D + 2);
#pragma unroll
        for (int k = 0; k < kPer; k += 2)
          *reinterpret_cast<float2*>(to + 2 + d0 + k) = make_float2(x[k], x[k + 1]);
        if (d0 == 0) *reinterpret_cast<float2*>(to) = make_float2(mm, s);
      }
    }

    // ---- join the parts of a head: the last CTA of it to arrive ----
    if (!whole_head && rows > 0) {
      // the CTAs c0 .. c0 + n_part - 1 have this head
      int c0, n_part;
      if constexpr (W == kSmWarps) {
        c0 = blockIdx.x - begin / chunk;
        n_part = div_up(steps, chunk);
      } else {
        const int head_lo = at - begin;
        c0 = head_lo / chunk;
        n_part = (head_lo + steps - 1) / chunk - c0 + 1;
      }
      __syncthreads();  // the part is written, by all threads
      if (threadIdx.x == 0) {
        int seen;
        asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                     : "=r"(seen)
                     : "l"(sp.arrived + c0)
                     : "memory");
        s_last = seen == n_part - 1;
        if (s_last) sp.arrived[c0] = 0;  // ready for the next call
      }
      __syncthreads();
      if (s_last) {
        // the first CTA's part of a head that begins in it, then the others'
        auto part_of = [&](int i) {
          return sp.part + (2 * static_cast<size_t>(c0 + i) + (i == 0 ? 1 : 0)) * kSlot;
        };
        for (int i = threadIdx.x; i < Q * TPR; i += kThreads) {
          const int r = i / TPR, d0 = (i % TPR) * kPer;
          if (r >= rows) continue;
          float mm = -INFINITY, x[kPer], s = 0.f;
#pragma unroll
          for (int k = 0; k < kPer; ++k) x[k] = 0.f;
          // a few parts at a time, all their loads in flight together
          constexpr int kBatch = 6;
          for (int w0 = 0; w0 < n_part; w0 += kBatch) {
            float2 ml[kBatch], v[kBatch][kPer / 2];
            float top = mm;
#pragma unroll
            for (int w = 0; w < kBatch; ++w) {
              const float* from = part_of(min(w0 + w, n_part - 1)) + r * (D + 2);
              ml[w] = __ldcg(reinterpret_cast<const float2*>(from));
#pragma unroll
              for (int k = 0; k < kPer / 2; ++k)
                v[w][k] = __ldcg(reinterpret_cast<const float2*>(from + 2 + d0) + k);
            }
#pragma unroll
            for (int w = 0; w < kBatch; ++w) {
              if (w0 + w >= n_part) ml[w] = make_float2(-INFINITY, 0.f);
              top = fmaxf(top, ml[w].x);
            }
            const float ref = top == -INFINITY ? 0.f : top;
            const float keep = mm == -INFINITY ? 0.f : ex2(mm - ref);
            s *= keep;
#pragma unroll
            for (int k = 0; k < kPer; ++k) x[k] *= keep;
            mm = top;
#pragma unroll
            for (int w = 0; w < kBatch; ++w) {
              if (w0 + w < n_part) {
                const float f = ex2(ml[w].x - ref);
                s += f * ml[w].y;
#pragma unroll
                for (int k = 0; k < kPer / 2; ++k) {
                  x[2 * k] += f * v[w][k].x;
                  x[2 * k + 1] += f * v[w][k].y;
                }
              }
            }
          }
          write_row(c, a, l, b, h, rt * Q + r, nq, d0, x, mm, s);
        }
      }
    }

    // ---- the next head ----
    left -= end - begin;
    if (W == kSmWarps || left == 0) break;
    at += end - begin;
    begin = -kCost;
    if (++head == heads) {
      head = 0;
      do {
        if (++b == c.B) {
          b = 0;
          ++l;
        }
        steps = steps_of(c, a, b, &unused);
      } while (steps == 0);
    }
    __syncthreads();  // the parts become the rings again
  }
  if (bad) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
}

template <int D, int FMT, int NT, int W>
cudaError_t launch_few(const Cache& c, const AttendArgs& a, const Split& sp, cudaStream_t s) {
  constexpr int smem = smem_bytes<D, NT, W>();
  auto* kernel = attend_few_kernel<D, FMT, NT, W>;
  static std::atomic<uint64_t> told{0};
  const cudaError_t e = allow_smem(kernel, smem, told);
  if (e != cudaSuccess) return e;
  const int grid = min(a.num_sms * (kSmWarps / W), kMaxCtas);
  return launch(kernel, grid, 32 * W, smem, s, c, a, sp, make_div(c.bs));
}

template <int D, int FMT>
cudaError_t launch_few(const Cache& c, const AttendArgs& a, cudaStream_t s) {
  const int R = a.G * a.n, nt = R > 8 ? 2 : 1;
  Split sp;
  sp.row_tiles = (R + 8 * nt - 1) / (8 * nt);
  sp.arrived = static_cast<int*>(a.workspace);
  sp.part = reinterpret_cast<float*>(sp.arrived + kCounters);
  // One large CTA per SM where whole parts of at most 76 heads fill three quarters of the
  // SMs; else small ones, which share all steps evenly and whose beginnings and ends
  // overlap.  Large / small in us: 20 heads of 4096 tokens 12.9 / 14.9, 32 of 16384
  // 28.7 / 34, 48 of 4096 14.2 / 17.1, 64 of 4096 17.1 / 18.8.
  const long long heads = static_cast<long long>(c.L) * c.B * c.H * sp.row_tiles;
  const bool large = 2 * heads <= a.num_sms && 4 * heads * (a.num_sms / heads) >= 3 * a.num_sms;
  if (nt == 1)
    return large ? launch_few<D, FMT, 1, 12>(c, a, sp, s) : launch_few<D, FMT, 1, 4>(c, a, sp, s);
  return large ? launch_few<D, FMT, 2, 12>(c, a, sp, s) : launch_few<D, FMT, 2, 4>(c, a, sp, s);
}

}  // namespace

// Which kernel: this one reads a head's tokens once for each 16 query rows, the other
// takes 128 rows at a time but starts and turns slower.  By the product of heads,
// 16-row tiles and tokens (the table's capacity), this one / the other in us:
//   4 heads x 2048 tokens, 112 rows (57 k)     17 / 19
//   32 x 2048, 28 rows (131 k)                 17 / 23;   56 rows (262 k)  27 / 24
//   128 x 1536, 28 rows (393 k)                32 / 35;   35 rows (590 k)  41 / 36
//   16 x 16384, 28 rows (524 k)                33 / 44;   56 rows (1 M)    55 / 47
//   512 x 860, 32 rows (881 k)                 65 / 65;   64 rows (1.8 M) 109 / 66
constexpr int kFewRows = 32;
constexpr long long kFewWork = 150'000;

cudaError_t launch_attend(const Cache& c, int format, const AttendArgs& a, cudaStream_t s) {
  const int R = a.G * a.n;
  const long long work = static_cast<long long>(c.L) * c.B * c.H * ((R + 15) / 16) *
                         (static_cast<long long>(c.max_blocks) * c.bs);
  if (R > kFewRows && work >= kFewWork) return launch_attend_many(c, format, a, s);
  if (c.d == 64)
    return format == KVC_CACHE8_E4M3 ? launch_few<64, KVC_CACHE8_E4M3>(c, a, s)
                                     : launch_few<64, KVC_CACHE8_INT8>(c, a, s);
  return format == KVC_CACHE8_E4M3 ? launch_few<128, KVC_CACHE8_E4M3>(c, a, s)
                                   : launch_few<128, KVC_CACHE8_INT8>(c, a, s);
}

}  // namespace cache8

size_t cache8_attend_workspace(int d) {
  using namespace cache8;
  const size_t few = kMaxCtas * 2 * static_cast<size_t>(kRowTile) * (d + 2) * sizeof(float);
  const size_t many = attend_many_parts_bytes(d);
  return kCounters * sizeof(int) + (few > many ? few : many);
}

}  // namespace kvc
