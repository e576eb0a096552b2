// cache8_attend.cu -- attention of the newest tokens' queries over the 8-bit
// paged cache (kvc_cache8_attend), for few queries: decode steps.
//
//   out_r = sum_t w_rt v_t / sum_t w_rt,  w_rt = exp(scale q_r . k_t)
//
// for the R = G n query rows of a KV head.  Every key and value is read once for
// all rows, 2 d bytes a token, and the arithmetic on it is 4 R d operations: the
// kernel is bound by memory as long as the instructions around the loads keep up.
// A warp therefore takes its tokens straight from global memory into registers,
// in the layout the tensor-core instruction wants (no shared memory, no barrier in
// the loop), and holds the next 16 tokens' loads in flight while it works on the
// present ones.
//
// Per 16 tokens a warp computes S^T = K Q^T (m16n8k16, tokens on the M axis) and
// O^T += V^T P^T (values on the M axis), so that the 8 columns are query rows and
// nothing is wasted on a 16-row query tile that has 7 rows.  The order of d inside
// the products is free: a lane's 16-byte load of a key row is four k-slices' worth
// of its A fragment as it stands, with Q loaded in the same order; a lane's value
// loads (16 bytes of 4 tokens) become A fragments by two byte permutes for each
// pair of tokens.  Codes are converted to fp16, which holds both formats exactly;
// q is scaled by a power of two per row so that fp16 holds it as well.
//
// The softmax is kept in base 2 with a running maximum.  The value scale 2^e of a
// token's block joins its logit (x = z + e) instead of its weight, so that the
// fp16 weights of the second product stay near 1 whatever the blocks' scales are;
// the sum uses 2^-e again, in fp32.  The maximum is only raised when a logit
// passes it by 2^8 (fp16 has the room), which turns the reduction over lanes into
// one vote per 16 tokens.
//
// Tokens are split over the warps of a CTA and, when the heads alone do not fill
// the GPU, over CTAs; the last CTA of a head to finish joins the parts in order.
#include "cache8.cuh"

namespace kvc {
namespace cache8 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16;          // tokens of one step of a warp
constexpr int kRowTile = 16;       // query rows of a CTA at most
constexpr int kMaxParts = 2048;    // CTAs of a call that splits sequences
constexpr int kMinTiles = 2 * kWarps;  // tiles of a part at least
constexpr float kSlack = 8.f;      // log2 of how far a weight may pass 1

// Division by the block size: floor(t / bs) = umulhi(t, mul) >> shift for
// 0 <= t < 2^31 (bs > 1).
struct Div {
  uint32_t mul;
  int shift, bs;
  __device__ __forceinline__ int div(int t) const {
    return mul ? static_cast<int>(__umulhi(static_cast<uint32_t>(t), mul) >> shift) : t;
  }
};
Div make_div(int bs) {
  if (bs == 1) return {0, 0, 1};
  int s = 0;
  while ((1 << s) < bs) ++s;  // 2^(s-1) < bs <= 2^s
  return {static_cast<uint32_t>((1ull << (31 + s)) / bs + 1), s - 1, bs};
}

struct Split {
  int per_unit;    // CTAs of a head and row tile
  int row_tiles;
  float* part;     // [kMaxParts][kRowTile][D + 2]
  int* arrived;    // [kMaxParts] zero between calls
};

__device__ __forceinline__ uint4 load16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p));
  return v;
}

// Codes as signed integers, biased to 0..255, behind the exponent of 1024: the
// fp16 number 1024 + u, from which 1152 leaves the value.
__device__ __forceinline__ uint32_t unbias(uint32_t h) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
  return r;
}

// Four codes to two half2: (0, 1), (2, 3).
template <int FMT>
__device__ __forceinline__ void halves(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == KVC_CACHE8_E4M3) {
    lo = e4m3_to_half2(w);
    hi = e4m3_to_half2(w >> 16);
  } else {
    w ^= 0x80808080u;
    lo = unbias(__byte_perm(w, 0x64646464u, 0x4140));
    hi = unbias(__byte_perm(w, 0x64646464u, 0x4342));
  }
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

__device__ __forceinline__ uint32_t half2_of(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// One row tile of one head over one part of its tokens.
template <int D, int FMT, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : 3)
    attend_few_kernel(Cache c, AttendArgs a, Split sp, Div by_bs) {
  constexpr int KV = D / 64;   // 16-byte loads of a key row per lane
  constexpr int MT = D / 16;   // 16-value tiles of the output
  constexpr int Q = 8 * NT;    // query rows
  constexpr int OS = D + 4;    // row stride of the parts in shared memory
  __shared__ float s_o[kWarps][Q][OS];
  __shared__ float s_m[kWarps][Q], s_l[kWarps][Q];
  __shared__ int s_last;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, q4 = lane % 4;
  const int part = blockIdx.x % sp.per_unit;
  const int ur = blockIdx.x / sp.per_unit;  // unit and row tile
  const int rt = ur % sp.row_tiles;
  const int u = ur / sp.row_tiles;
  const int h = u % c.H, b = (u / c.H) % c.B, l = u / (c.H * c.B);
  bool bad = false;
  const int len = length_of(c, b, &bad);
  const int nq = a.n_q ? a.n_q[b] : a.n;
  if (bad || nq < 0 || nq > a.n) {
    if (threadIdx.x == 0) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
    return;
  }
  const int rows = min(a.G * nq - rt * Q, Q);  // rows of this tile: r = rt * Q + 0..rows-1
  if (rows <= 0) return;
  // the parts of this sequence: `per` tiles each
  const int tiles = (len + kTile - 1) / kTile;
  const int per = max((tiles + sp.per_unit - 1) / sp.per_unit, kMinTiles);
  const int parts = max((tiles + per - 1) / per, 1);
  if (part >= parts) return;
  const int tile_end = min((part + 1) * per, tiles);

  // ---- queries: row g of each 8-row tile, in the order of the key loads ----
  // row r is head r / nq, query r % nq
  uint32_t qf[NT][KV * 4][2];
  float qscale[NT][2];  // of rows 2 q4, 2 q4 + 1: scale log2(e) 2^e
  int limit[NT][2];     // last token that they see
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = rt * Q + nt * 8 + g;
    const bool there = nt * 8 + g < rows;
    uint4 w[KV][2];
    float mx = 0.f;
    const uint16_t* qp = a.q.at(l, b, h * a.G + (there ? r / nq : 0), there ? r % nq : 0);
#pragma unroll
    for (int k = 0; k < KV; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[k][i] = there ? __ldg(reinterpret_cast<const uint4*>(qp + (k * 4 + q4) * 16 + i * 8))
                        : make_uint4(0, 0, 0, 0);
        const uint32_t x[4] = {w[k][i].x, w[k][i].y, w[k][i].z, w[k][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(x[j])), fabsf(bf16_hi(x[j]))));
      }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // the row's largest magnitude to [1, 2)
    const int e = min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100), 100);
    const float down = exp2_int(-e);
#pragma unroll
    for (int k = 0; k < KV; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t x[4] = {w[k][i].x, w[k][i].y, w[k][i].z, w[k][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          qf[nt][k * 4 + i * 2 + j / 2][j % 2] = half2_of(bf16_lo(x[j]) * down, bf16_hi(x[j]) * down);
      }
    const float up = a.scale_log2 * exp2_int(e);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      qscale[nt][i] = __shfl_sync(0xffffffffu, up, (2 * q4 + i) * 4);
      const int rr = rt * Q + nt * 8 + 2 * q4 + i;
      limit[nt][i] = len - nq + rr % nq;
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

  const uint8_t* kp = c.pool[0] + block_row(c, l, 0, h) * D;
  const uint8_t* vp = c.pool[1] + block_row(c, l, 0, h) * D;
  const float* ksp = c.scale[0] + scale_at(c, l, 0, h);
  const float* vsp = c.scale[1] + scale_at(c, l, 0, h);
  const int32_t* table = c.table + static_cast<size_t>(b) * c.max_blocks;

  // Lane i (and i + 16) looks after token i of a tile: its block two tiles ahead,
  // its row and scales one tile ahead.
  const int tok = lane % 16;
  auto block_of = [&](int tile) {
    const int t = tile * kTile + tok;
    return tile < tile_end && t < len ? __ldg(table + by_bs.div(t)) : -1;
  };
  int row = -1;        // of the tile whose loads are in flight
  float ks = 0.f, vs = 1.f;
  auto resolve = [&](int tile, int blk) {
    const int t = tile * kTile + tok;
    row = -1;
    ks = 0.f;
    vs = 1.f;
    if (tile < tile_end && t < len) {
      if (blk < 0 || blk >= c.n_blocks) {
        bad = true;
      } else {
        const int in = t - by_bs.div(t) * by_bs.bs;
        row = blk * c.H * by_bs.bs + in;  // below 2^31: checked on the host
        ks = __ldg(ksp + static_cast<size_t>(blk) * c.H);
        vs = __ldg(vsp + static_cast<size_t>(blk) * c.H);
      }
    }
  };
  uint4 kr[2][KV];
  uint4 vr[4];
  auto load_keys = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = __shfl_sync(0xffffffffu, row, g + 8 * i);
#pragma unroll
      for (int k = 0; k < KV; ++k)
        kr[i][k] = r >= 0 ? load16(kp + static_cast<size_t>(r) * D + (k * 4 + q4) * 16)
                          : make_uint4(0, 0, 0, 0);
    }
  };
  auto load_values = [&]() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = __shfl_sync(0xffffffffu, row, 2 * q4 + (i & 1) + 8 * (i >> 1));
      if constexpr (D == 128) {
        vr[i] = r >= 0 ? load16(vp + static_cast<size_t>(r) * D + g * 16) : make_uint4(0, 0, 0, 0);
      } else {
        const uint2 v = r >= 0 ? load8(vp + static_cast<size_t>(r) * D + g * 8) : make_uint2(0, 0);
        vr[i] = make_uint4(v.x, v.y, 0, 0);
      }
    }
  };

  int tile = part * per + warp;
  int blk = block_of(tile);
  resolve(tile, blk);
  blk = block_of(tile + kWarps);
  load_keys();
  load_values();
  for (; tile < tile_end; tile += kWarps) {
    const int t0 = tile * kTile;
    // this tile's scales and which of its tokens are there, by lane
    const float ks_now = ks, vs_now = vs;
    const int row_now = row;
    resolve(tile + kWarps, blk);
    blk = block_of(tile + 2 * kWarps);

    // ---- S^T = K Q^T ----
    float z[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) z[nt][j] = 0.f;
#pragma unroll
    for (int k = 0; k < KV; ++k) {
      const uint32_t x[4] = {kr[0][k].x, kr[0][k].y, kr[0][k].z, kr[0][k].w};
      const uint32_t y[4] = {kr[1][k].x, kr[1][k].y, kr[1][k].z, kr[1][k].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t a0, a1, a2, a3;
        halves<FMT>(x[j], a0, a2);
        halves<FMT>(y[j], a1, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma(z[nt], a0, a1, a2, a3, qf[nt][k * 4 + j][0], qf[nt][k * 4 + j][1]);
      }
    }
    load_keys();

    // ---- weights ----
    const float ks0 = __shfl_sync(0xffffffffu, ks_now, g);
    const float ks1 = __shfl_sync(0xffffffffu, ks_now, g + 8);
    const int there0 = __shfl_sync(0xffffffffu, row_now, g);
    const int there1 = __shfl_sync(0xffffffffu, row_now, g + 8);
    const float vs0 = __shfl_sync(0xffffffffu, vs_now, g);
    const float vs1 = __shfl_sync(0xffffffffu, vs_now, g + 8);
    const float e0 = static_cast<float>(static_cast<int>(__float_as_uint(vs0) >> 23) - 127);
    const float e1 = static_cast<float>(static_cast<int>(__float_as_uint(vs1) >> 23) - 127);
    const bool whole = t0 + kTile <= len - nq + 1;  // every query sees the tile
    bool up = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x0 = fmaf(z[nt][i], ks0 * qscale[nt][i], e0);
        float x1 = fmaf(z[nt][2 + i], ks1 * qscale[nt][i], e1);
        if (there0 < 0 || (!whole && t0 + g > limit[nt][i])) x0 = -INFINITY;
        if (there1 < 0 || (!whole && t0 + g + 8 > limit[nt][i])) x1 = -INFINITY;
        z[nt][i] = x0;
        z[nt][2 + i] = x1;
        up = up || fmaxf(x0, x1) > m[nt][i] + kSlack;
      }
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = fmaxf(z[nt][i], z[nt][2 + i]);
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          x = fmaxf(x, m[nt][i]);
          const float f = x > m[nt][i] ? ex2(m[nt][i] - x) : 1.f;
          m[nt][i] = x;
          sum[nt][i] *= f;
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            o[nt][t][i] *= f;
            o[nt][t][2 + i] *= f;
          }
        }
    }
    const float back0 = exp2_int(-static_cast<int>(e0)), back1 = exp2_int(-static_cast<int>(e1));
    uint32_t p[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float w[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mm = m[nt][i] == -INFINITY ? 0.f : m[nt][i];
        w[i] = ex2(z[nt][i] - mm);
        w[2 + i] = ex2(z[nt][2 + i] - mm);
        sum[nt][i] += w[i] * back0 + w[2 + i] * back1;
      }
      p[nt][0] = transpose8x8(half2_of(w[0], w[1]));
      p[nt][1] = transpose8x8(half2_of(w[2], w[3]));
    }

    // ---- O^T += V^T P^T ----
#pragma unroll
    for (int j = 0; j < MT / 2; ++j) {
      const uint32_t x[4] = {j == 0 ? vr[0].x : j == 1 ? vr[0].y : j == 2 ? vr[0].z : vr[0].w,
                             j == 0 ? vr[1].x : j == 1 ? vr[1].y : j == 2 ? vr[1].z : vr[1].w,
                             j == 0 ? vr[2].x : j == 1 ? vr[2].y : j == 2 ? vr[2].z : vr[2].w,
                             j == 0 ? vr[3].x : j == 1 ? vr[3].y : j == 2 ? vr[3].z : vr[3].w};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t sel = i == 0 ? 0x5140 : 0x7362;
        uint32_t a0, a1, a2, a3;
        halves<FMT>(__byte_perm(x[0], x[1], sel), a0, a1);
        halves<FMT>(__byte_perm(x[2], x[3], sel), a2, a3);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma(o[nt][2 * j + i], a0, a1, a2, a3, p[nt][0], p[nt][1]);
      }
    }
    load_values();
  }

  // ---- join the warps ----
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
  if (bad) atomicOr(c.status, KVC_STATUS_BAD_INDEX);
  __syncthreads();

  // a thread has kPer neighbouring values of a row
  constexpr int kPer = 8;
  constexpr int TPR = D / kPer;  // threads of a row
  const size_t slot_floats = static_cast<size_t>(kRowTile) * (D + 2);
  float* mine = sp.part + static_cast<size_t>(blockIdx.x) * slot_floats;
  for (int i = threadIdx.x; i < Q * TPR; i += kThreads) {
    const int r = i / TPR, d0 = (i % TPR) * kPer;
    if (r >= rows) continue;
    float mm = s_m[0][r];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, s_m[w][r]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float x[kPer], s = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) x[k] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(s_m[w][r] - ref);
      s += f * s_l[w][r];
#pragma unroll
      for (int k = 0; k < kPer; ++k) x[k] += f * s_o[w][r][d0 + k];
    }
    if (parts > 1) {
      float* to = mine + r * (D + 2);
#pragma unroll
      for (int k = 0; k < kPer; ++k) to[2 + d0 + k] = x[k];
      if (d0 == 0) {
        to[0] = mm;
        to[1] = s;
      }
    } else {
      const int rr = rt * Q + r;
      const int hq = h * a.G + rr / nq, j = rr % nq;
      const float inv = s == 0.f ? 0.f : 1.f / s;
      *reinterpret_cast<uint4*>(a.out.at(l, b, hq, j) + d0) =
          make_uint4(bf16x2(x[0] * inv, x[1] * inv), bf16x2(x[2] * inv, x[3] * inv),
                     bf16x2(x[4] * inv, x[5] * inv), bf16x2(x[6] * inv, x[7] * inv));
      if (a.lse && d0 == 0)
        a.lse[((static_cast<size_t>(l) * c.B + b) * c.H * a.G + hq) * a.n + j] =
            (mm + __log2f(s)) * 0.6931471805599453f;
    }
  }
  if (parts == 1) return;

  // ---- join the parts: the last CTA to arrive, in the order of the parts ----
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) s_last = atomicAdd(&sp.arrived[ur], 1) == parts - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  if (threadIdx.x == 0) sp.arrived[ur] = 0;  // ready for the next call
  const float* first = sp.part + static_cast<size_t>(ur) * sp.per_unit * slot_floats;
  for (int i = threadIdx.x; i < Q * TPR; i += kThreads) {
    const int r = i / TPR, d0 = (i % TPR) * kPer;
    if (r >= rows) continue;
    const float* from = first + r * (D + 2);
    float mm = -INFINITY;
    for (int w = 0; w < parts; ++w) mm = fmaxf(mm, __ldcg(from + w * slot_floats));
    const float ref = mm == -INFINITY ? 0.f : mm;
    float x[kPer], s = 0.f;
#pragma unroll
    for (int k = 0; k < kPer; ++k) x[k] = 0.f;
    for (int w = 0; w < parts; ++w) {
      const float* pw = from + w * slot_floats;
      const float f = ex2(__ldcg(pw) - ref);
      s += f * __ldcg(pw + 1);
#pragma unroll
      for (int k = 0; k < kPer; k += 2) {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(pw + 2 + d0 + k));
        x[k] += f * v.x;
        x[k + 1] += f * v.y;
      }
    }
    const int rr = rt * Q + r;
    const int hq = h * a.G + rr / nq, j = rr % nq;
    const float inv = s == 0.f ? 0.f : 1.f / s;
    *reinterpret_cast<uint4*>(a.out.at(l, b, hq, j) + d0) =
        make_uint4(bf16x2(x[0] * inv, x[1] * inv), bf16x2(x[2] * inv, x[3] * inv),
                   bf16x2(x[4] * inv, x[5] * inv), bf16x2(x[6] * inv, x[7] * inv));
    if (a.lse && d0 == 0)
      a.lse[((static_cast<size_t>(l) * c.B + b) * c.H * a.G + hq) * a.n + j] =
          (mm + __log2f(s)) * 0.6931471805599453f;
  }
}

template <int D, int FMT>
cudaError_t launch_few(const Cache& c, const AttendArgs& a, cudaStream_t s) {
  const int R = a.G * a.n;
  const int nt = R > 8 ? 2 : 1;
  Split sp;
  sp.row_tiles = (R + 8 * nt - 1) / (8 * nt);
  const long long heads = static_cast<long long>(c.L) * c.B * c.H * sp.row_tiles;
  // split sequences while the heads leave CTAs' places free
  const long long places = static_cast<long long>(a.num_sms) * (nt == 1 ? 4 : 3);
  const int tiles = static_cast<int>((static_cast<long long>(c.max_blocks) * c.bs + kTile - 1) / kTile);
  long long per = heads < 2 * places ? 2 * places / heads : 1;
  per = per < (tiles + kMinTiles - 1) / kMinTiles ? per : (tiles + kMinTiles - 1) / kMinTiles;
  while (per > 1 && per * heads > kMaxParts) --per;
  sp.per_unit = static_cast<int>(per < 1 ? 1 : per);
  sp.arrived = static_cast<int*>(a.workspace);
  sp.part = reinterpret_cast<float*>(sp.arrived + kMaxParts);
  const int grid = static_cast<int>(heads * sp.per_unit);
  auto* kernel = nt == 1 ? attend_few_kernel<D, FMT, 1> : attend_few_kernel<D, FMT, 2>;
  kernel<<<grid, kThreads, 0, s>>>(c, a, sp, make_div(c.bs));
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend(const Cache& c, int format, const AttendArgs& a, cudaStream_t s) {
  if (c.d == 64)
    return format == KVC_CACHE8_E4M3 ? launch_few<64, KVC_CACHE8_E4M3>(c, a, s)
                                     : launch_few<64, KVC_CACHE8_INT8>(c, a, s);
  return format == KVC_CACHE8_E4M3 ? launch_few<128, KVC_CACHE8_E4M3>(c, a, s)
                                   : launch_few<128, KVC_CACHE8_INT8>(c, a, s);
}

}  // namespace cache8

size_t cache8_attend_workspace(int d) {
  return cache8::kMaxParts * (sizeof(int) + static_cast<size_t>(cache8::kRowTile) * (d + 2) * 4);
}

}  // namespace kvc
