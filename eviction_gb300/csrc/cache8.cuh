// cache8.cuh -- the 8-bit paged cache: what its kernels share.  Codes and their
// conversions, the block scale, and the walk from a token to its row.
//
// A code c of a block with scale s stands for c * s.  Scales are powers of two:
// dividing by one is exact, so a value has one nearest code whatever computes it,
// and growing a block's scale is a shift of its codes.
#pragma once

#include "kvc_internal.cuh"

namespace kvc {
namespace cache8 {

constexpr int kScaleExpMin = -64, kScaleExpMax = 64;

// The cache as kernels take it (validated sizes).
struct Cache {
  uint8_t* pool[2];   // keys, values: [L][n_blocks][H][bs][d]
  float* scale[2];    // [L][n_blocks][H]
  int32_t* table;     // [B][max_blocks]
  int32_t* seq_len;   // [B]
  int32_t* free_list;
  int32_t* free_top;
  int32_t* ref_count;
  int L, B, H, d, n_blocks, bs, max_blocks;
  uint32_t* status;   // the handle's status bits
  uint32_t* err;      // the running call's error word
};

// Strided rows of bf16 values.
struct Rows {
  uint16_t* data;
  long long layer, seq, head, token;
  __host__ __device__ uint16_t* at(int l, int b, int h, int j) const {
    return data + l * layer + b * seq + h * head + j * token;
  }
};

struct CompactArgs {
  int T, budget;
  const int32_t* pad;
  const int32_t* kept;
  const int32_t* n_kept;
  const float* credit_post;
  float* credit_out;
};

cudaError_t launch_grow(const Cache& c, const int32_t* n_new, cudaStream_t s);
cudaError_t launch_free(const Cache& c, int n, const int32_t* seqs, cudaStream_t s);
cudaError_t launch_fork(const Cache& c, int n, const int32_t* src, const int32_t* dst,
                        int num_sms, cudaStream_t s);
cudaError_t launch_append(const Cache& c, int format, const Rows& k, const Rows& v, int n,
                          const int32_t* n_new, cudaStream_t s);
cudaError_t launch_gather(const Cache& c, int format, int T, uint16_t* k_out, uint16_t* v_out,
                          int32_t* pad, cudaStream_t s);
cudaError_t launch_compact(const Cache& src, int src_format, const Cache& dst, int dst_format,
                           const CompactArgs& a, cudaStream_t s);

struct AttendArgs {
  Rows q, out;
  float* lse;
  const int32_t* n_q;  // NULL: n for every sequence
  int n, G;
  float scale_log2;    // softmax scale * log2(e)
  int num_sms;
  void* workspace;
};
cudaError_t launch_attend(const Cache& c, int format, const AttendArgs& a, cudaStream_t s);

#if defined(__CUDACC__)

// Every kernel of the cache may be launched while the one before it on the stream still
// runs (a decode step is a chain of kernels of a few microseconds: their launch
// latencies overlap).  before_all() comes first in a kernel: nothing is read or written
// until that one has completed and its writes are visible; the next kernel's launch
// may begin then.  No kernel reads through the read-only path (__ldg, restrict): that is
// for data that does not change while a kernel runs, and the one before still writes.
__device__ __forceinline__ void before_all() {
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}

template <class... Params, class... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t s,
                   Args... args) {
  cudaLaunchAttribute overlap;
  overlap.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  overlap.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &overlap;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

__device__ __forceinline__ float exp2_int(int e) {  // 2^e, -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Exponent of the smallest power of two s with amax <= TOP * s (clamped): with
// amax = m 2^x, 1 <= m < 2, and TOP = t 2^y, that is x - y, one more if m > t.
template <int FMT>
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const uint32_t edge = FMT == KVC_CACHE8_E4M3 ? 0x600000u : 0x7E0000u;  // 448 = 1.75 2^8, 127 = 1.984375 2^6
  const int y = FMT == KVC_CACHE8_E4M3 ? 8 : 6;
  const int x = static_cast<int>(bits >> 23) - 127;  // 0 and subnormals: clamped below
  return min(max(x - y + ((bits & 0x7FFFFFu) > edge ? 1 : 0), kScaleExpMin), kScaleExpMax);
}

// The nearest codes of a (low byte) and b, which are in units of the scale.
// NaN becomes 0 (if NAN_TOO), what is too large the largest code.
template <int FMT, bool NAN_TOO = true>
__device__ __forceinline__ uint32_t encode2(float a, float b) {
  if constexpr (NAN_TOO) {
    a = a == a ? a : 0.f;
    b = b == b ? b : 0.f;
  }
  if constexpr (FMT == KVC_CACHE8_E4M3) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
  } else {
    const int x = min(max(__float2int_rn(a), -127), 127), y = min(max(__float2int_rn(b), -127), 127);
    return (x & 0xFF) | ((y & 0xFF) << 8);
  }
}

// Two fp16 values from the low 16 bits (two codes) of `two`.
__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(two));
  return r;
}

// Four fp32 values of four codes.
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t four, float (&x)[4]) {
  if constexpr (FMT == KVC_CACHE8_E4M3) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t two = e4m3_to_half2(four >> (16 * i));
      asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\t"
          "cvt.f32.f16 %1, hi;\n\t}"
          : "=f"(x[2 * i]), "=f"(x[2 * i + 1])
          : "r"(two));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(static_cast<int8_t>(four >> (8 * i)));
  }
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

__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t clamp_half2(uint32_t a, uint32_t lo, uint32_t hi) {
  uint32_t r;
  asm("{\n\t.reg .b32 t;\n\tmax.f16x2 t, %1, %2;\n\tmin.f16x2 %0, t, %3;\n\t}"
      : "=r"(r)
      : "r"(a), "r"(lo), "r"(hi));
  return r;
}

// 2^e as both halves of a pair of fp16, e <= 15; 0 below its last step.
__device__ __forceinline__ uint32_t exp2_half2(int e) {
  const uint32_t h = e >= -14 ? (15 + e) << 10 : e >= -24 ? 1u << (24 + e) : 0u;
  return h * 0x00010001u;
}

// Pairs (0, 1) and (2, 3) of fp16 values, at most the largest code (integers; e4m3
// saturates by itself), to four codes.
template <int FMT>
__device__ __forceinline__ uint32_t codes_of(uint32_t lo, uint32_t hi) {
  if constexpr (FMT == KVC_CACHE8_E4M3) {
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tcvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n\tmov.b32 %0, {a, b};\n\t}"
        : "=r"(r)
        : "r"(lo), "r"(hi));
    return r;
  } else {
    // plus 1.5 2^10: steps of 1 there, so that the sum rounds to the nearest integer
    // (ties to even), whose low byte it ends in
    uint32_t a, b;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(a) : "r"(lo), "r"(0x66006600u));
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(b) : "r"(hi), "r"(0x66006600u));
    return __byte_perm(a, b, 0x6420);
  }
}

// The block that holds entry i of sequence b, or -1 if it is out of range.
__device__ __forceinline__ int block_at(const Cache& c, int b, int i) {
  if (i < 0 || i >= c.max_blocks) return -1;
  const int blk = c.table[static_cast<size_t>(b) * c.max_blocks + i];
  return blk >= 0 && blk < c.n_blocks ? blk : -1;
}

// First row of a block's head, in rows of d codes; times d: its offset in a pool.
__device__ __forceinline__ size_t block_row(const Cache& c, int l, int blk, int h) {
  return ((static_cast<size_t>(l) * c.n_blocks + blk) * c.H + h) * c.bs;
}
__device__ __forceinline__ size_t scale_at(const Cache& c, int l, int blk, int h) {
  return (static_cast<size_t>(l) * c.n_blocks + blk) * c.H + h;
}

// The tokens that sequence b holds, 0 where its length is out of range.
__device__ __forceinline__ int length_of(const Cache& c, int b, bool* bad) {
  const int len = c.seq_len[b];
  if (len < 0 || len > c.max_blocks * c.bs) {
    *bad = true;
    return 0;
  }
  return len;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float bf16_lo(uint32_t two) { return __uint_as_float(two << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t two) { return __uint_as_float(two & 0xffff0000u); }

// Two bf16 (nearest even), a in the low half.
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

#endif  // __CUDACC__

}  // namespace cache8
}  // namespace kvc
