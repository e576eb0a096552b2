// prompt.cuh -- a prompt's way into a cache and eviction by gathered weight: what the
// entry points hand to the kernels (rotary.cu, prompt_attend.cu, weigh.cu, heaviest.cu).
#pragma once

#include "cache8.cuh"

namespace kvc {
namespace prompt {

using cache8::Rows;

struct RotaryArgs {
  kvc_rope rope;
  Rows in[2], out[2];  // queries, keys
  int heads[2];        // 0: none
  bool in_place[2];
  int L, S, n, d;
  const int32_t* pos;
  const int32_t* n_tok;
  int num_sms;
  uint32_t* status;
};
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t s);

struct AttendArgs {
  Rows q, k, v, out;
  float* lse;
  int S, n, H, G, d;
  const int32_t* first;
  const int32_t* n_tok;
  float scale_log2;
  int num_sms;
  uint32_t* status;
};
cudaError_t launch_attend(const AttendArgs& a, cudaStream_t s);

struct WeighArgs {
  Rows q;
  const int32_t* first;
  const int32_t* n_q;
  const float* lse;
  float* w;
  int n, G, cap;
  float scale_log2, decay;
  int num_sms;
  void* workspace;  // weigh_workspace() bytes
};
// (what is cut is fewer than 1.5 pairs of tiles an SM, in fewer than 3.5 parts, of 256 tokens each)
constexpr size_t weigh_workspace(int num_sms) { return static_cast<size_t>(num_sms) * 4 * 256 * sizeof(float); }
cudaError_t launch_weigh(const cache8::Cache& c, int format, const WeighArgs& a, cudaStream_t s);

struct HeaviestArgs {
  const float* w;
  const int32_t* seq_len;
  int32_t* kept;
  int32_t* n_kept;
  float* out;
  int L, B, H, cap, budget, n_sink, n_recent;
  uint32_t* status;
};
cudaError_t launch_heaviest(const HeaviestArgs& a, cudaStream_t s);

#if defined(__CUDACC__)

// Products issued by the lanes for which `issue` holds, one of a converged warp: without a
// branch around them their operands stay in uniform registers.  (A branch on the lane,
// with 64-bit descriptors made for each product, took 110 cycles a product to issue;
// 128 x 128 x 16 take 64 to compute.)  Descriptors: the low word, the high one is the same for all.
constexpr uint32_t kDescHigh = 1024 >> 4 | 1u << 14 | 2u << 29;  // as in sw128_desc
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t block) {
  return (addr & 0x3FFFFu) >> 4 | (block >> 4) << 16;
}
__device__ __forceinline__ void mma_ss_if(bool issue, uint32_t d_tmem, uint32_t a_low, uint32_t b_low,
                                          uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_low), "r"(b_low), "r"(idesc), "r"(static_cast<int>(accumulate)),
      "r"(static_cast<int>(issue)), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(bool issue, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low,
                                          uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 b, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_low), "r"(idesc), "r"(static_cast<int>(accumulate)),
      "r"(static_cast<int>(issue)), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void commit_if(bool issue, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(static_cast<int>(issue))
      : "memory");
}

#endif  // __CUDACC__

}  // namespace prompt
}  // namespace kvc
