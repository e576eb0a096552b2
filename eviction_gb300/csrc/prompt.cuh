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
// (cut items are fewer than two a SM, their parts fewer than four, of 256 tokens each)
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

}  // namespace prompt
}  // namespace kvc
