// prompt_api.cu -- host side of rotary positions, prompt attention and the choice of the
// heaviest tokens: argument checks and the entry points.
#include <cfloat>
#include <climits>
#include <cmath>

#include "api_util.cuh"
#include "prompt.cuh"

using kvc::aligned4;
using kvc::check_device;
using kvc::check_rows;
using kvc::fail;
using kvc::guarded;
using kvc::run;

namespace {

kvc::cache8::Rows rows(const kvc_rows& r) {
  return {r.data, r.layer, r.seq, r.head, r.token};
}

bool same_rows(const kvc_rows& a, const kvc_rows& b) {
  return a.data == b.data && a.layer == b.layer && a.seq == b.seq && a.head == b.head &&
         a.token == b.token;
}

int check_counts(kvc_handle* h, const int32_t* n_tok) {
  return n_tok && !aligned4(n_tok) ? fail(h, KVC_ERR_ALIGN, "not 4-byte aligned: n_tok") : KVC_OK;
}

}  // namespace

extern "C" {

int kvc_rope_init(const kvc_rope_config* c, kvc_rope* r) {
  if (!c || !r) return KVC_ERR_ARG;
  auto positive = [](double x) { return std::isfinite(x) && x > 0; };
  if (c->dim < 16 || c->dim > 128 || c->dim % 16 || (c->interleaved & ~1) || !std::isfinite(c->base) ||
      c->base < 1 || !positive(c->factor) || !positive(c->magnitude) ||
      c->scaling < KVC_ROPE_NONE || c->scaling > KVC_ROPE_BANDS)
    return KVC_ERR_ARG;
  if (c->scaling == KVC_ROPE_BANDS &&
      (!(c->low >= 0) || !std::isfinite(c->high) || c->high <= c->low || !positive(c->original)))
    return KVC_ERR_ARG;
  // (what a float holds as a normal number)
  if (!(c->magnitude >= FLT_MIN && c->magnitude <= FLT_MAX)) return KVC_ERR_ARG;
  constexpr double kTurn = 6.283185307179586476925;
  constexpr double kFastest = 4294967296.0;  // turns a token: 20 bits of a turn are left in a double
  double base = c->base;
  if (c->scaling == KVC_ROPE_NTK) base *= std::pow(c->factor, c->dim / (c->dim - 2.0));
  if (!positive(base)) return KVC_ERR_ARG;
  kvc_rope made = {};
  made.dim = c->dim;
  made.interleaved = c->interleaved;
  made.magnitude = static_cast<float>(c->magnitude);
  for (int i = 0; i < 64; ++i) {
    double turns = 0;  // per token
    if (i < c->dim / 2) turns = std::pow(base, -2.0 * i / c->dim) / kTurn;
    if (c->scaling == KVC_ROPE_LINEAR) turns /= c->factor;
    if (c->scaling == KVC_ROPE_BANDS) {
      const double m = std::fmin(std::fmax((c->original * turns - c->low) / (c->high - c->low), 0.0), 1.0);
      turns = (1 - m) * turns / c->factor + m * turns;
    }
    if (!(turns >= 0 && turns < kFastest)) return KVC_ERR_ARG;
    turns -= std::floor(turns);
    made.turn[i] = static_cast<uint64_t>(std::ldexp(turns, 64));
  }
  *r = made;
  return KVC_OK;
}

int kvc_rotary(kvc_handle* h, const kvc_rope* rope, const kvc_rows* q, const kvc_rows* k,
               const kvc_rows* q_out, const kvc_rows* k_out, int n_layers, int n_seq, int n,
               const int32_t* pos, const int32_t* n_tok, void* stream) {
  if (!h) return KVC_ERR_ARG;
  return guarded([&] {
    if (!rope) return fail(h, KVC_ERR_ARG, "null pointer: rope");
    if (rope->dim < 16 || rope->dim > 128 || rope->dim % 16)
      return fail(h, KVC_ERR_ARG, "the rope is not one of kvc_rope_init");
    if (rope->dim > h->dims.d) return fail(h, KVC_ERR_SHAPE, "the rope's dim is larger than head_dim");
    if (n_layers < 1 || n_seq < 1 || n < 1)
      return fail(h, KVC_ERR_SHAPE, "n_layers, n_seq and n must be >= 1");
    if (n_layers > 65535 || static_cast<long long>(n_seq) * n > (1 << 30))
      return fail(h, KVC_ERR_UNSUPPORTED, "n_layers must be < 2^16, n_seq * n <= 2^30");
    if (!q != !q_out || !k != !k_out || (!q && !k))
      return fail(h, KVC_ERR_ARG, "q and q_out go together, k and k_out too, and one of the pairs has to be there");
    KVC_TRY(check_device(h));
    kvc::prompt::RotaryArgs a = {};
    const kvc_rows* in[2] = {q, k};
    const kvc_rows* out[2] = {q_out, k_out};
    const char* const names[2][2] = {{"q", "k"}, {"q_out", "k_out"}};
    for (int w = 0; w < 2; ++w) {
      if (!in[w]) continue;
      const int heads = w ? h->dims.H : h->dims.H * h->dims.G;
      KVC_TRY(check_rows(h, in[w], names[0][w], false, n_layers, n_seq, heads, n));
      KVC_TRY(check_rows(h, out[w], names[1][w], true, n_layers, n_seq, heads, n));
      a.heads[w] = heads;
      a.in[w] = rows(*in[w]);
      a.out[w] = rows(*out[w]);
      a.in_place[w] = same_rows(*in[w], *out[w]);
    }
    KVC_REQUIRE_INTS(pos);
    KVC_TRY(check_counts(h, n_tok));
    a.rope = *rope;
    a.L = n_layers, a.S = n_seq, a.n = n, a.d = h->dims.d;
    a.pos = pos, a.n_tok = n_tok;
    a.num_sms = h->num_sms, a.status = h->ws.status;
    return run(h, kvc::kKernelRotary, "rotary", stream,
               [&](cudaStream_t s) { return kvc::prompt::launch_rotary(a, s); });
  });
}

int kvc_prompt_attend(kvc_handle* h, const kvc_rows* q, const kvc_rows* k, const kvc_rows* v,
                      int n_seq, int n, const int32_t* first, const int32_t* n_tok,
                      const kvc_rows* out, float* lse, void* stream) {
  if (!h) return KVC_ERR_ARG;
  return guarded([&] {
    if (n_seq < 1 || n < 1) return fail(h, KVC_ERR_SHAPE, "n_seq and n must be >= 1");
    const int H = h->dims.H, Hq = H * h->dims.G, S = first ? 1 : n_seq;
    // (the kernel counts pairs of tiles of 8 tokens at least, and one more a sequence)
    const long long tokens = static_cast<long long>(S) * n;
    if (n_seq > 1 << 20 || tokens >= 1 << 30 || Hq > 65535 || (tokens / 16 + n_seq) * Hq > INT_MAX)
      return fail(h, KVC_ERR_UNSUPPORTED, "n_seq must be <= 2^20, the tokens < 2^30, n_kv_heads * group < "
                                          "2^16 and (tokens / 16 + n_seq) * n_kv_heads * group < 2^31");
    if (first && !n_tok) return fail(h, KVC_ERR_ARG, "packed sequences need n_tok");
    KVC_TRY(check_device(h));
    const struct {
      const kvc_rows* r;
      const char* name;
      int heads;
    } all[4] = {{q, "q", Hq}, {k, "k", H}, {v, "v", H}, {out, "out", Hq}};
    for (const auto& x : all) {
      KVC_TRY(check_rows(h, x.r, x.name, x.r == out, 1, S, x.heads, n));
      const int64_t most = int64_t{1} << 39;
      if (x.r->seq >= most || x.r->head >= most || x.r->token >= most)
        return fail(h, KVC_ERR_UNSUPPORTED, std::string("strides must be < 2^39: ") + x.name);
      if ((n > 1 && x.r->token == 0) || (x.r == q && Hq > 1 && q->head == 0))
        return fail(h, KVC_ERR_UNSUPPORTED, std::string("rows of tokens (of q: also of heads) must not "
                                                        "be the same: ") + x.name);
    }
    if (first && !aligned4(first)) return fail(h, KVC_ERR_ALIGN, "not 4-byte aligned: first");
    KVC_TRY(check_counts(h, n_tok));
    if (lse && !aligned4(lse)) return fail(h, KVC_ERR_ALIGN, "not 4-byte aligned: lse");
    kvc::prompt::AttendArgs a{rows(*q), rows(*k), rows(*v), rows(*out), lse, n_seq, n, H, h->dims.G,
                              h->dims.d, first, n_tok, kvc::scale_log2_of(h->cfg), h->num_sms,
                              h->ws.status};
    return run(h, kvc::kKernelPromptAttend, "prompt attend", stream,
               [&](cudaStream_t s) { return kvc::prompt::launch_attend(a, s); });
  });
}

int kvc_keep_heaviest(kvc_handle* h, const float* weights, int n_layers, int cap,
                      const int32_t* seq_len, int32_t* kept_idx, int32_t* n_kept,
                      float* weights_out, void* stream) {
  if (!h) return KVC_ERR_ARG;
  return guarded([&] {
    if (n_layers < 1) return fail(h, KVC_ERR_SHAPE, "n_layers must be >= 1");
    if (cap < 1 || cap > h->cfg.max_T) return fail(h, KVC_ERR_SHAPE, "cap must lie in [1, max_T]");
    if (static_cast<long long>(n_layers) * h->dims.B * h->dims.H > INT_MAX)
      return fail(h, KVC_ERR_UNSUPPORTED, "n_layers * batch * n_kv_heads must be < 2^31");
    KVC_TRY(check_device(h));
    KVC_REQUIRE_INTS(weights);
    KVC_REQUIRE_INTS(seq_len);
    KVC_REQUIRE_INTS(kept_idx);
    KVC_REQUIRE_INTS(n_kept);
    KVC_REQUIRE_INTS(weights_out);
    kvc::prompt::HeaviestArgs a{weights, seq_len, kept_idx, n_kept, weights_out, n_layers, h->dims.B,
                                h->dims.H, cap, h->cfg.budget, h->cfg.n_sink, h->cfg.n_recent,
                                h->ws.status};
    return run(h, kvc::kKernelKeepHeaviest, "keep heaviest", stream,
               [&](cudaStream_t s) { return kvc::prompt::launch_heaviest(a, s); });
  });
}

}  // extern "C"
