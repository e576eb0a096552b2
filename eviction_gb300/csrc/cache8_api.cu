// cache8_api.cu -- host side of the 8-bit paged cache: argument checks and the
// entry points.
#include <algorithm>
#include <climits>

#include "api_util.cuh"
#include "cache8.cuh"
#include "prompt.cuh"

using kvc::aligned16;
using kvc::aligned4;
using kvc::check_device;
using kvc::check_rows;
using kvc::fail;
using kvc::guarded;
using kvc::run;

namespace {

int check_cache(const kvc_config& cfg, const kvc_cache8* c, const char** why) {
  auto bad = [&](int code, const char* m) {
    *why = m;
    return code;
  };
  if (!c) return bad(KVC_ERR_ARG, "the cache is null");
  if (!c->k_pool || !c->v_pool || !c->k_scale || !c->v_scale || !c->table || !c->seq_len ||
      !c->free_list || !c->free_top || !c->ref_count)
    return bad(KVC_ERR_ARG, "null pointer in the cache");
  if (!aligned16(c->k_pool) || !aligned16(c->v_pool))
    return bad(KVC_ERR_ALIGN, "pools must be 16-byte aligned");
  if (!aligned4(c->k_scale) || !aligned4(c->v_scale) || !aligned4(c->table) ||
      !aligned4(c->seq_len) || !aligned4(c->free_list) || !aligned4(c->free_top) ||
      !aligned4(c->ref_count))
    return bad(KVC_ERR_ALIGN, "scales, tables and counts must be 4-byte aligned");
  if (c->format != KVC_CACHE8_E4M3 && c->format != KVC_CACHE8_INT8)
    return bad(KVC_ERR_ARG, "format must be KVC_CACHE8_E4M3 or KVC_CACHE8_INT8");
  if (c->n_layers < 1 || c->n_blocks < 1 || c->max_blocks < 1)
    return bad(KVC_ERR_ARG, "n_layers, n_blocks and max_blocks must be >= 1");
  if (c->block_size < 1 || c->block_size > 1024)
    return bad(KVC_ERR_ARG, "block_size must lie in [1, 1024]");
  const long long B = cfg.batch, H = cfg.n_kv_heads, N = c->n_blocks, M = c->max_blocks;
  if (N > INT_MAX / H || N * H > INT_MAX / c->block_size)
    return bad(KVC_ERR_UNSUPPORTED, "n_blocks * n_kv_heads * block_size must be < 2^31");
  if (B * M > INT_MAX || M * c->block_size > (1 << 30))
    return bad(KVC_ERR_UNSUPPORTED,
               "batch * max_blocks must be < 2^31, max_blocks * block_size <= 2^30");
  if (B * H * c->n_layers > INT_MAX / 2)
    return bad(KVC_ERR_UNSUPPORTED, "n_layers * batch * n_kv_heads must be < 2^30");
  return KVC_OK;
}

int check(kvc_handle* h, const kvc_cache8* c) {
  const char* why = "";
  const int rc = check_cache(h->cfg, c, &why);
  return rc ? fail(h, rc, why) : check_device(h);
}

kvc::cache8::Cache view(const kvc_handle* h, const kvc_cache8& c) {
  return {{c.k_pool, c.v_pool}, {c.k_scale, c.v_scale}, c.table, c.seq_len, c.free_list,
          c.free_top, c.ref_count, c.n_layers, h->dims.B, h->dims.H, h->dims.d, c.n_blocks,
          c.block_size, c.max_blocks, h->ws.status, h->ws.status + 1};
}

kvc::cache8::Rows rows(const kvc_rows& r) {
  return {r.data, r.layer, r.seq, r.head, r.token};
}

// Both forms of append: `seqs` sequences of n rows each, or all among n rows, from row0[b] on.
int append(kvc_handle* h, const kvc_cache8* c, const kvc_rows* k, const kvc_rows* v, int n, int seqs,
           const int32_t* row0, const int32_t* n_new, void* stream) {
  KVC_TRY(check(h, c));
  if (n < 1) return fail(h, KVC_ERR_SHAPE, "n must be >= 1");
  KVC_TRY(check_rows(h, k, "k", false, c->n_layers, seqs, h->dims.H, n));
  KVC_TRY(check_rows(h, v, "v", false, c->n_layers, seqs, h->dims.H, n));
  KVC_REQUIRE_INTS(n_new);
  const long long units = static_cast<long long>(c->n_layers) * h->dims.B * h->dims.H;
  const long long most = std::min<long long>(n, static_cast<long long>(c->max_blocks) * c->block_size);
  if (units > INT_MAX / ((most + c->block_size - 2) / c->block_size + 1))
    return fail(h, KVC_ERR_UNSUPPORTED, "too many blocks to write in one call");
  kvc::cache8::Rows kr = rows(*k), vr = rows(*v);
  if (row0) kr.seq = vr.seq = 0;
  return run(h, kvc::kKernelCache8Append, "cache8 append", stream, [&](cudaStream_t s) {
    return kvc::cache8::launch_append(view(h, *c), c->format, kr, vr, n, row0, n_new, s);
  });
}

}  // namespace

extern "C" {

int kvc_cache8_check(const kvc_config* cfg, const kvc_cache8* c, const char** why) {
  return guarded([&] {
    const char* none = "";
    if (!why) why = &none;
    *why = "";
    std::string bad;
    const int rc = kvc::validate_config(cfg, &bad);
    if (rc) {
      *why = "the configuration is not valid";
      return rc;
    }
    return check_cache(*cfg, c, why);
  });
}

int kvc_cache8_grow(kvc_handle* h, const kvc_cache8* c, const int32_t* n_new, void* stream) {
  if (!h) return KVC_ERR_ARG;
  return guarded([&] {
    KVC_TRY(check(h, c));
    KVC_REQUIRE_INTS(n_new);
    return run(h, kvc::kKernelCache8Grow, "cache8 grow", stream, [&](cudaStream_t s) {
      return kvc::cache8::launch_grow(view(h, *c), n_new, s);
    });
  });
}

int kvc_cache8_append(kvc_handle* h, const kvc_cache8* c, const kvc_rows* k, const kvc_rows* v,
                      int n, const int32_t* n_new, void* stream) {
  if (!h) return KVC_ERR_ARG;
  return guarded([&] { return append(h, c, k, v, n, h->dims.B, nullptr, n_new, stream); });
}

int kvc_cache8_append_packed(kvc_handle* h, const kvc_cache8* c, const kvc_rows* k, const kvc_rows* v,
                             int n, const int32_t* first, const int32_t* n_new, void* stream) {
  if (!h) return KVC_ERR_ARG;
  return guarded([&] {
    KVC_REQUIRE_INTS(first);
    return append(h, c, k, v, n, 1, first, n_new, stream);
  });
}

int kvc_cache8_attend(kvc_handle* h, const kvc_cache8* c, const kvc_rows* q, int n,
                      const int32_t* n_q, const kvc_rows* out, float* lse, void* stream) {
  if (!h) return KVC_ERR_ARG;
  return guarded([&] {
    KVC_TRY(check(h, c));
    if (n < 1 || n > h->cfg.window)
      return fail(h, KVC_ERR_SHAPE, "n must lie in [1, window]");
    const int Hq = h->dims.H * h->dims.G;
    KVC_TRY(check_rows(h, q, "q", false, c->n_layers, h->dims.B, Hq, n));
    KVC_TRY(check_rows(h, out, "out", true, c->n_layers, h->dims.B, Hq, n));
    if (n_q && !aligned4(n_q)) return fail(h, KVC_ERR_ALIGN, "not 4-byte aligned: n_q");
    if (lse && !aligned4(lse)) return fail(h, KVC_ERR_ALIGN, "not 4-byte aligned: lse");
    const long long rows_all = static_cast<long long>(c->n_layers) * h->dims.B * Hq * n;
    if (rows_all > INT_MAX)
      return fail(h, KVC_ERR_UNSUPPORTED, "n_layers * batch * query heads * n must be < 2^31");
    // (the kernels count 8 query rows by steps of 32 tokens, and a few more a head)
    if (static_cast<long long>(c->n_layers) * h->dims.B * h->dims.H *
            ((static_cast<long long>(h->dims.G) * n + 7) / 8) *
            ((static_cast<long long>(c->max_blocks) * c->block_size + 31) / 32 + 8) >
        INT_MAX / 2)
      return fail(h, KVC_ERR_UNSUPPORTED, "n_layers * batch * n_kv_heads * ceil(G n / 8) * "
                                          "(max_blocks * block_size / 32 + 8) must be < 2^30");
    kvc::cache8::AttendArgs a{rows(*q), rows(*out), lse, n_q, n, h->dims.G,
                              kvc::scale_log2_of(h->cfg), h->num_sms, h->ws.attend};
    return run(h, kvc::kKernelCache8Attend, "cache8 attend", stream, [&](cudaStream_t s) {
      return kvc::cache8::launch_attend(view(h, *c), c->format, a, s);
    });
  });
}

int kvc_cache8_weigh(kvc_handle* h, const kvc_cache8* c, const kvc_rows* q, int n,
                     const int32_t* first, const int32_t* n_q, const float* lse, float decay,
                     float* weights, int cap, void* stream) {
  if (!h) return KVC_ERR_ARG;
  return guarded([&] {
    KVC_TRY(check(h, c));
    if (n < 1 || n >= 1 << 30) return fail(h, KVC_ERR_SHAPE, "n must lie in [1, 2^30)");
    if (cap < 1 || cap >= 1 << 30) return fail(h, KVC_ERR_SHAPE, "cap must lie in [1, 2^30)");
    if (!(decay >= 0.f && decay <= 1.f)) return fail(h, KVC_ERR_ARG, "decay must lie in [0, 1]");
    if (first && !n_q) return fail(h, KVC_ERR_ARG, "packed queries need n_q");
    const int Hq = h->dims.H * h->dims.G;
    KVC_TRY(check_rows(h, q, "q", false, c->n_layers, first ? 1 : h->dims.B, Hq, n));
    if ((n > 1 && q->token == 0) || (Hq > 1 && q->head == 0))
      return fail(h, KVC_ERR_UNSUPPORTED, "rows of tokens and heads must not be the same: q");
    const int64_t most = int64_t{1} << 39;
    if (q->layer >= most || q->seq >= most || q->head >= most || q->token >= most)
      return fail(h, KVC_ERR_UNSUPPORTED, "strides must be < 2^39: q");
    if (first && !aligned4(first)) return fail(h, KVC_ERR_ALIGN, "not 4-byte aligned: first");
    if (n_q && !aligned4(n_q)) return fail(h, KVC_ERR_ALIGN, "not 4-byte aligned: n_q");
    KVC_REQUIRE_INTS(lse);
    KVC_REQUIRE_INTS(weights);
    const long long units = static_cast<long long>(c->n_layers) * h->dims.B * h->dims.H;
    if (units > INT_MAX / (cap / 32 + 8ll))
      return fail(h, KVC_ERR_UNSUPPORTED, "n_layers * batch * n_kv_heads * (cap / 32 + 8) must be < 2^31");
    kvc::prompt::WeighArgs a{rows(*q), first, n_q, lse, weights, n, h->dims.G, cap,
                             kvc::scale_log2_of(h->cfg), decay, h->num_sms,
                             h->ws.weigh};
    return run(h, kvc::kKernelCache8Weigh, "cache8 weigh", stream, [&](cudaStream_t s) {
      return kvc::prompt::launch_weigh(view(h, *c), c->format, a, s);
    });
  });
}

int kvc_cache8_gather(kvc_handle* h, const kvc_cache8* c, int T, uint16_t* k_out,
                      uint16_t* v_out, int32_t* pad, void* stream) {
  if (!h) return KVC_ERR_ARG;
  return guarded([&] {
    KVC_TRY(check(h, c));
    if (T < 1 || T > h->cfg.max_T) return fail(h, KVC_ERR_SHAPE, "T must lie in [1, max_T]");
    KVC_REQUIRE_PTR(k_out);
    if (v_out && !aligned16(v_out)) return fail(h, KVC_ERR_ALIGN, "not 16-byte aligned: v_out");
    KVC_REQUIRE_INTS(pad);
    if (static_cast<long long>(c->n_layers) * h->dims.B * h->dims.H * T > INT_MAX)
      return fail(h, KVC_ERR_UNSUPPORTED, "n_layers * batch * n_kv_heads * T must be < 2^31");
    return run(h, kvc::kKernelCache8Gather, "cache8 gather", stream, [&](cudaStream_t s) {
      return kvc::cache8::launch_gather(view(h, *c), c->format, T, k_out, v_out, pad, s);
    });
  });
}

int kvc_cache8_compact(kvc_handle* h, const kvc_cache8* src, const kvc_cache8* dst, int T,
                       const int32_t* pad, const int32_t* kept_idx, const int32_t* n_kept,
                       const float* credit_post, float* credit_out, void* stream) {
  if (!h) return KVC_ERR_ARG;
  return guarded([&] {
    KVC_TRY(check(h, src));
    KVC_TRY(check(h, dst));
    if (T < 1 || T > h->cfg.max_T) return fail(h, KVC_ERR_SHAPE, "T must lie in [1, max_T]");
    if (src->n_layers != dst->n_layers)
      return fail(h, KVC_ERR_ARG, "both caches must have the same layers");
    if (src->table == dst->table || src->seq_len == dst->seq_len)
      return fail(h, KVC_ERR_ARG, "dst must have a table and lengths of its own");
    KVC_REQUIRE_INTS(pad);
    KVC_REQUIRE_INTS(kept_idx);
    KVC_REQUIRE_INTS(n_kept);
    if (!credit_post != !credit_out)
      return fail(h, KVC_ERR_ARG, "credit_post and credit_out go together");
    if (credit_post && (!aligned4(credit_post) || !aligned4(credit_out)))
      return fail(h, KVC_ERR_ALIGN, "not 4-byte aligned: credit");
    const long long units = static_cast<long long>(src->n_layers) * h->dims.B * h->dims.H;
    const int per_unit = (h->cfg.budget - 1) / dst->block_size + 1;
    if (units > INT_MAX / per_unit)
      return fail(h, KVC_ERR_UNSUPPORTED, "too many blocks to write in one call");
    kvc::cache8::CompactArgs a{T, h->cfg.budget, pad, kept_idx, n_kept, credit_post, credit_out};
    return run(h, kvc::kKernelCache8Compact, "cache8 compact", stream, [&](cudaStream_t s) {
      return kvc::cache8::launch_compact(view(h, *src), src->format, view(h, *dst), dst->format, a,
                                         s);
    });
  });
}

int kvc_cache8_fork(kvc_handle* h, const kvc_cache8* c, int n, const int32_t* src,
                    const int32_t* dst, void* stream) {
  if (!h) return KVC_ERR_ARG;
  return guarded([&] {
    KVC_TRY(check(h, c));
    if (n < 0) return fail(h, KVC_ERR_ARG, "n must be >= 0");
    if (n == 0) return KVC_OK;
    KVC_REQUIRE_INTS(src);
    KVC_REQUIRE_INTS(dst);
    return run(h, kvc::kKernelCache8Fork, "cache8 fork", stream, [&](cudaStream_t s) {
      return kvc::cache8::launch_fork(view(h, *c), n, src, dst, h->num_sms, s);
    });
  });
}

int kvc_cache8_free(kvc_handle* h, const kvc_cache8* c, int n, const int32_t* seqs, void* stream) {
  if (!h) return KVC_ERR_ARG;
  return guarded([&] {
    KVC_TRY(check(h, c));
    if (n < 0) return fail(h, KVC_ERR_ARG, "n must be >= 0");
    if (n == 0) return KVC_OK;
    KVC_REQUIRE_INTS(seqs);
    return run(h, kvc::kKernelCache8Free, "cache8 free", stream, [&](cudaStream_t s) {
      return kvc::cache8::launch_free(view(h, *c), n, seqs, s);
    });
  });
}

}  // extern "C"
