// cache8_api.cu -- host side of the 8-bit paged cache: argument checks and the
// entry points.
#include <algorithm>
#include <climits>

#include "api_util.cuh"
#include "cache8.cuh"

using kvc::aligned16;
using kvc::cuda_fail;
using kvc::fail;
using kvc::mark_begin;
using kvc::mark_end;

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

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

// Strides are multiples of 8 values and not negative.  An output's rows may not share
// memory: each axis has to step over all that the axes of smaller strides span (true of
// any slice or permutation of a dense array).  Strides of axes of size 1 do not matter.
int check_rows(kvc_handle* h, const kvc_rows* r, const char* name, bool written, int L, int B,
               int heads, int n) {
  if (!r || !r->data) return fail(h, KVC_ERR_ARG, std::string("null pointer: ") + name);
  if (!aligned16(r->data)) return fail(h, KVC_ERR_ALIGN, std::string("not 16-byte aligned: ") + name);
  const int64_t stride[4] = {r->layer, r->seq, r->head, r->token};
  const int size[4] = {L, B, heads, n};
  for (int i = 0; i < 4; ++i) {
    if (size[i] > 1 && (stride[i] < 0 || stride[i] % 8))
      return fail(h, KVC_ERR_ALIGN, std::string("strides must be multiples of 8 and >= 0: ") + name);
    if (!written || size[i] == 1) continue;
    __int128 span = h->dims.d;  // values from the first to past the last of the axes below
    for (int k = 0; k < 4; ++k)
      if (size[k] > 1 && (stride[k] < stride[i] || (stride[k] == stride[i] && k < i)))
        span += static_cast<__int128>(stride[k]) * (size[k] - 1);
    if (stride[i] < span) return fail(h, KVC_ERR_ARG, std::string("rows overlap: ") + name);
  }
  return KVC_OK;
}

// The handle's device has to be the current one.
int check_device(kvc_handle* h) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(h, e, "current device");
  if (dev != h->device)
    return fail(h, KVC_ERR_DEVICE, "the handle belongs to another device than the current one");
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

// What an entry point does after its checks: the launch between two tracing marks.
// Nothing thrown (an allocation of the error text or of a mark) leaves the C ABI.
template <class F>
int run(kvc_handle* h, int kernel, const char* name, void* stream, F launch) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaEvent_t b = mark_begin(h, s);
  cudaError_t e = launch(s);
  if (e != cudaSuccess) return cuda_fail(h, e, name);
  mark_end(h, kernel, b, s);
  return KVC_OK;
}
template <class F>
int guarded(F f) {
  try {
    return f();
  } catch (...) {
    return KVC_ERR_NOMEM;
  }
}

#define KVC_TRY(expr)               \
  do {                              \
    if (const int rc_ = (expr)) return rc_; \
  } while (0)

#define KVC_REQUIRE_INTS(p)                                                       \
  do {                                                                            \
    if (!(p)) return fail(h, KVC_ERR_ARG, "null pointer: " #p);                   \
    if (!aligned4(p)) return fail(h, KVC_ERR_ALIGN, "not 4-byte aligned: " #p);   \
  } while (0)

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
  return guarded([&] {
    KVC_TRY(check(h, c));
    if (n < 1) return fail(h, KVC_ERR_SHAPE, "n must be >= 1");
    KVC_TRY(check_rows(h, k, "k", false, c->n_layers, h->dims.B, h->dims.H, n));
    KVC_TRY(check_rows(h, v, "v", false, c->n_layers, h->dims.B, h->dims.H, n));
    KVC_REQUIRE_INTS(n_new);
    const long long units = static_cast<long long>(c->n_layers) * h->dims.B * h->dims.H;
    const long long most = std::min<long long>(n, static_cast<long long>(c->max_blocks) * c->block_size);
    if (units > INT_MAX / ((most + c->block_size - 2) / c->block_size + 1))
      return fail(h, KVC_ERR_UNSUPPORTED, "too many blocks to write in one call");
    return run(h, kvc::kKernelCache8Append, "cache8 append", stream, [&](cudaStream_t s) {
      return kvc::cache8::launch_append(view(h, *c), c->format, rows(*k), rows(*v), n, n_new, s);
    });
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
