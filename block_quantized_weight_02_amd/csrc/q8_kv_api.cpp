// q8_kv_api.cpp -- host side of the cache and attention calls declared in
// include/q8gemv.h: argument validation before any launch, and errors.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/q8gemv.h"
#include "q8_internal.h"
#include "q8_kv.h"

namespace {

using q8::report_error;

// Workspace bytes of the arrival counters: the products' counter region, so
// that one zeroed workspace serves both.
constexpr size_t kCounterBytes = (size_t)4 << 20;
constexpr int64_t kMaxInt = 0x7fffffff;
constexpr int64_t kMaxTokens = (int64_t)1 << 30;   // of a sequence that attention reads

int ok() {
  report_error(Q8_OK, "%s", "");
  return Q8_OK;
}

int check_ptr(const void *p, const char *name) {
  if (!p) return report_error(Q8_ERR_NULL, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % 16 != 0)
    return report_error(Q8_ERR_ALIGN, "%s = %p is not 16-byte aligned", name, p);
  return Q8_OK;
}

int check_opt(const void *p, const char *name) { return p ? check_ptr(p, name) : (int)Q8_OK; }

int check_range(int64_t v, int64_t lo, int64_t hi, const char *name) {
  if (v < lo || v > hi)
    return report_error(Q8_ERR_SHAPE, "%s = %lld out of range: need %lld <= %s <= %lld", name,
                        (long long)v, (long long)lo, name, (long long)hi);
  return Q8_OK;
}

int check_page(int64_t page) {
  if (page != 16 && page != 32 && page != 64 && page != 128 && page != 256)
    return report_error(Q8_ERR_SHAPE, "page = %lld: need 16, 32, 64, 128 or 256 tokens",
                        (long long)page);
  return Q8_OK;
}

int check_cache_shape(int fmt, int64_t kv_heads, int64_t head_dim, int64_t page, int64_t n_pages) {
  int st;
  if (fmt != Q8_KV_BF16 && fmt != Q8_KV_Q8_0)
    return report_error(Q8_ERR_ACT_FMT, "cache fmt = %d: need 0 (bf16) or 1 (Q8_0)", fmt);
  if ((st = check_range(kv_heads, 1, 128, "kv_heads"))) return st;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return report_error(Q8_ERR_SHAPE, "head_dim = %lld: need 64, 128 or 256", (long long)head_dim);
  if ((st = check_page(page))) return st;
  return check_range(n_pages, 1, kMaxInt / page, "n_pages");
}

int check_cache(const q8_kv_cache *c, q8::KvCache *out) {
  int st;
  if (!c) return report_error(Q8_ERR_NULL, "cache is NULL");
  if ((st = check_cache_shape(c->fmt, c->kv_heads, c->head_dim, c->page, c->n_pages))) return st;
  if (out) {
    if ((st = check_ptr(c->k, "cache k"))) return st;
    if ((st = check_ptr(c->v, "cache v"))) return st;
    out->k = static_cast<char *>(c->k);
    out->v = static_cast<char *>(c->v);
    out->n_pages = (int)c->n_pages;
    out->heads = c->kv_heads;
    out->dim = c->head_dim;
    out->fmt = c->fmt;
    out->page_log2 = 0;
    while ((1 << out->page_log2) < c->page) ++out->page_log2;
  }
  return Q8_OK;
}

int check_heads(int64_t q_heads, int64_t kv_heads) {
  const int st = check_range(q_heads, 1, 1024, "q_heads");
  if (st) return st;
  if (q_heads % kv_heads)
    return report_error(Q8_ERR_SHAPE, "q_heads = %lld is not a multiple of kv_heads = %lld",
                        (long long)q_heads, (long long)kv_heads);
  return Q8_OK;
}

int check_ld(int64_t ld, int64_t width, const char *name) {
  if (ld < width || ld % 4 || ld > kMaxInt)
    return report_error(Q8_ERR_SHAPE, "%s = %lld: need a multiple of 4, at least %lld", name,
                        (long long)ld, (long long)width);
  return Q8_OK;
}

int done(hipError_t e, const char *what) {
  if (e == hipSuccess) return ok();
  (void)hipGetLastError();   // do not leave the failure for the caller's next HIP call
  return report_error(Q8_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

size_t attn_ws_bytes(int64_t m, int64_t n, int64_t q_heads, const q8_kv_cache *c) {
  const int64_t kv_heads = c->kv_heads, dim = c->head_dim;
  const size_t p = m > 0 ? q8::attn_rows_partial_bytes(m, n, q_heads, kv_heads, dim, c->fmt)
                         : q8::attn_decode_partial_bytes(n, q_heads, kv_heads, dim);
  return p ? kCounterBytes + (size_t)round_up((int64_t)p, 256) : 0;
}

int check_attn_sizes(int64_t m, int64_t n, int64_t q_heads, const q8_kv_cache *cache, bool rows) {
  int st;
  if ((st = check_range(n, 1, Q8_MAX_SEQS, "n"))) return st;
  if (rows && (st = check_range(m, 1, 8192, "m"))) return st;
  if ((st = check_cache(cache, nullptr))) return st;
  return check_heads(q_heads, cache->kv_heads);
}

int run_attn(const uint16_t *q, int64_t m, int64_t q_heads, const q8_kv_cache *cache,
             const int32_t *table, int64_t max_pages, const int32_t *lens,
             const int32_t *row_start, int64_t n, const q8_attn *attn, uint16_t *o, void *o_q8,
             hipStream_t stream, void *workspace, size_t ws_bytes, bool rows) {
  int st;
  if ((st = check_attn_sizes(m, n, q_heads, cache, rows))) return st;
  // positions, and a tile or a window past them, stay in 32 bits
  if ((st = check_range(max_pages, 1, std::min(kMaxInt / n, kMaxTokens / cache->page),
                        "max_pages"))) return st;
  if (n * max_pages > (int64_t(1) << 35) / cache->page)
    return report_error(Q8_ERR_SHAPE, "n * max_pages * page = %lld exceeds 2^35",
                        (long long)(n * max_pages * cache->page));
  if (!attn) return report_error(Q8_ERR_NULL, "attn is NULL");
  const float scale_log2 = (float)((double)attn->scale * 1.4426950408889634074);
  if (!std::isfinite(scale_log2))
    return report_error(Q8_ERR_SHAPE, "scale = %g: need |scale| < 2^127", (double)attn->scale);
  if ((st = check_range(attn->window, 0, kMaxInt, "window"))) return st;
  if ((st = check_range(attn->sinks, 0, kMaxInt, "sinks"))) return st;
  q8::AttnArgs a{};
  if ((st = check_cache(cache, &a.cache))) return st;
  if ((st = check_ptr(q, "q"))) return st;
  if ((st = check_ptr(table, "table"))) return st;
  if ((st = check_ptr(lens, "lens"))) return st;
  if (rows && (st = check_ptr(row_start, "row_start"))) return st;
  if (!o && !o_q8) return report_error(Q8_ERR_NULL, "neither o nor o_q8 is given");
  if ((st = check_opt(o, "o")) || (st = check_opt(o_q8, "o_q8"))) return st;
  const int64_t M = rows ? m : n, K = q_heads * cache->head_dim;
  const size_t need = attn_ws_bytes(rows ? m : 0, n, q_heads, cache);
  if (need) {
    if (!workspace || ws_bytes < need)
      return report_error(Q8_ERR_WORKSPACE, "workspace of %zu bytes given, %zu needed",
                          workspace ? ws_bytes : (size_t)0, need);
    if ((st = check_ptr(workspace, "workspace"))) return st;
    a.counters = static_cast<unsigned *>(workspace);
    a.partial = reinterpret_cast<float *>(static_cast<char *>(workspace) + kCounterBytes);
  }
  a.q = q;
  a.m = (int)M;
  a.n = (int)n;
  a.q_heads = (int)q_heads;
  a.group = (int)(q_heads / cache->kv_heads);
  a.table = table;
  a.max_pages = max_pages;
  a.lens = lens;
  a.row_start = rows ? row_start : nullptr;
  a.scale_log2 = scale_log2;
  a.window = (int)std::min<int64_t>(attn->window, kMaxTokens);   // all of a sequence, as it was
  a.sinks = (int)std::min<int64_t>(attn->sinks, kMaxTokens);
  a.o = o;
  if (o_q8) {
    a.oq = static_cast<int8_t *>(o_q8);
    a.oq_scale = reinterpret_cast<float *>(a.oq + q8_act_scales_offset(M, K));
    a.oq_view = a.oq + q8_act_view_offset(M, K);
  }
  (void)hipGetLastError();  // clear a stale error so the launch's own is seen
  if (rows) {
    a.chunks = q8::attn_rows_splits(m, n, q_heads, cache->kv_heads, cache->head_dim, cache->fmt);
    return done(q8::launch_attn_rows(a, stream), "attn_rows launch");
  }
  const int64_t units = cache->kv_heads * ((a.group + 15) / 16);
  a.chunks = q8::attn_decode_chunks(units);
  return done(q8::launch_attn_decode(a, stream), "attn_decode launch");
}

}  // namespace

extern "C" {

size_t q8_kv_bytes(int fmt, int64_t kv_heads, int64_t head_dim, int64_t page, int64_t n_pages) {
  if (check_cache_shape(fmt, kv_heads, head_dim, page, n_pages)) return 0;
  q8::KvCache c{};
  c.heads = (int)kv_heads;
  c.dim = (int)head_dim;
  c.fmt = fmt;
  while ((1 << c.page_log2) < page) ++c.page_log2;
  return c.page_bytes() * (size_t)n_pages;
}

int q8_kv_step(const q8_kv_step_args *s, hipStream_t stream) {
  int st;
  if (!s) return report_error(Q8_ERR_NULL, "step is NULL");
  if ((st = check_range(s->n, 1, Q8_MAX_SEQS, "n"))) return st;
  if ((st = check_range(s->m, 1, Q8_MAX_GEMM_ROWS, "m"))) return st;
  if ((st = check_page(s->page))) return st;
  if ((st = check_range(s->max_pages, 1, kMaxInt / 2 / s->n, "max_pages"))) return st;
  if ((st = check_range(s->free_cap, 1, kMaxInt, "free_cap"))) return st;
  const struct { const void *p; const char *name; } ptrs[] = {
      {s->lens, "lens"}, {s->new_rows, "new_rows"}, {s->table, "table"},
      {s->free_pages, "free_pages"}, {s->free_count, "free_count"}, {s->lens_out, "lens_out"},
      {s->free_count_out, "free_count_out"}, {s->row_start, "row_start"},
      {s->positions, "positions"}, {s->slots, "slots"}, {s->status, "status"}};
  for (const auto &p : ptrs)
    if ((st = check_ptr(p.p, p.name))) return st;
  (void)hipGetLastError();
  return done(q8::launch_kv_step(*s, stream), "kv_step launch");
}

int q8_rope_freqs(const q8_rope *r, double *freqs, hipStream_t stream) {
  int st;
  if (!r) return report_error(Q8_ERR_NULL, "rope is NULL");
  if (r->rot < 8 || r->rot > 256 || r->rot % 8)
    return report_error(Q8_ERR_SHAPE, "rot = %d: need a multiple of 8, 8 <= rot <= 256", r->rot);
  if (r->scaling < Q8_ROPE_SCALE_NONE || r->scaling > Q8_ROPE_SCALE_INDEX)
    return report_error(Q8_ERR_ACT_FMT, "scaling = %d: need 0 .. 3", r->scaling);
  if (!(std::isfinite(r->base) && r->base > 1.0))
    return report_error(Q8_ERR_SHAPE, "base = %g: need base > 1", r->base);
  if (r->scaling != Q8_ROPE_SCALE_NONE && !(std::isfinite(r->factor) && r->factor >= 1.0))
    return report_error(Q8_ERR_SHAPE, "factor = %g: need factor >= 1", r->factor);
  if (r->scaling == Q8_ROPE_SCALE_TURNS || r->scaling == Q8_ROPE_SCALE_INDEX) {
    if (!(std::isfinite(r->high) && r->low > 0.0 && r->high > r->low))
      return report_error(Q8_ERR_SHAPE, "low = %g, high = %g: need high > low > 0", r->low, r->high);
    if ((st = check_range(r->original, 1, kMaxInt, "original"))) return st;
  }
  if ((st = check_ptr(freqs, "freqs"))) return st;
  (void)hipGetLastError();
  return done(q8::launch_rope_freqs(*r, freqs, stream), "rope_freqs launch");
}

int q8_qkv_heads(const float *q, int64_t ldq, const float *k, int64_t ldk, const float *v,
                 int64_t ldv, int64_t m, int64_t q_heads, const q8_heads *h,
                 const int32_t *positions, const int32_t *slots, uint16_t *q_out,
                 const q8_kv_cache *cache, hipStream_t stream) {
  int st;
  q8::HeadsArgs a{};
  if ((st = check_range(m, 1, Q8_MAX_GEMM_ROWS, "m"))) return st;
  if ((st = check_cache(cache, &a.cache))) return st;
  if ((st = check_heads(q_heads, cache->kv_heads))) return st;
  const int64_t D = cache->head_dim;
  if ((st = check_ld(ldq, q_heads * D, "ldq"))) return st;
  if ((st = check_ld(ldk, cache->kv_heads * D, "ldk"))) return st;
  if ((st = check_ld(ldv, cache->kv_heads * D, "ldv"))) return st;
  if (!h) return report_error(Q8_ERR_NULL, "heads is NULL");
  if (h->rot < 0 || h->rot > D || h->rot % 8)
    return report_error(Q8_ERR_SHAPE, "rot = %d: need a multiple of 8, 0 <= rot <= head_dim = %lld",
                        h->rot, (long long)D);
  if (h->layout != Q8_ROPE_HALF && h->layout != Q8_ROPE_INTERLEAVED)
    return report_error(Q8_ERR_ACT_FMT, "layout = %d: need 0 (half) or 1 (interleaved)", h->layout);
  if (!(std::isfinite(h->eps) && h->eps >= 0.0f))
    return report_error(Q8_ERR_SHAPE, "eps = %g: need eps >= 0", (double)h->eps);
  if (!std::isfinite(h->attn_factor)) return report_error(Q8_ERR_SHAPE, "attn_factor is not finite");
  if ((st = check_ptr(q, "q")) || (st = check_ptr(k, "k")) || (st = check_ptr(v, "v"))) return st;
  if ((st = check_opt(h->q_norm, "q_norm")) || (st = check_opt(h->k_norm, "k_norm"))) return st;
  if (h->rot > 0 && (st = check_ptr(h->freqs, "freqs"))) return st;
  if ((st = check_ptr(positions, "positions")) || (st = check_ptr(slots, "slots")) ||
      (st = check_ptr(q_out, "q_out")))
    return st;
  a.q = q;
  a.k = k;
  a.v = v;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.m = (int)m;
  a.q_heads = (int)q_heads;
  a.q_norm = h->q_norm;
  a.k_norm = h->k_norm;
  a.freqs = h->freqs;
  a.eps = h->eps;
  a.attn_factor = h->attn_factor;
  a.rot = h->rot;
  a.layout = h->layout;
  a.positions = positions;
  a.slots = slots;
  a.q_out = q_out;
  (void)hipGetLastError();
  return done(q8::launch_qkv_heads(a, stream), "qkv_heads launch");
}

int q8_kv_gather(const q8_kv_cache *cache, const int32_t *slots, int64_t rows, uint16_t *k_out,
                 uint16_t *v_out, hipStream_t stream) {
  int st;
  q8::KvCache c{};
  if ((st = check_range(rows, 1, 1 << 24, "rows"))) return st;
  if ((st = check_cache(cache, &c))) return st;
  if ((st = check_ptr(slots, "slots"))) return st;
  if (!k_out && !v_out) return report_error(Q8_ERR_NULL, "neither k_out nor v_out is given");
  if ((st = check_opt(k_out, "k_out")) || (st = check_opt(v_out, "v_out"))) return st;
  (void)hipGetLastError();
  return done(q8::launch_kv_gather(c, slots, (int)rows, k_out, v_out, stream), "kv_gather launch");
}

size_t q8_attn_workspace_bytes(int64_t m, int64_t n, int64_t q_heads, const q8_kv_cache *cache) {
  if (m < 0 || check_attn_sizes(m, n, q_heads, cache, m > 0)) return 0;
  return attn_ws_bytes(m, n, q_heads, cache);
}

int q8_attn_decode(const uint16_t *q, int64_t q_heads, const q8_kv_cache *cache,
                   const int32_t *table, int64_t max_pages, const int32_t *lens, int64_t n,
                   const q8_attn *attn, uint16_t *o, void *o_q8, hipStream_t stream,
                   void *workspace, size_t ws_bytes) {
  return run_attn(q, n, q_heads, cache, table, max_pages, lens, nullptr, n, attn, o, o_q8, stream,
                  workspace, ws_bytes, false);
}

int q8_attn_rows(const uint16_t *q, int64_t m, int64_t q_heads, const q8_kv_cache *cache,
                 const int32_t *table, int64_t max_pages, const int32_t *lens,
                 const int32_t *row_start, int64_t n, const q8_attn *attn, uint16_t *o, void *o_q8,
                 hipStream_t stream, void *workspace, size_t ws_bytes) {
  return run_attn(q, m, q_heads, cache, table, max_pages, lens, row_start, n, attn, o, o_q8, stream,
                  workspace, ws_bytes, true);
}

}  // extern "C"
