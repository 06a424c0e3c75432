// api_decode.hip -- the exported calls of include/mnb_decode.h: argument validation, workspace
// sizes and kernel launches.
#include <math.h>
#include <stdio.h>

#include "checks.h"
#include "decode.h"
#include "mnb_decode.h"

using namespace mnb;

namespace {

constexpr int64_t kMaxTokens = 1 << 30;        // positions of a sequence, and rows x heads of a call

bool bad_head(int D) { return D != 64 && D != 96 && D != 128 && D != 192 && D != 256; }
bool bad_page(int S) { return S < 16 || S > 65536 || (S & (S - 1)); }

int check_sizes(const mnb_kv_cache *c, const mnb_kv_rows *r) {
  if (!c || !r || c->pages < 0 || c->kv_heads < 0 || r->batch < 0 || r->width < 0 || r->rows < 0) return MNB_ERR_INVALID_ARG;
  if (bad_head(c->head_dim) || bad_page(c->page_size) || c->kv_heads > 65536) return MNB_ERR_UNSUPPORTED;
  if (!r->starts && r->rows != r->batch) return MNB_ERR_INVALID_ARG;
  // a launch has fewer than 2^32 threads, up to 1024 a row
  if ((int64_t)r->width * c->page_size > kMaxTokens || r->rows >= 1 << 22 || r->batch >= 1 << 22) return MNB_ERR_UNSUPPORTED;
  return MNB_OK;
}
bool nothing(const mnb_kv_cache *c, const mnb_kv_rows *r) { return r->rows == 0 || r->batch == 0 || c->kv_heads == 0; }

int check_buffers(const mnb_kv_cache *c, const mnb_kv_rows *r) {
  if (!c->data || !r->lengths || c->pages == 0 || (r->width && !r->pages)) return MNB_ERR_INVALID_ARG;
  if (c->page_stride < (int64_t)mnb_kv_page_bytes(c->kv_heads, c->head_dim, c->page_size) || c->page_stride > 1ll << 40)
    return MNB_ERR_INVALID_ARG;
  if (bad_ld(r->ldp, r->width)) return MNB_ERR_INVALID_ARG;
  if (off16(c->data) || off16(c->page_stride) || (((uintptr_t)r->pages | (uintptr_t)r->lengths | (uintptr_t)r->starts) & 3))
    return MNB_ERR_MISALIGNED;
  return MNB_OK;
}

KvCache cache_of(const mnb_kv_cache *c) {
  KvCache k{};
  k.data = static_cast<uint8_t *>(c->data);
  k.page_stride = c->page_stride;
  k.pages = c->pages;
  k.heads = c->kv_heads;
  k.D = c->head_dim;
  k.shift = __builtin_ctz(c->page_size);
  return k;
}
KvRows rows_of(const mnb_kv_rows *r) { return KvRows{r->pages, r->ldp, r->lengths, r->starts, r->batch, r->width, r->rows}; }

Span cache_span(const mnb_kv_cache *c) {
  return Span{c->data, c->pages, c->page_stride, (int64_t)mnb_kv_page_bytes(c->kv_heads, c->head_dim, c->page_size)};
}
// the tables of numbers that a call reads
struct Tables {
  Span s[3];
};
Tables tables_of(const mnb_kv_rows *r) {
  return Tables{{{r->width ? r->pages : nullptr, r->batch, r->ldp * 4, (int64_t)r->width * 4},
                 {r->lengths, 1, 0, (int64_t)r->batch * 4},
                 {r->starts, 1, 0, ((int64_t)r->batch + 1) * 4}}};
}
bool over_tables(const Span &out, const mnb_kv_rows *r) {
  const Tables t = tables_of(r);
  return overlap(out, t.s[0]) || overlap(out, t.s[1]) || overlap(out, t.s[2]);
}

// a tensor [rows, heads, head_dim] of `size` bytes an element
int check_heads(const void *p, int64_t ld, int heads, int D, int size) {
  if (!p || bad_ld(ld, (int64_t)heads * D)) return MNB_ERR_INVALID_ARG;
  return off16(p) || off16(ld * size) ? MNB_ERR_MISALIGNED : MNB_OK;
}
Span heads_span(const void *p, int64_t ld, int rows, int heads, int D, int size) {
  return Span{p, rows, ld * size, (int64_t)heads * D * size};
}

// a window that reaches past every position is none
int window_of(const mnb_kv_cache *c, const mnb_kv_rows *r, int window) {
  return window >= (int64_t)r->width * c->page_size ? 0 : window;
}
int check_attention(const mnb_kv_cache *c, const mnb_kv_rows *r, int q_heads, int window) {
  const int st = check_sizes(c, r);
  if (st) return st;
  if (q_heads < 0 || window < 0 || (c->kv_heads && q_heads % c->kv_heads)) return MNB_ERR_INVALID_ARG;
  if ((int64_t)r->rows * q_heads > kMaxTokens) return MNB_ERR_UNSUPPORTED;
  if (nothing(c, r) || q_heads == 0) return MNB_OK;
  // a launch has fewer than 2^32 threads
  if (kv_attn_plan(cache_of(c), rows_of(r), q_heads / c->kv_heads, window_of(c, r, window)).items > 1 << 23) return MNB_ERR_UNSUPPORTED;
  return MNB_OK;
}

}  // namespace

extern "C" {

int mnb_decode_version(void) { return 100; }

size_t mnb_kv_page_bytes(int kv_heads, int head_dim, int page_size) {
  if (kv_heads < 0 || kv_heads > 65536 || bad_head(head_dim) || bad_page(page_size)) return 0;
  return (size_t)kv_heads * kv_head_bytes(page_size, head_dim);
}

int mnb_kv_append(const mnb_kv_cache *cache, const mnb_kv_rows *rows, const void *q, int64_t ldq, int q_heads, const void *k,
                  int64_t ldk, const void *v, int64_t ldv, int dtype, const float *table, int table_rows, int rot,
                  int interleaved, const void *q_weight, const void *k_weight, float eps, void *q_out, int64_t ldo,
                  void *stream) {
  int st = check_sizes(cache, rows);
  if (st) return st;
  if (bad_dtype(dtype, false) || q_heads < 0 || rot < 0 || table_rows < 0 || !(eps >= 0.f)) return MNB_ERR_INVALID_ARG;
  const int D = cache->head_dim;
  if (rot > D || (rot && !table) || (q_heads && !q)) return MNB_ERR_INVALID_ARG;
  if (rot % 16 || q_heads > 65536 || (int64_t)rows->rows * q_heads > kMaxTokens) return MNB_ERR_UNSUPPORTED;
  if (rows->rows == 0 || rows->batch == 0 || (cache->kv_heads == 0 && q_heads == 0)) return MNB_OK;
  if ((st = check_buffers(cache, rows))) return st;
  if ((q_heads && (st = check_heads(q, ldq, q_heads, D, 2))) || (q_heads && (st = check_heads(q_out, ldo, q_heads, D, 2)))) return st;
  if ((cache->kv_heads && (st = check_heads(k, ldk, cache->kv_heads, D, 2))) ||
      (cache->kv_heads && (st = check_heads(v, ldv, cache->kv_heads, D, 2))))
    return st;
  if (off16(q_weight) || off16(k_weight) || ((uintptr_t)table & 15)) return MNB_ERR_MISALIGNED;
  const Span c = cache_span(cache), sq = heads_span(q_heads ? q : nullptr, ldq, rows->rows, q_heads, D, 2),
             so = heads_span(q_heads ? q_out : nullptr, ldo, rows->rows, q_heads, D, 2),
             sk = heads_span(k, ldk, rows->rows, cache->kv_heads, D, 2), sv = heads_span(v, ldv, rows->rows, cache->kv_heads, D, 2),
             wq{q_weight, 1, 0, 2 * D}, wk{k_weight, 1, 0, 2 * D}, tb{rot ? table : nullptr, 1, 0, (int64_t)table_rows * rot * 4};
  const Span in[] = {sk, sv, wq, wk, tb};
  for (const Span &s : in)
    if (overlap(c, s) || overlap(so, s)) return MNB_ERR_ALIAS;
  if (overlap(c, sq) || overlap(c, so) || (overlap(so, sq) && !same(so, sq))) return MNB_ERR_ALIAS;
  if (over_tables(c, rows) || over_tables(so, rows)) return MNB_ERR_ALIAS;
  KvAppendParams p{};
  p.cache = cache_of(cache);
  p.rows = rows_of(rows);
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.qw = static_cast<const uint16_t *>(q_weight);
  p.kw = static_cast<const uint16_t *>(k_weight);
  p.out = static_cast<uint16_t *>(q_out);
  p.table = table;
  p.ldq = ldq;
  p.ldk = ldk;
  p.ldv = ldv;
  p.ldo = ldo;
  p.q_heads = q_heads;
  p.table_rows = table_rows;
  p.rot = rot;
  p.interleaved = interleaved;
  p.eps = eps;
  return status(launch_kv_append(dtype, p, as_stream(stream)));
}

int mnb_kv_read(const mnb_kv_cache *cache, const mnb_kv_rows *rows, void *k, int64_t ldk, void *v, int64_t ldv, int dtype,
                void *stream) {
  int st = check_sizes(cache, rows);
  if (st) return st;
  if (bad_dtype(dtype, true)) return MNB_ERR_INVALID_ARG;
  if (nothing(cache, rows) || (!k && !v)) return MNB_OK;
  if ((st = check_buffers(cache, rows))) return st;
  const int D = cache->head_dim, sz = elem_size(dtype);
  if ((k && (st = check_heads(k, ldk, cache->kv_heads, D, sz))) || (v && (st = check_heads(v, ldv, cache->kv_heads, D, sz)))) return st;
  const Span c = cache_span(cache), sk = heads_span(k, ldk, rows->rows, cache->kv_heads, D, sz),
             sv = heads_span(v, ldv, rows->rows, cache->kv_heads, D, sz);
  if (overlap(sk, c) || overlap(sv, c) || overlap(sk, sv) || over_tables(sk, rows) || over_tables(sv, rows)) return MNB_ERR_ALIAS;
  return status(launch_kv_read(dtype, KvReadParams{cache_of(cache), rows_of(rows), k, v, ldk, ldv}, as_stream(stream)));
}

size_t mnb_kv_attention_workspace_bytes(const mnb_kv_cache *cache, const mnb_kv_rows *rows, int q_heads, int window) {
  if (check_attention(cache, rows, q_heads, window) || nothing(cache, rows) || q_heads == 0) return 0;
  return kv_attn_plan(cache_of(cache), rows_of(rows), q_heads / cache->kv_heads, window_of(cache, rows, window)).bytes;
}

int mnb_kv_describe_route(const mnb_kv_cache *cache, const mnb_kv_rows *rows, int q_heads, int window, char *buf, size_t buf_len) {
  const int st = check_attention(cache, rows, q_heads, window);
  if (st) return st;
  if (!buf || buf_len == 0) return MNB_ERR_INVALID_ARG;
  if (nothing(cache, rows) || q_heads == 0) {
    snprintf(buf, buf_len, "noop");
    return MNB_OK;
  }
  const KvPlan k = kv_attn_plan(cache_of(cache), rows_of(rows), q_heads / cache->kv_heads, window_of(cache, rows, window));
  snprintf(buf, buf_len, "kv_attention tile=%d workgroups=%d%s", k.tile_rows, k.workgroups, k.whole ? "" : " join");
  return MNB_OK;
}

int mnb_kv_attention(const mnb_kv_cache *cache, const mnb_kv_rows *rows, const void *q, int64_t ldq, int q_heads, int dtype,
                     float scale, int window, void *y, int64_t ldy, void *workspace, size_t ws_bytes, void *stream) {
  int st = check_attention(cache, rows, q_heads, window);
  if (st) return st;
  if (bad_dtype(dtype, false) || !isfinite(scale)) return MNB_ERR_INVALID_ARG;
  if (nothing(cache, rows) || q_heads == 0) return MNB_OK;
  if ((st = check_buffers(cache, rows))) return st;
  const int D = cache->head_dim;
  if ((st = check_heads(q, ldq, q_heads, D, 2)) || (st = check_heads(y, ldy, q_heads, D, 2))) return st;
  if (off16(workspace)) return MNB_ERR_MISALIGNED;
  KvAttnParams p{};
  p.cache = cache_of(cache);
  p.rows = rows_of(rows);
  p.G = q_heads / cache->kv_heads;
  p.window = window_of(cache, rows, window);
  const KvPlan k = kv_attn_plan(p.cache, p.rows, p.G, p.window);
  const size_t need = k.bytes;
  if (need && (!workspace || ws_bytes < need)) return MNB_ERR_WORKSPACE;
  const Span c = cache_span(cache), sq = heads_span(q, ldq, rows->rows, q_heads, D, 2), sy = heads_span(y, ldy, rows->rows, q_heads, D, 2),
             ws{need ? workspace : nullptr, 1, 0, (int64_t)need};
  if (overlap(sy, c) || (overlap(sy, sq) && !same(sy, sq)) || overlap(ws, c) || overlap(ws, sq) || overlap(ws, sy)) return MNB_ERR_ALIAS;
  if (over_tables(sy, rows) || over_tables(ws, rows)) return MNB_ERR_ALIAS;
  p.q = static_cast<const uint16_t *>(q);
  p.y = static_cast<uint16_t *>(y);
  p.ldq = ldq;
  p.ldy = ldy;
  // at 0 a masked score would be no number (infinity times 0): the least scale instead, which leaves finite scores alike
  p.scale = scale == 0.f ? 0x1p-126f : fabsf(scale) * 1.4426950408889634f;
  p.flip = scale < 0.f ? 0x80008000u : 0;
  p.whole = k.whole;
  p.workgroups = k.workgroups;
  p.lone = k.lone;
  p.sharers = k.sharers;
  p.least = k.least;
  p.tile_rows = k.tile_rows;
  p.slot_rows = k.slot_rows;
  p.part = static_cast<float *>(workspace);
  return status(launch_kv_attn(dtype, p, as_stream(stream)));
}

int mnb_sample(const void *logits, int dtype, int M, int V, int64_t ldl, const float *u, const float *temperature,
               float temperature_all, const int32_t *top_k, int top_k_all, const float *top_p, float top_p_all,
               const float *min_p, float min_p_all, int64_t *tokens, void *stream) {
  if (M < 0 || V < 0 || bad_dtype(dtype, true)) return MNB_ERR_INVALID_ARG;
  if (V > 1 << 22) return MNB_ERR_UNSUPPORTED;
  if (M == 0) return MNB_OK;
  if (V == 0 || !logits || bad_ld(ldl, V) || !u || !tokens) return MNB_ERR_INVALID_ARG;
  const int sz = elem_size(dtype);
  if (((uintptr_t)logits & (sz - 1)) || ((uintptr_t)tokens & 7) ||
      (((uintptr_t)u | (uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p) & 3))
    return MNB_ERR_MISALIGNED;
  const Span out{tokens, 1, 0, (int64_t)M * 8}, in[] = {{logits, M, ldl * sz, (int64_t)V * sz}, {u, 1, 0, (int64_t)M * 4},
                                                        {temperature, 1, 0, (int64_t)M * 4}, {top_k, 1, 0, (int64_t)M * 4},
                                                        {top_p, 1, 0, (int64_t)M * 4}, {min_p, 1, 0, (int64_t)M * 4}};
  for (const Span &s : in)
    if (overlap(out, s)) return MNB_ERR_ALIAS;
  SampleParams p{logits, ldl, u, temperature, top_p, min_p, top_k, temperature_all, top_p_all, min_p_all, top_k_all, tokens, M, V};
  // a launch has fewer than 2^32 threads, 1024 a row
  for (int m0 = 0; m0 < M; m0 += 1 << 20) {
    SampleParams q = p;
    q.M = M - m0 < 1 << 20 ? M - m0 : 1 << 20;
    q.x = static_cast<const char *>(logits) + (int64_t)m0 * ldl * sz;
    q.u += m0;
    if (temperature) q.temperature += m0;
    if (top_k) q.top_k += m0;
    if (top_p) q.top_p += m0;
    if (min_p) q.min_p += m0;
    q.tokens += m0;
    const hipError_t e = launch_sample(dtype, q, as_stream(stream));
    if (e != hipSuccess) return MNB_ERR_HIP;
    if (M - m0 <= 1 << 20) break;
  }
  return MNB_OK;
}

}  // extern "C"
