// C ABI of the attention side (declared in include/pi_attn.h): host checks and
// launches.  Every check comes before the first launch.
#include <math.h>

#include "attn_internal.h"
#include "pi.h"

namespace {

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int64_t kMaxInt = 0x7fffffff;
constexpr int kMaxBlocks = 1 << 24;      // blocks of a table row: token numbers fit 32 bits
constexpr int64_t kMaxStride = int64_t(1) << 40;

int elem_bytes(int dtype) { return dtype == PI_F32 ? 4 : 2; }

// Rows [n_tok][n][d] with strides: each head is 16-byte aligned and the heads of a token do not
// overlap, nor do the tokens.
pi_status check_rows(const void* p, int64_t ts, int64_t hs, int n, int n_tok, int d, int dtype) {
  if (!p) return PI_E_NULL;
  if (n < 1) return PI_E_SHAPE;
  const int64_t v = 16 / elem_bytes(dtype);
  if (n > 1 && (hs % v || hs < d || hs > kMaxStride)) return PI_E_SHAPE;
  if (n_tok > 1 && (ts % v || ts < d || ts > kMaxStride)) return PI_E_SHAPE;
  // one of the strides spans the other's extent
  if (n > 1 && n_tok > 1 && ts < hs * (n - 1) + d && hs < ts * (n_tok - 1) + d) return PI_E_SHAPE;
  if (!al16(p)) return PI_E_ALIGN;
  return PI_OK;
}

// Bytes from the first element to the end of the last.
size_t span(int64_t ts, int64_t hs, int n, int n_tok, int d, int dtype) {
  return (size_t)(ts * (n_tok - 1) + (n > 1 ? hs * (n - 1) : 0) + d) * elem_bytes(dtype);
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// Whether rows [n_tok][n][d] and [n_tok][m][d] share a byte (or may: rows of unlike
// token strides, or of very many heads, whose spans meet).  Parts of one buffer lie
// in each other's spans: first their places inside a token are compared, then
// every head with every other.
bool rows_meet(const void* p, int64_t ts, int64_t hs, int n, const void* r, int64_t rts, int64_t rhs, int m, int n_tok,
               int d, int dtype) {
  if (n == 1) hs = 0;
  if (m == 1) rhs = 0;
  if (!overlap(p, span(ts, hs, n, n_tok, d, dtype), r, span(rts, rhs, m, n_tok, d, dtype))) return false;
  if (n_tok > 1 && ts != rts) return true;
  const int64_t size = elem_bytes(dtype), row = n_tok > 1 ? ts * size : 0, w = d * size;
  const int64_t gap = (int64_t)(reinterpret_cast<uintptr_t>(r) - reinterpret_cast<uintptr_t>(p));
  const int64_t np = hs * (n - 1) * size + w, nr = rhs * (m - 1) * size + w;
  if (row && np <= row && nr <= row) {
    const int64_t at = ((gap % row) + row) % row;             // where r's heads begin inside p's token
    if (at >= np && at + nr <= row) return false;
  }
  if ((int64_t)n * m > 1 << 16) return true;
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < m; ++j) {
      const int64_t x = gap + (j * rhs - i * hs) * size;      // between the heads' first tokens
      int64_t k = row ? -x / row : 0;                         // tokens that bring them nearest, one more or less
      k = k > n_tok - 2 ? n_tok - 2 : k < 2 - n_tok ? 2 - n_tok : k;
      for (int64_t e = row ? -1 : 0; e <= (row ? 1 : 0); ++e) {
        const int64_t y = x + (k + e) * row;
        if (y < w && -y < w) return true;
      }
    }
  return false;
}

pi_status check_cache(const pi_kv_cache* c) {
  if (!c) return PI_E_NULL;
  if (c->dtype != PI_F16 && c->dtype != PI_F32) return PI_E_DTYPE;
  if (c->head_dim != 64 && c->head_dim != 128) return PI_E_SHAPE;
  if (c->n_seqs < 1 || c->n_kv_heads < 1 || c->max_blocks < 1 || c->max_blocks > kMaxBlocks || c->n_pages < 1)
    return PI_E_SHAPE;
  if ((int64_t)c->n_seqs * c->n_kv_heads > kMaxInt) return PI_E_SHAPE;
  if (!c->pages || !c->scales || !c->open || !c->table) return PI_E_NULL;
  if (!al16(c->pages) || !al16(c->scales) || !al16(c->open) || !al16(c->table) || !al16(c->score)) return PI_E_ALIGN;
  return PI_OK;
}

pi::HeadRows head_rows(const void* p, int64_t ts, int64_t hs, int n) {
  pi::HeadRows r;
  r.p = const_cast<void*>(p);
  r.ts = ts;
  r.hs = n > 1 ? hs : 0;
  r.n = n;
  return r;
}

// What pi_kv_append and pi_kv_read share.
pi_status cache_args(const pi_kv_cache* c, const int32_t* lens, const int32_t* q_start, int max_new, const void* k,
                     int64_t k_ts, int64_t k_hs, const void* v, int64_t v_ts, int64_t v_hs, int n_tok,
                     pi::CacheArgs* a) {
  pi_status st = check_cache(c);
  if (st != PI_OK) return st;
  if (!lens) return PI_E_NULL;
  if (n_tok < 1 || max_new < 1 || max_new > (int64_t)c->max_blocks * PI_KV_BLOCK) return PI_E_SHAPE;
  if (!q_start && (int64_t)c->n_seqs * max_new > n_tok) return PI_E_SHAPE;
  if ((st = check_rows(k, k_ts, k_hs, c->n_kv_heads, n_tok, c->head_dim, c->dtype)) != PI_OK) return st;
  if ((st = check_rows(v, v_ts, v_hs, c->n_kv_heads, n_tok, c->head_dim, c->dtype)) != PI_OK) return st;
  if (!al4(lens) || !al4(q_start)) return PI_E_ALIGN;
  a->n_seqs = c->n_seqs;
  a->hk = c->n_kv_heads;
  a->d = c->head_dim;
  a->max_blocks = c->max_blocks;
  a->n_pages = c->n_pages;
  a->dtype = c->dtype;
  a->pages = c->pages;
  a->scales = c->scales;
  a->open = c->open;
  a->table = c->table;
  a->lens = lens;
  a->q_start = q_start;
  a->max_new = max_new;
  a->n_tok = n_tok;
  a->kv[0] = head_rows(k, k_ts, k_hs, c->n_kv_heads);
  a->kv[1] = head_rows(v, v_ts, v_hs, c->n_kv_heads);
  return pi::kv_cache_threads(*a) > pi::kMaxThreads ? PI_E_SHAPE : PI_OK;
}

pi_status plan_for(const pi_kv_cache* c, int n_heads, int max_q, int max_len, bool score, pi::AttendPlan* p) {
  const pi_status st = check_cache(c);
  if (st != PI_OK) return st;
  if (n_heads < 1 || n_heads % c->n_kv_heads || max_q < 1) return PI_E_SHAPE;
  if (max_len < 1 || max_len > (int64_t)c->max_blocks * PI_KV_BLOCK) return PI_E_RANGE;
  const int group = n_heads / c->n_kv_heads;
  if ((int64_t)c->n_seqs * n_heads * max_q > kMaxInt / 2) return PI_E_SHAPE;
  *p = pi::attend_plan(c->n_seqs, c->n_kv_heads, group, c->head_dim, c->dtype, max_q, max_len, score);
  const int64_t pairs = (int64_t)c->n_seqs * c->n_kv_heads;
  if (p->threads > pi::kMaxThreads || pairs * (p->r_max + p->max_nb) > kMaxInt) return PI_E_SHAPE;
  return PI_OK;
}

}  // namespace

extern "C" {

pi_status pi_qk_rope(const pi_rope* rope, const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                     int32_t n_heads, const void* k, int64_t k_tok_stride, int64_t k_head_stride,
                     int32_t n_kv_heads, const int32_t* pos, int32_t n_tok, int32_t dtype, void* q_out,
                     int64_t qo_tok_stride, int64_t qo_head_stride, void* k_out, int64_t ko_tok_stride,
                     int64_t ko_head_stride, void* stream) {
  if (!rope || !pos || !rope->freqs) return PI_E_NULL;
  if (dtype != PI_F16 && dtype != PI_F32) return PI_E_DTYPE;
  if (rope->layout != PI_ROPE_HALF && rope->layout != PI_ROPE_INTERLEAVED) return PI_E_DTYPE;
  const int d = rope->head_dim;
  if (d < 8 || d > 256 || d % 8 || rope->rot < 2 || rope->rot % 2 || rope->rot > d || n_tok < 1) return PI_E_SHAPE;
  if (!isfinite(rope->scale) || !isfinite(rope->eps) || rope->eps < 0.0f) return PI_E_RANGE;
  if (n_heads < 0 || n_kv_heads < 0 || (n_heads == 0 && n_kv_heads == 0)) return PI_E_SHAPE;
  if ((int64_t)n_heads + n_kv_heads > (1 << 20)) return PI_E_SHAPE;
  if (!al4(pos) || (reinterpret_cast<uintptr_t>(rope->freqs) & 7u) || !al4(rope->q_norm) || !al4(rope->k_norm))
    return PI_E_ALIGN;
  pi::RopeArgs a;
  const struct { const void* in; int64_t ts, hs; void* out; int64_t ots, ohs; int n; } two[2] = {
      {q, q_tok_stride, q_head_stride, q_out, qo_tok_stride, qo_head_stride, n_heads},
      {k, k_tok_stride, k_head_stride, k_out, ko_tok_stride, ko_head_stride, n_kv_heads}};
  for (int i = 0; i < 2; ++i) {
    const auto& x = two[i];
    a.in[i] = head_rows(x.in, x.ts, x.hs, x.n);
    a.out[i] = head_rows(x.out, x.ots, x.ohs, x.n);
    if (x.n == 0) continue;
    pi_status st = check_rows(x.in, x.ts, x.hs, x.n, n_tok, d, dtype);
    if (st == PI_OK) st = check_rows(x.out, x.ots, x.ohs, x.n, n_tok, d, dtype);
    if (st != PI_OK) return st;
  }
  // An output is its own input, or apart from both inputs.
  for (int o = 0; o < 2; ++o)
    for (int i = 0; i < 2; ++i) {
      const pi::HeadRows &x = a.out[o], &y = a.in[i];
      if (x.n == 0 || y.n == 0) continue;
      const bool same = o == i && x.p == y.p && x.hs == y.hs && (n_tok == 1 || x.ts == y.ts);
      if (!same && rows_meet(x.p, x.ts, x.hs, x.n, y.p, y.ts, y.hs, y.n, n_tok, d, dtype)) return PI_E_RANGE;
    }
  if (a.out[0].n && a.out[1].n &&
      rows_meet(a.out[0].p, a.out[0].ts, a.out[0].hs, a.out[0].n, a.out[1].p, a.out[1].ts, a.out[1].hs, a.out[1].n, n_tok,
                d, dtype))
    return PI_E_RANGE;
  a.d = d;
  a.rot = rope->rot;
  a.layout = rope->layout;
  a.dtype = dtype;
  a.n_tok = n_tok;
  a.scale = rope->scale;
  a.eps = rope->eps;
  a.freqs = rope->freqs;
  a.w[0] = rope->q_norm;
  a.w[1] = rope->k_norm;
  a.pos = pos;
  if (pi::qk_rope_threads(a) > pi::kMaxThreads) return PI_E_SHAPE;
  const hipError_t e = pi::launch_qk_rope(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? PI_OK : pi::hip_failed(e);
}

pi_status pi_kv_append(const pi_kv_cache* cache, const void* k, int64_t k_tok_stride, int64_t k_head_stride,
                       const void* v, int64_t v_tok_stride, int64_t v_head_stride, int32_t n_tok,
                       const int32_t* lens, const int32_t* q_start, int32_t max_new, void* stream) {
  pi::CacheArgs a;
  const pi_status st = cache_args(cache, lens, q_start, max_new, k, k_tok_stride, k_head_stride, v, v_tok_stride,
                                  v_head_stride, n_tok, &a);
  if (st != PI_OK) return st;
  const hipError_t e = pi::launch_kv_append(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? PI_OK : pi::hip_failed(e);
}

pi_status pi_kv_read(const pi_kv_cache* cache, const int32_t* lens, const int32_t* q_start, int32_t max_new,
                     void* k_out, int64_t k_tok_stride, int64_t k_head_stride, void* v_out, int64_t v_tok_stride,
                     int64_t v_head_stride, int32_t n_tok, void* stream) {
  pi::CacheArgs a;
  const pi_status st = cache_args(cache, lens, q_start, max_new, k_out, k_tok_stride, k_head_stride, v_out,
                                  v_tok_stride, v_head_stride, n_tok, &a);
  if (st != PI_OK) return st;
  if (rows_meet(k_out, k_tok_stride, k_head_stride, cache->n_kv_heads, v_out, v_tok_stride, v_head_stride,
                cache->n_kv_heads, n_tok, cache->head_dim, cache->dtype))
    return PI_E_RANGE;
  const hipError_t e = pi::launch_kv_read(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? PI_OK : pi::hip_failed(e);
}

size_t pi_attend_workspace_bytes(const pi_kv_cache* cache, int32_t n_heads, int32_t max_q, int32_t max_len,
                                 int32_t add_score) {
  pi::AttendPlan p;
  return plan_for(cache, n_heads, max_q, max_len, add_score != 0, &p) == PI_OK ? p.total : 0;
}

pi_status pi_attend(const pi_kv_cache* cache, const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                    int32_t n_heads, int32_t n_tok, const int32_t* lens, const int32_t* q_start, int32_t max_q,
                    int32_t max_len, float scale, int32_t add_score, void* out, int64_t o_tok_stride,
                    int64_t o_head_stride, void* ws, size_t ws_bytes, void* stream) {
  pi::AttendPlan p;
  pi_status st = plan_for(cache, n_heads, max_q, max_len, add_score != 0, &p);
  if (st != PI_OK) return st;
  const int d = cache->head_dim, dtype = cache->dtype;
  if (!lens || (add_score && !cache->score)) return PI_E_NULL;
  if (n_tok < 1 || (int64_t)n_tok * n_heads > kMaxInt / 2) return PI_E_SHAPE;
  if (!q_start && (int64_t)cache->n_seqs * max_q > n_tok) return PI_E_SHAPE;
  if ((st = check_rows(q, q_tok_stride, q_head_stride, n_heads, n_tok, d, dtype)) != PI_OK) return st;
  if ((st = check_rows(out, o_tok_stride, o_head_stride, n_heads, n_tok, d, dtype)) != PI_OK) return st;
  if (!al4(lens) || !al4(q_start)) return PI_E_ALIGN;
  if (!isfinite(scale) || scale < 0.0f) return PI_E_RANGE;
  if (rows_meet(q, q_tok_stride, q_head_stride, n_heads, out, o_tok_stride, o_head_stride, n_heads, n_tok, d, dtype))
    return PI_E_RANGE;
  if (!ws) return PI_E_WORKSPACE;
  if (!al16(ws)) return PI_E_ALIGN;
  if (ws_bytes < p.total) return PI_E_WORKSPACE;
  char* w = static_cast<char*>(ws);
  pi::AttendArgs a;
  a.q = q;
  a.q_ts = q_tok_stride;
  a.q_hs = q_head_stride;
  a.out = out;
  a.o_ts = o_tok_stride;
  a.o_hs = o_head_stride;
  a.lens = lens;
  a.q_start = q_start;
  a.pages = cache->pages;
  a.scales = cache->scales;
  a.table = cache->table;
  a.score = add_score ? cache->score : nullptr;
  a.n_seqs = cache->n_seqs;
  a.hk = cache->n_kv_heads;
  a.group = n_heads / cache->n_kv_heads;
  a.n_tok = n_tok;
  a.max_q = max_q;
  a.max_len = max_len;
  a.max_blocks = cache->max_blocks;
  a.n_pages = cache->n_pages;
  a.scale = (float)((double)scale * 1.4426950408889634);
  a.r_max = p.r_max;
  a.max_nb = p.max_nb;
  a.tiles = p.tiles;
  a.splits = p.splits;
  a.slots = p.slots;
  a.share_even = p.share_even;
  a.share_safe = p.share_safe;
  a.splits_max = p.splits_max;
  a.part = reinterpret_cast<float*>(w + p.part);
  a.ml = reinterpret_cast<float2*>(w + p.ml);
  a.count = reinterpret_cast<int*>(w + p.count);
  a.lse = reinterpret_cast<float*>(w + p.lse);
  a.flags = reinterpret_cast<unsigned*>(w) + PI_WS_FLAGS;
  const hipError_t e = pi::launch_attend(a, p, d, dtype, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? PI_OK : pi::hip_failed(e);
}

pi_status pi_kv_evict(const int32_t* table, const float* score, const int32_t* lens, int32_t n_seqs,
                      int32_t n_kv_heads, int32_t max_blocks, int32_t keep, int32_t recent, int32_t* table_out,
                      float* score_out, int32_t* lens_out, void* stream) {
  if (!table || !score || !lens || !table_out || !score_out || !lens_out) return PI_E_NULL;
  if (n_seqs < 1 || n_kv_heads < 1 || max_blocks < 1 || max_blocks > kMaxBlocks) return PI_E_SHAPE;
  if ((int64_t)n_seqs * n_kv_heads > kMaxInt) return PI_E_SHAPE;
  if (!al4(table) || !al4(score) || !al4(lens) || !al4(table_out) || !al4(score_out) || !al4(lens_out))
    return PI_E_ALIGN;
  if (recent < 1 || recent > keep) return PI_E_RANGE;
  const size_t n = (size_t)n_seqs * n_kv_heads * max_blocks * 4, m = (size_t)n_seqs * 4;
  const bool in_place = table_out == table && score_out == score;
  if (in_place && max_blocks > PI_KV_EVICT_IN_PLACE) return PI_E_RANGE;
  const struct { const void* p; size_t n; } in[3] = {{table, n}, {score, n}, {lens, m}},
                                            out[3] = {{table_out, n}, {score_out, n}, {lens_out, m}};
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < 3; ++j) {
      const bool own = in_place && i == j && i < 2;
      if (!own && overlap(in[i].p, in[i].n, out[j].p, out[j].n)) return PI_E_RANGE;
      if (i < j && overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return PI_E_RANGE;
    }
  pi::EvictArgs a;
  a.table = table;
  a.score = score;
  a.lens = lens;
  a.n_seqs = n_seqs;
  a.hk = n_kv_heads;
  a.max_blocks = max_blocks;
  a.keep = keep;
  a.recent = recent;
  a.table_out = table_out;
  a.score_out = score_out;
  a.lens_out = lens_out;
  if (pi::kv_evict_threads(a) > pi::kMaxThreads) return PI_E_SHAPE;
  const hipError_t e = pi::launch_kv_evict(a, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? PI_OK : pi::hip_failed(e);
}

}  // extern "C"
