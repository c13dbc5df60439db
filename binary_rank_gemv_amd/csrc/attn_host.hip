// C ABI of the operators between the projections: argument validation and
// dispatch.  No allocation, no synchronisation.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <string>

#include "attn_launch.h"

namespace {

thread_local std::string g_last_error;

lb_status fail(lb_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

lb_status done(hipError_t e, const char* name) {
  if (e == hipSuccess) return LB_OK;
  return fail(LB_ERR_HIP, "%s launch: %s (%d)", name, hipGetErrorString(e), (int)e);
}

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMaxTokens = 1 << 21;
constexpr int kMaxHeads = 1 << 10;
constexpr int64_t kMaxStride = 1ll << 40;
constexpr int64_t kMaxGroups = 1 << 22;  // workgroups of 512 threads: a grid holds fewer than 2^32
constexpr int64_t kMaxRows = 1 << 30;

#define LB_TRY(expr)                   \
  do {                                 \
    const lb_status st_ = (expr);      \
    if (st_ != LB_OK) return st_;      \
  } while (0)

lb_status check_type(const char* name, int dtype) {
  if (dtype != LB_F16 && dtype != LB_BF16) return fail(LB_ERR_INVALID_ARG, "%s: bad dtype %d", name, dtype);
  return LB_OK;
}

lb_status check_tokens(const char* name, int64_t tokens) {
  if (tokens < 0) return fail(LB_ERR_INVALID_ARG, "%s: tokens=%lld must not be negative", name, (long long)tokens);
  if (tokens > kMaxTokens)
    return fail(LB_ERR_UNSUPPORTED, "%s: %lld tokens exceed %lld", name, (long long)tokens, (long long)kMaxTokens);
  return LB_OK;
}

lb_status check_heads_count(const char* name, const char* what, int heads) {
  if (heads < 1) return fail(LB_ERR_INVALID_ARG, "%s: %s has %d heads", name, what, heads);
  if (heads > kMaxHeads) return fail(LB_ERR_UNSUPPORTED, "%s: %d heads of %s exceed %d", name, heads, what, kMaxHeads);
  return LB_OK;
}

// Rows of heads; of an output, rows that do not overlap.
lb_status check_heads(const char* name, const char* what, const lb_heads* h, int64_t tokens, int dim, bool output) {
  if (!h) return fail(LB_ERR_INVALID_ARG, "%s: %s is NULL", name, what);
  LB_TRY(check_heads_count(name, what, h->heads));
  if (tokens == 0) return LB_OK;
  if (!h->p) return fail(LB_ERR_INVALID_ARG, "%s: %s is NULL", name, what);
  if (!aligned(h->p, 2)) return fail(LB_ERR_INVALID_ARG, "%s: %s must be 2-byte aligned", name, what);
  if (h->token_stride < 0 || h->head_stride < 0) return fail(LB_ERR_INVALID_ARG, "%s: negative stride of %s", name, what);
  if (h->token_stride > kMaxStride || h->head_stride > kMaxStride)
    return fail(LB_ERR_UNSUPPORTED, "%s: a stride of %s is too large", name, what);
  if (output) {
    const bool by_token = (h->heads == 1 || h->head_stride >= dim) &&
                          (tokens == 1 || h->token_stride >= (h->heads - 1) * h->head_stride + dim);
    const bool by_head = (tokens == 1 || h->token_stride >= dim) &&
                         (h->heads == 1 || h->head_stride >= (tokens - 1) * h->token_stride + dim);
    if (!by_token && !by_head) return fail(LB_ERR_INVALID_ARG, "%s: rows of %s overlap", name, what);
  }
  return LB_OK;
}

// Whether two tensors of heads have the same strides, where more than one token or head uses them.
bool same_strides(const lb_heads* a, const lb_heads* b, int64_t tokens) {
  return (tokens == 1 || a->token_stride == b->token_stride) && (a->heads == 1 || a->head_stride == b->head_stride);
}

// An output beside its input: as many heads, and in place only with the same strides.
lb_status check_pair(const char* name, const char* what, const lb_heads* in, const char* out_what, const lb_heads* out,
                     int64_t tokens, int dim) {
  LB_TRY(check_heads(name, what, in, tokens, dim, false));
  LB_TRY(check_heads(name, out_what, out, tokens, dim, true));
  if (in->heads != out->heads)
    return fail(LB_ERR_INVALID_ARG, "%s: %s has %d heads, %s %d", name, what, in->heads, out_what, out->heads);
  if (tokens > 0 && in->p == out->p && !same_strides(in, out, tokens))
    return fail(LB_ERR_INVALID_ARG, "%s: %s in place needs the same strides", name, out_what);
  return LB_OK;
}

lb_status check_rope(const char* name, const lb_rope* r, int64_t tokens, int dim) {
  if (!r) return fail(LB_ERR_INVALID_ARG, "%s: rope is NULL", name);
  if (r->rot < 0 || r->rot > dim || r->rot % 2)
    return fail(LB_ERR_INVALID_ARG, "%s: rot=%d must be even and 0 to %d", name, r->rot, dim);
  if (!(r->eps >= 0.0f) || !isfinite(r->eps)) return fail(LB_ERR_INVALID_ARG, "%s: eps must be >= 0 and finite", name);
  if (tokens == 0) return LB_OK;
  if (r->rot > 0 && (!r->positions || !aligned(r->positions, 4)))
    return fail(LB_ERR_INVALID_ARG, "%s: positions must be given, 4-byte aligned", name);
  if (r->rot > 0 && (!r->inv_freq || !aligned(r->inv_freq, 4)))
    return fail(LB_ERR_INVALID_ARG, "%s: inv_freq must be given, 4-byte aligned", name);
  if (!aligned(r->q_weight, 2) || !aligned(r->k_weight, 2))
    return fail(LB_ERR_INVALID_ARG, "%s: a weight must be 2-byte aligned", name);
  return LB_OK;
}

lb_status check_dim(const char* name, int dim) {
  if (dim < 2 || dim % 2) return fail(LB_ERR_INVALID_ARG, "%s: dim=%d must be even and positive", name, dim);
  if (dim > LB_HEAD_MAX_DIM) return fail(LB_ERR_UNSUPPORTED, "%s: dim=%d exceeds %d", name, dim, LB_HEAD_MAX_DIM);
  return LB_OK;
}

lb_status check_cache(const char* name, const lb_cache* c) {
  if (!c) return fail(LB_ERR_INVALID_ARG, "%s: cache is NULL", name);
  LB_TRY(check_type(name, c->dtype));
  LB_TRY(check_dim(name, c->dim));
  if (c->dim % 8) return fail(LB_ERR_INVALID_ARG, "%s: the cache's dim=%d must be a multiple of 8", name, c->dim);
  LB_TRY(check_heads_count(name, "cache", c->heads));
  if (c->pages < 1) return fail(LB_ERR_INVALID_ARG, "%s: the cache has %d pages", name, c->pages);
  if (c->page_size < 8 || c->page_size > 65536 || (c->page_size & (c->page_size - 1)))
    return fail(LB_ERR_INVALID_ARG, "%s: page_size=%d must be a power of two from 8 to 65536", name, c->page_size);
  if (!c->k || !c->v || !aligned(c->k, 16) || !aligned(c->v, 16))
    return fail(LB_ERR_INVALID_ARG, "%s: k and v must be given, 16-byte aligned", name);
  if (c->page_stride % 8 || c->head_stride % 8 || c->slot_stride % 8)
    return fail(LB_ERR_INVALID_ARG, "%s: the cache's strides must be multiples of 8", name);
  if (c->page_stride < 0 || c->head_stride < 0 || c->slot_stride < c->dim)
    return fail(LB_ERR_INVALID_ARG, "%s: slots of the cache overlap", name);
  if (c->slot_stride > (1 << 24) || c->head_stride > kMaxStride || c->page_stride > kMaxStride)
    return fail(LB_ERR_UNSUPPORTED, "%s: a stride of the cache is too large", name);
  const int64_t slots = (c->page_size - 1) * c->slot_stride, heads = (c->heads - 1) * c->head_stride;
  const bool apart = c->heads == 1 || c->head_stride >= slots + c->dim ||
                     (c->head_stride >= c->dim && c->slot_stride >= heads + c->dim);
  if (!apart || (c->pages > 1 && c->page_stride < c->dim))
    return fail(LB_ERR_INVALID_ARG, "%s: rows of the cache overlap", name);
  return LB_OK;
}

lb_status check_batch(const char* name, const lb_cache* c, const lb_cache_batch* b) {
  if (!b) return fail(LB_ERR_INVALID_ARG, "%s: batch is NULL", name);
  if (b->seqs < 1 || b->columns < 1)
    return fail(LB_ERR_INVALID_ARG, "%s: %d sequences of %d columns", name, b->seqs, b->columns);
  if (b->seqs >= (1 << 16)) return fail(LB_ERR_UNSUPPORTED, "%s: %d sequences are too many", name, b->seqs);
  if (b->columns > (1 << 24) || (int64_t)b->columns * c->page_size >= (1 << 30))
    return fail(LB_ERR_UNSUPPORTED, "%s: %d columns of %d slots are too many", name, b->columns, c->page_size);
  if (!b->starts || !b->lens || !b->table || !aligned(b->starts, 4) || !aligned(b->lens, 4) || !aligned(b->table, 4))
    return fail(LB_ERR_INVALID_ARG, "%s: starts, lens and table must be given, 4-byte aligned", name);
  if (b->seqs > 1 && b->table_stride < b->columns)
    return fail(LB_ERR_INVALID_ARG, "%s: row stride %lld of the table is smaller than %d", name, (long long)b->table_stride,
                b->columns);
  if (b->table_stride > kMaxStride) return fail(LB_ERR_UNSUPPORTED, "%s: the table's row stride is too large", name);
  return LB_OK;
}

LbPages pages_of(const lb_cache* c, const lb_cache_batch* b) {
  LbPages p = {};
  p.k = (char*)c->k;
  p.v = (char*)c->v;
  p.page = 2 * c->page_stride;
  p.head = 2 * c->head_stride;
  p.slot = 2 * c->slot_stride;
  p.pages = c->pages;
  p.shift = __builtin_ctz(c->page_size);
  p.starts = b->starts;
  p.lens = b->lens;
  p.table = b->table;
  p.table_stride = b->table_stride;
  p.seqs = b->seqs;
  p.columns = b->columns;
  return p;
}

template <typename A>
void set_heads(A& a, int i, const lb_heads* in, const lb_heads* out) {
  a.x[i] = in->p; a.xt[i] = in->token_stride; a.xh[i] = in->head_stride;
  a.heads[i] = in->heads;
  if (out) {
    a.y[i] = out->p; a.yt[i] = out->token_stride; a.yh[i] = out->head_stride;
  }
}

template <typename A>
void set_rope(A& a, const lb_rope* r) {
  a.positions = r->positions;
  a.inv_freq = r->inv_freq;
  a.rot = r->rot;
  a.interleaved = r->interleaved != 0;
  a.weight[0] = r->q_weight;
  a.weight[1] = r->k_weight;
  a.eps = r->eps;
}

}  // namespace

extern "C" {

lb_status littlebit_rope_fwd(const lb_heads* q, const lb_heads* k, const lb_rope* rope, int dtype, int64_t tokens,
                             int32_t dim, const lb_heads* q_out, const lb_heads* k_out, void* stream) {
  const char* name = "littlebit_rope_fwd";
  LB_TRY(check_type(name, dtype));
  LB_TRY(check_dim(name, dim));
  LB_TRY(check_tokens(name, tokens));
  LB_TRY(check_rope(name, rope, tokens, dim));
  if (!q && !k) return fail(LB_ERR_INVALID_ARG, "%s: neither q nor k is given", name);
  if (!q != !q_out || !k != !k_out) return fail(LB_ERR_INVALID_ARG, "%s: q and q_out, k and k_out go together", name);
  if (q) LB_TRY(check_pair(name, "q", q, "q_out", q_out, tokens, dim));
  if (k) LB_TRY(check_pair(name, "k", k, "k_out", k_out, tokens, dim));
  if (tokens == 0) return LB_OK;
  LbRopeArgs a = {};
  if (q) set_heads(a, 0, q, q_out);
  if (k) set_heads(a, 1, k, k_out);
  set_rope(a, rope);
  a.turn = 1.0f;
  a.tokens = tokens;
  a.dim = dim;
  return done(lb_launch_rope(a, dtype, (hipStream_t)stream), name);
}

size_t littlebit_rope_bwd_workspace_bytes(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t dim) {
  if (tokens < 1 || tokens > kMaxTokens || heads < 0 || heads > kMaxHeads || kv_heads < 0 || kv_heads > kMaxHeads ||
      dim < 2 || dim > LB_HEAD_MAX_DIM)
    return 0;
  int groups[2];
  lb_rope_bwd_groups(tokens, heads, kv_heads, dim, groups);
  return (size_t)(groups[0] + groups[1]) * dim * sizeof(float);
}

lb_status littlebit_rope_bwd(const lb_heads* dq, const lb_heads* dk, const lb_heads* q, const lb_heads* k,
                             const lb_rope* rope, int dtype, int64_t tokens, int32_t dim, const lb_heads* dq_in,
                             const lb_heads* dk_in, float* dq_weight, float* dk_weight, void* ws, size_t ws_bytes,
                             void* stream) {
  const char* name = "littlebit_rope_bwd";
  LB_TRY(check_type(name, dtype));
  LB_TRY(check_dim(name, dim));
  LB_TRY(check_tokens(name, tokens));
  LB_TRY(check_rope(name, rope, tokens, dim));
  if (!dq && !dk) return fail(LB_ERR_INVALID_ARG, "%s: neither dq nor dk is given", name);
  LbRopeBwdArgs a = {};
  const lb_heads* dy[2] = {dq, dk};
  const lb_heads* x[2] = {q, k};
  const lb_heads* dx[2] = {dq_in, dk_in};
  float* dw[2] = {dq_weight, dk_weight};
  const void* weight[2] = {rope->q_weight, rope->k_weight};
  static const char* const names[2][3] = {{"dq", "q", "dq_in"}, {"dk", "k", "dk_in"}};
  for (int i = 0; i < 2; ++i) {
    if (!dy[i]) {
      if (dx[i] || dw[i]) return fail(LB_ERR_INVALID_ARG, "%s: %s and what goes with it are given together", name, names[i][0]);
      continue;
    }
    LB_TRY(check_pair(name, names[i][0], dy[i], names[i][2], dx[i], tokens, dim));
    if (!weight[i] != !dw[i]) return fail(LB_ERR_INVALID_ARG, "%s: a weight and its gradient go together", name);
    if (!aligned(dw[i], 4)) return fail(LB_ERR_INVALID_ARG, "%s: a weight's gradient must be 4-byte aligned", name);
    if (weight[i]) {
      LB_TRY(check_heads(name, names[i][1], x[i], tokens, dim, false));
      if (x[i]->heads != dy[i]->heads)
        return fail(LB_ERR_INVALID_ARG, "%s: %s has %d heads, %s %d", name, names[i][1], x[i]->heads, names[i][0], dy[i]->heads);
      if (tokens > 0 && x[i]->p == dx[i]->p && !same_strides(x[i], dx[i], tokens))
        return fail(LB_ERR_INVALID_ARG, "%s: %s in place needs the same strides", name, names[i][2]);
      a.x[i] = x[i]->p; a.xt[i] = x[i]->token_stride; a.xh[i] = x[i]->head_stride;
      a.weight[i] = weight[i];
      a.dweight[i] = dw[i];
    }
    a.dy[i] = dy[i]->p; a.dyt[i] = dy[i]->token_stride; a.dyh[i] = dy[i]->head_stride;
    a.dx[i] = dx[i]->p; a.dxt[i] = dx[i]->token_stride; a.dxh[i] = dx[i]->head_stride;
    a.heads[i] = dy[i]->heads;
  }
  if (tokens > 0 && (a.weight[0] || a.weight[1])) {
    const size_t need = littlebit_rope_bwd_workspace_bytes(tokens, a.heads[0], a.heads[1], dim);
    if (!ws || !aligned(ws, 16)) return fail(LB_ERR_WORKSPACE, "%s: workspace must be given, 16-byte aligned", name);
    if (ws_bytes < need) return fail(LB_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", name, ws_bytes, need);
  }
  if (tokens == 0 && !dq_weight && !dk_weight) return LB_OK;
  a.positions = rope->positions;
  a.inv_freq = rope->inv_freq;
  a.rot = rope->rot;
  a.interleaved = rope->interleaved != 0;
  a.eps = rope->eps;
  a.partial = (float*)ws;
  a.tokens = tokens;
  a.dim = dim;
  lb_rope_bwd_groups(tokens, a.heads[0], a.heads[1], dim, a.groups);
  return done(lb_launch_rope_bwd(a, dtype, (hipStream_t)stream), name);
}

lb_status littlebit_cache_append(const lb_cache* cache, const lb_cache_batch* batch, int64_t tokens, const lb_heads* k,
                                 const lb_heads* v, const lb_heads* q, const lb_rope* rope, const lb_heads* q_out,
                                 void* stream) {
  const char* name = "littlebit_cache_append";
  LB_TRY(check_cache(name, cache));
  LB_TRY(check_batch(name, cache, batch));
  LB_TRY(check_tokens(name, tokens));
  LB_TRY(check_heads(name, "k", k, tokens, cache->dim, false));
  LB_TRY(check_heads(name, "v", v, tokens, cache->dim, false));
  if (k->heads != cache->heads || v->heads != cache->heads)
    return fail(LB_ERR_INVALID_ARG, "%s: k has %d heads, v %d, the cache %d", name, k->heads, v->heads, cache->heads);
  if (!q != !q_out) return fail(LB_ERR_INVALID_ARG, "%s: q and q_out go together", name);
  if (q) LB_TRY(check_pair(name, "q", q, "q_out", q_out, tokens, cache->dim));
  if (rope) LB_TRY(check_rope(name, rope, tokens, cache->dim));
  if (tokens == 0) return LB_OK;
  LbRopeArgs a = {};
  if (q) set_heads(a, 0, q, q_out);
  set_heads(a, 1, k, nullptr);
  set_heads(a, 2, v, nullptr);
  if (rope) set_rope(a, rope);
  a.turn = 1.0f;
  a.tokens = tokens;
  a.dim = cache->dim;
  a.append = true;
  a.pages = pages_of(cache, batch);
  return done(lb_launch_rope(a, cache->dtype, (hipStream_t)stream), name);
}

size_t littlebit_cache_attention_workspace_bytes(const lb_cache* cache, const lb_cache_batch* batch, int64_t tokens,
                                                 int32_t heads) {
  if (!cache || !batch || tokens < 1 || tokens > kMaxTokens || cache->heads < 1 || cache->heads > kMaxHeads || heads < 1 ||
      heads > kMaxHeads || heads % cache->heads || batch->seqs < 1 || batch->seqs >= (1 << 16) || batch->columns < 1 ||
      cache->page_size < 1 || cache->dim < 2 || cache->dim > LB_HEAD_MAX_DIM)
    return 0;
  return lb_attn_workspace(lb_attn_plan(tokens, batch->seqs, (int64_t)batch->columns * cache->page_size, heads, cache->heads, cache->dim), tokens, heads, cache->heads,
                           cache->dim);
}

lb_status littlebit_cache_attention_fwd(const lb_cache* cache, const lb_cache_batch* batch, int64_t tokens,
                                        const lb_heads* q, const int64_t* tree, float scale, const lb_heads* out,
                                        float* lse, void* ws, size_t ws_bytes, void* stream) {
  const char* name = "littlebit_cache_attention_fwd";
  LB_TRY(check_cache(name, cache));
  LB_TRY(check_batch(name, cache, batch));
  LB_TRY(check_tokens(name, tokens));
  LB_TRY(check_pair(name, "q", q, "out", out, tokens, cache->dim));
  if (q->heads % cache->heads)
    return fail(LB_ERR_INVALID_ARG, "%s: %d heads are no multiple of the cache's %d", name, q->heads, cache->heads);
  if (!(fabsf(scale) <= 1e30f)) return fail(LB_ERR_INVALID_ARG, "%s: scale must be finite, at most 1e30", name);
  if (!aligned(tree, 8)) return fail(LB_ERR_INVALID_ARG, "%s: tree must be 8-byte aligned", name);
  if (!aligned(lse, 4)) return fail(LB_ERR_INVALID_ARG, "%s: lse must be 4-byte aligned", name);
  if (tokens == 0) return LB_OK;
  if (q->p == out->p) return fail(LB_ERR_INVALID_ARG, "%s: out must not be q", name);
  const LbAttnPlan plan = lb_attn_plan(tokens, batch->seqs, (int64_t)batch->columns * cache->page_size, q->heads, cache->heads, cache->dim);
  if (plan.grid > kMaxGroups || tokens * q->heads > kMaxRows)
    return fail(LB_ERR_UNSUPPORTED, "%s: %lld tokens of %d heads are too many for one call", name, (long long)tokens, q->heads);
  const size_t need = lb_attn_workspace(plan, tokens, q->heads, cache->heads, cache->dim);
  if (need > 0 && (!ws || !aligned(ws, 16)))
    return fail(LB_ERR_WORKSPACE, "%s: workspace must be given, 16-byte aligned", name);
  if (ws_bytes < need) return fail(LB_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", name, ws_bytes, need);
  LbAttnArgs a = {};
  a.pages = pages_of(cache, batch);
  a.q = q->p; a.qt = q->token_stride; a.qh = q->head_stride;
  a.out = out->p; a.ot = out->token_stride; a.oh = out->head_stride;
  a.tree = tree;
  a.lse = lse;
  a.partial = (float*)ws;
  if (plan.groups) a.groups = (int*)((char*)ws + lb_attn_groups_at(plan, tokens, q->heads, cache->heads, cache->dim));
  a.slots = plan.slots;
  a.tokens = tokens;
  a.heads = q->heads;
  a.kv_heads = cache->heads;
  a.group = q->heads / cache->heads;
  a.dim = cache->dim;
  a.scale = (float)(fabs((double)scale) * 1.4426950408889634074);
  a.sign = scale < 0.0f ? 0x80008000u : 0u;
  a.keep = a.scale > 0.0f ? ~0u : 0u;
  if (a.keep == 0) a.scale = 1.0f;
  a.round = plan.round;
  a.target = plan.target;
  a.least = plan.least;
  return done(lb_launch_attn(a, plan, cache->dtype, (hipStream_t)stream), name);
}

lb_status littlebit_cache_accept(const lb_cache* cache, const lb_cache_batch* batch, const int32_t* path, int32_t columns,
                                 void* stream) {
  const char* name = "littlebit_cache_accept";
  LB_TRY(check_cache(name, cache));
  LB_TRY(check_batch(name, cache, batch));
  if (columns < 1 || columns > LB_TREE_MAX)
    return fail(LB_ERR_INVALID_ARG, "%s: a path has %d columns, 1 to %d are possible", name, columns, LB_TREE_MAX);
  if (!path || !aligned(path, 4)) return fail(LB_ERR_INVALID_ARG, "%s: path must be given, 4-byte aligned", name);
  return done(lb_launch_accept(pages_of(cache, batch), cache->heads, cache->dim, path, columns, (hipStream_t)stream), name);
}

const char* littlebit_attn_last_error(void) { return g_last_error.c_str(); }

}  // extern "C"
