// C ABI of the dense operators around the LittleBit layers: argument
// validation and dispatch.  No allocation, no synchronisation.
#include <stdarg.h>
#include <stdio.h>

#include <string>

#include "littlebit_head.h"
#include "head_launch.h"

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
inline int dtype_bytes(int dtype) { return dtype == LB_F32 ? 4 : 2; }

constexpr int64_t kMaxRows = 1 << 21;  // a grid holds fewer than 2^32 threads
constexpr int64_t kMaxStride = 1ll << 40;
constexpr int kMaxCodes = 131071;      // 128^2 n < 2^31
constexpr int64_t kMaxVocab = 1ll << 30;

lb_status check_rows(const char* name, int64_t rows, int64_t n, int64_t max_n) {
  if (rows < 0) return fail(LB_ERR_INVALID_ARG, "%s: rows=%lld must not be negative", name, (long long)rows);
  if (n < 1) return fail(LB_ERR_INVALID_ARG, "%s: row length %lld must be >= 1", name, (long long)n);
  if (rows > kMaxRows) return fail(LB_ERR_UNSUPPORTED, "%s: %lld rows exceed %lld", name, (long long)rows, (long long)kMaxRows);
  if (n > max_n) return fail(LB_ERR_UNSUPPORTED, "%s: row length %lld exceeds %lld", name, (long long)n, (long long)max_n);
  return LB_OK;
}

// One matrix argument: present, aligned to its elements, rows of n.
lb_status check_matrix(const char* name, const char* what, const void* p, int64_t ld, int64_t n, int bytes) {
  if (!p) return fail(LB_ERR_INVALID_ARG, "%s: %s is NULL", name, what);
  if (!aligned(p, bytes)) return fail(LB_ERR_INVALID_ARG, "%s: %s must be %d-byte aligned", name, what, bytes);
  if (ld < n) return fail(LB_ERR_INVALID_ARG, "%s: row stride %lld of %s is smaller than %lld", name, (long long)ld, what, (long long)n);
  if (ld > kMaxStride) return fail(LB_ERR_UNSUPPORTED, "%s: row stride %lld of %s is too large", name, (long long)ld, what);
  return LB_OK;
}

lb_status check_vector(const char* name, const char* what, const void* p, int bytes) {
  if (!p) return fail(LB_ERR_INVALID_ARG, "%s: %s is NULL", name, what);
  if (!aligned(p, bytes)) return fail(LB_ERR_INVALID_ARG, "%s: %s must be %d-byte aligned", name, what, bytes);
  return LB_OK;
}

lb_status check_workspace(const char* name, const void* ws, size_t have, size_t need) {
  if (need == 0) return LB_OK;
  if (!ws) return fail(LB_ERR_WORKSPACE, "%s: workspace is NULL", name);
  if (!aligned(ws, 16)) return fail(LB_ERR_WORKSPACE, "%s: workspace must be 16-byte aligned", name);
  if (have < need) return fail(LB_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", name, have, need);
  return LB_OK;
}

// Whether `dst` is a matrix that shares its first element with `src` but not
// its rows (an in-place call with another stride would overwrite unread rows).
inline bool skewed(const void* dst, int64_t ldd, const void* src, int64_t lds) { return dst == src && ldd != lds; }

#define LB_TRY(expr)                   \
  do {                                 \
    const lb_status st_ = (expr);      \
    if (st_ != LB_OK) return st_;      \
  } while (0)

}  // namespace

extern "C" {

lb_status littlebit_rmsnorm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                                int dtype, int64_t rows, int64_t n, float eps, void* hidden, int64_t ldh, void* y,
                                int64_t ldy, int8_t* q, int64_t ldq, float* scale, void* stream) {
  const char* name = "littlebit_rmsnorm_fwd";
  if (dtype != LB_F16 && dtype != LB_BF16) return fail(LB_ERR_INVALID_ARG, "%s: bad dtype %d", name, dtype);
  LB_TRY(check_rows(name, rows, n, LB_NORM_MAX_N));
  if (!(eps >= 0.0f)) return fail(LB_ERR_INVALID_ARG, "%s: eps must be >= 0", name);
  if (rows == 0) return LB_OK;
  if (!y && !q) return fail(LB_ERR_INVALID_ARG, "%s: neither y nor q is given", name);
  if (!q != !scale) return fail(LB_ERR_INVALID_ARG, "%s: q and scale go together", name);
  if (!residual != !hidden) return fail(LB_ERR_INVALID_ARG, "%s: residual and hidden go together", name);
  LB_TRY(check_matrix(name, "x", x, ldx, n, 2));
  LB_TRY(check_vector(name, "weight", weight, 2));
  if (residual) {
    LB_TRY(check_matrix(name, "residual", residual, ldr, n, 2));
    LB_TRY(check_matrix(name, "hidden", hidden, ldh, n, 2));
    if (skewed(hidden, ldh, x, ldx) || skewed(hidden, ldh, residual, ldr))
      return fail(LB_ERR_INVALID_ARG, "%s: hidden in place needs the same row stride", name);
  }
  if (y) LB_TRY(check_matrix(name, "y", y, ldy, n, 2));
  if (q) {
    LB_TRY(check_matrix(name, "q", q, ldq, n, 1));
    LB_TRY(check_vector(name, "scale", scale, 4));
  }
  LbNormArgs a = {};
  a.x = x; a.ldx = ldx;
  a.residual = residual; a.ldr = ldr;
  a.weight = weight;
  a.hidden = hidden; a.ldh = ldh;
  a.y = y; a.ldy = ldy;
  a.q = q; a.ldq = ldq;
  a.scale = scale;
  a.rows = rows; a.n = (int)n; a.eps = eps;
  return done(lb_launch_norm(a, dtype, (hipStream_t)stream), name);
}

size_t littlebit_rmsnorm_bwd_workspace_bytes(int64_t rows, int64_t n) {
  if (rows < 1 || n < 1 || n > LB_NORM_MAX_N) return 0;
  return (size_t)lb_norm_bwd_groups(rows, n) * n * sizeof(float);
}

lb_status littlebit_rmsnorm_bwd(const void* dy, int64_t lddy, const void* dhidden, int64_t lddh, const void* hidden,
                                int64_t ldh, const void* weight, int dtype, int64_t rows, int64_t n, float eps,
                                void* dx, int64_t lddx, float* dweight, void* ws, size_t ws_bytes, void* stream) {
  const char* name = "littlebit_rmsnorm_bwd";
  if (dtype != LB_F16 && dtype != LB_BF16) return fail(LB_ERR_INVALID_ARG, "%s: bad dtype %d", name, dtype);
  LB_TRY(check_rows(name, rows, n, LB_NORM_MAX_N));
  if (!(eps >= 0.0f)) return fail(LB_ERR_INVALID_ARG, "%s: eps must be >= 0", name);
  LB_TRY(check_vector(name, "dweight", dweight, 4));
  LbNormBwdArgs a = {};
  if (rows > 0) {
    LB_TRY(check_matrix(name, "dy", dy, lddy, n, 2));
    if (dhidden) LB_TRY(check_matrix(name, "dhidden", dhidden, lddh, n, 2));
    LB_TRY(check_matrix(name, "hidden", hidden, ldh, n, 2));
    LB_TRY(check_vector(name, "weight", weight, 2));
    LB_TRY(check_matrix(name, "dx", dx, lddx, n, 2));
    if (skewed(dx, lddx, dy, lddy) || skewed(dx, lddx, dhidden, lddh) || skewed(dx, lddx, hidden, ldh))
      return fail(LB_ERR_INVALID_ARG, "%s: dx in place needs the same row stride", name);
    LB_TRY(check_workspace(name, ws, ws_bytes, littlebit_rmsnorm_bwd_workspace_bytes(rows, n)));
    a.groups = lb_norm_bwd_groups(rows, n);
  }
  a.dy = dy; a.lddy = lddy;
  a.dhidden = dhidden; a.lddh = lddh;
  a.hidden = hidden; a.ldh = ldh;
  a.weight = weight;
  a.dx = dx; a.lddx = lddx;
  a.dweight = dweight;
  a.partial = static_cast<float*>(ws);
  a.rows = rows; a.n = (int)n; a.eps = eps;
  return done(lb_launch_norm_bwd(a, dtype, (hipStream_t)stream), name);
}

lb_status littlebit_q8_quantize(const void* x, int64_t ldx, int dtype, int64_t rows, int64_t n, int8_t* q, int64_t ldq,
                                float* scale, void* stream) {
  const char* name = "littlebit_q8_quantize";
  if (dtype != LB_F32 && dtype != LB_F16 && dtype != LB_BF16)
    return fail(LB_ERR_INVALID_ARG, "%s: bad dtype %d", name, dtype);
  LB_TRY(check_rows(name, rows, n, LB_NORM_MAX_N));
  if (rows == 0) return LB_OK;
  LB_TRY(check_matrix(name, "x", x, ldx, n, dtype_bytes(dtype)));
  LB_TRY(check_matrix(name, "q", q, ldq, n, 1));
  LB_TRY(check_vector(name, "scale", scale, 4));
  LbNormArgs a = {};
  a.x = x; a.ldx = ldx;
  a.q = q; a.ldq = ldq;
  a.scale = scale;
  a.rows = rows; a.n = (int)n;
  return done(lb_launch_q8_quantize(a, dtype, (hipStream_t)stream), name);
}

lb_status littlebit_q8_linear_fwd(const int8_t* xq, int64_t ldx, const float* xscale, const int8_t* wq, int64_t ldw,
                                  const float* wscale, int64_t batch, int64_t m, int64_t n, void* y, int64_t ldy,
                                  int y_dtype, void* stream) {
  const char* name = "littlebit_q8_linear_fwd";
  if (y_dtype != LB_F32 && y_dtype != LB_F16 && y_dtype != LB_BF16)
    return fail(LB_ERR_INVALID_ARG, "%s: bad y_dtype %d", name, y_dtype);
  LB_TRY(check_rows(name, batch, n, kMaxCodes));
  if (m < 1) return fail(LB_ERR_INVALID_ARG, "%s: m=%lld must be >= 1", name, (long long)m);
  if (m > (1 << 24)) return fail(LB_ERR_UNSUPPORTED, "%s: m=%lld exceeds %d", name, (long long)m, 1 << 24);
  if (batch * m > (1ll << 38))
    return fail(LB_ERR_UNSUPPORTED, "%s: %lld x %lld outputs are too many for one call", name, (long long)batch, (long long)m);
  if (batch == 0) return LB_OK;
  LB_TRY(check_matrix(name, "xq", xq, ldx, n, 1));
  LB_TRY(check_matrix(name, "wq", wq, ldw, n, 1));
  LB_TRY(check_vector(name, "xscale", xscale, 4));
  LB_TRY(check_vector(name, "wscale", wscale, 4));
  LB_TRY(check_matrix(name, "y", y, ldy, m, dtype_bytes(y_dtype)));
  LbQ8LinearArgs a = {};
  a.xq = xq; a.ldx = ldx;
  a.xscale = xscale;
  a.wq = wq; a.ldw = ldw;
  a.wscale = wscale;
  a.batch = batch; a.m = (int)m; a.n = (int)n;
  a.y = y; a.ldy = ldy;
  return done(lb_launch_q8_linear(a, y_dtype, (hipStream_t)stream), name);
}

size_t littlebit_logprobs_workspace_bytes(int64_t rows, int64_t vocab, int dtype, int top) {
  if (dtype != LB_F32 && dtype != LB_F16 && dtype != LB_BF16) return 0;
  if (rows < 1 || rows > kMaxRows || vocab < 1 || vocab > kMaxVocab || top < 0 || top > LB_TOP_MAX) return 0;
  int span = 0;
  return lb_logprobs_partial_bytes(rows, lb_logprobs_splits(rows, vocab, &span), top);
}

lb_status littlebit_logprobs_fwd(const void* logits, int64_t ld, int dtype, int64_t rows, int64_t vocab,
                                 const int64_t* targets, float* logprob, float* entropy, float* lse, int top,
                                 float* top_logprob, int64_t* top_index, void* ws, size_t ws_bytes, void* stream) {
  const char* name = "littlebit_logprobs_fwd";
  if (dtype != LB_F32 && dtype != LB_F16 && dtype != LB_BF16)
    return fail(LB_ERR_INVALID_ARG, "%s: bad dtype %d", name, dtype);
  LB_TRY(check_rows(name, rows, vocab, kMaxVocab));
  if (top < 0 || top > vocab) return fail(LB_ERR_INVALID_ARG, "%s: top=%d must be 0 to vocab", name, top);
  if (top > LB_TOP_MAX) return fail(LB_ERR_UNSUPPORTED, "%s: top=%d exceeds %d", name, top, LB_TOP_MAX);
  if (rows == 0) return LB_OK;
  LB_TRY(check_matrix(name, "logits", logits, ld, vocab, dtype_bytes(dtype)));
  if (!targets != !logprob) return fail(LB_ERR_INVALID_ARG, "%s: targets and logprob go together", name);
  if (targets) {
    LB_TRY(check_vector(name, "targets", targets, 8));
    LB_TRY(check_vector(name, "logprob", logprob, 4));
  }
  if (entropy) LB_TRY(check_vector(name, "entropy", entropy, 4));
  LB_TRY(check_vector(name, "lse", lse, 4));
  if (top > 0) {
    LB_TRY(check_vector(name, "top_logprob", top_logprob, 4));
    LB_TRY(check_vector(name, "top_index", top_index, 8));
  }
  LbLogprobsArgs a = {};
  a.splits = lb_logprobs_splits(rows, vocab, &a.span);
  LB_TRY(check_workspace(name, ws, ws_bytes, lb_logprobs_partial_bytes(rows, a.splits, top)));
  a.logits = logits; a.ld = ld;
  a.targets = targets;
  a.logprob = logprob;
  a.entropy = entropy;
  a.lse = lse;
  a.top_logprob = top_logprob;
  a.top_index = top_index;
  a.ws = ws;
  a.rows = rows; a.vocab = (int)vocab; a.top = top;
  return done(lb_launch_logprobs(a, dtype, (hipStream_t)stream), name);
}

lb_status littlebit_logprobs_bwd(const void* logits, int64_t ld, int dtype, int64_t rows, int64_t vocab,
                                 const int64_t* targets, const float* lse, const float* entropy,
                                 const float* dlogprob, const float* dentropy, int top, const int64_t* top_index,
                                 const float* dtop, void* dlogits, int64_t ldd, void* stream) {
  const char* name = "littlebit_logprobs_bwd";
  if (dtype != LB_F32 && dtype != LB_F16 && dtype != LB_BF16)
    return fail(LB_ERR_INVALID_ARG, "%s: bad dtype %d", name, dtype);
  LB_TRY(check_rows(name, rows, vocab, kMaxVocab));
  if (top < 0 || top > vocab) return fail(LB_ERR_INVALID_ARG, "%s: top=%d must be 0 to vocab", name, top);
  if (top > LB_TOP_MAX) return fail(LB_ERR_UNSUPPORTED, "%s: top=%d exceeds %d", name, top, LB_TOP_MAX);
  if (rows * ((vocab + 8191) / 8192) >= (1ll << 24))
    return fail(LB_ERR_UNSUPPORTED, "%s: %lld rows of %lld are too many for one call", name, (long long)rows, (long long)vocab);
  if (rows == 0) return LB_OK;
  if (!targets != !dlogprob) return fail(LB_ERR_INVALID_ARG, "%s: targets and dlogprob go together", name);
  if (!entropy != !dentropy) return fail(LB_ERR_INVALID_ARG, "%s: entropy and dentropy go together", name);
  LB_TRY(check_matrix(name, "logits", logits, ld, vocab, dtype_bytes(dtype)));
  LB_TRY(check_matrix(name, "dlogits", dlogits, ldd, vocab, dtype_bytes(dtype)));
  if (skewed(dlogits, ldd, logits, ld))
    return fail(LB_ERR_INVALID_ARG, "%s: dlogits in place needs the same row stride", name);
  LB_TRY(check_vector(name, "lse", lse, 4));
  if (targets) {
    LB_TRY(check_vector(name, "targets", targets, 8));
    LB_TRY(check_vector(name, "dlogprob", dlogprob, 4));
  }
  if (entropy) {
    LB_TRY(check_vector(name, "entropy", entropy, 4));
    LB_TRY(check_vector(name, "dentropy", dentropy, 4));
  }
  if (top > 0) {
    LB_TRY(check_vector(name, "top_index", top_index, 8));
    LB_TRY(check_vector(name, "dtop", dtop, 4));
  }
  LbLogprobsBwdArgs a = {};
  a.logits = logits; a.ld = ld;
  a.targets = targets;
  a.lse = lse;
  a.entropy = entropy;
  a.dlogprob = dlogprob;
  a.dentropy = dentropy;
  a.top_index = top_index;
  a.dtop = dtop;
  a.dlogits = dlogits; a.ldd = ldd;
  a.rows = rows; a.vocab = (int)vocab; a.top = top;
  return done(lb_launch_logprobs_bwd(a, dtype, (hipStream_t)stream), name);
}

const char* littlebit_head_last_error(void) { return g_last_error.c_str(); }

}  // extern "C"
