/*
 * littlebit_attn.h -- C ABI of what lies between a block's projections on
 * MI355X (gfx950): the norm of each head of queries and keys with the position
 * rotation, a paged cache of keys and values, and the attention over it, of
 * single tokens, prompts and trees of drafted tokens.
 *
 * A LittleBit model replaces the linear layers of its Transformer blocks and
 * keeps the rest (trueseeker.com case, "The trace / claim to source": only
 * the Transformer blocks are quantized).  littlebit_block_fwd gives a block's
 * q, k and v and takes x_o, the attention's output: these are the operators
 * from the one to the other.  One pass over the packed weights takes up to 16
 * tokens for little more than the time of one, so drafted tokens, verified
 * together, are the way to use it; at 0.1 to 0.5 bits per weight the cache is
 * the larger read of a step over long texts.
 *
 * A library of its own (liblittlebit_attn.so).  The conventions of
 * littlebit.h hold: device pointers, caller-owned memory, nothing is
 * allocated, freed or synchronised, work is enqueued on `stream` of the
 * current device, arguments are validated before anything is enqueued, a
 * negative lb_status reports a refusal and littlebit_attn_last_error its
 * reason (thread-local).  Calls may overlap where none writes what another
 * reads; a workspace holds nothing between calls and needs no initialization,
 * but calls that run at the same time must not share one.  The structs are
 * read during the call only.
 */
#ifndef LITTLEBIT_ATTN_H
#define LITTLEBIT_ATTN_H

#include "littlebit.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bfloat16, beside lb_dtype's LB_F16 (dtype arguments are ints). */
#define LB_BF16 2

/* Largest head. */
#define LB_HEAD_MAX_DIM 256
/* Most drafted tokens of a tree. */
#define LB_TREE_MAX 64

/*
 * Rows of heads: element (t, h, d) of a tokens x heads x dim tensor lies at
 * p + t * token_stride + h * head_stride + d (elements).  Heads of a token may
 * lie anywhere (a slice of a fused projection's output), any alignment of a
 * whole element is accepted; 16 bytes are fastest.  tokens <= 2^21, heads <= 2^10.
 */
typedef struct {
  void *p;
  int64_t token_stride, head_stride;
  int32_t heads;
} lb_heads;

/*
 * Head norm and rotation.  Of each head x of dim channels
 *     y_d = x_d * weight_d / sqrt(mean_i x_i^2 + eps)      (y = x where weight is NULL)
 * and of y the first `rot` channels are turned in pairs by angle_j = position * inv_freq_j:
 *     (a, b) -> (a cos angle_j - b sin angle_j, b cos angle_j + a sin angle_j)
 * pair j being channels j and j + rot / 2, or 2 j and 2 j + 1 (interleaved).
 *   positions  int32 [tokens], any values; may be NULL where rot is 0.
 *   inv_freq   fp32 [rot / 2]; may be NULL where rot is 0.
 *   rot        even, 0 <= rot <= dim.
 *   q_weight, k_weight  [dim], of the heads' type, or NULL each.
 * Angles are formed in 64 bits and their turns taken off there, so far positions
 * keep their digits; everything else is in fp32, rounded to the type once.
 * Values of any size are normed, those whose squares fp32 does not hold (bf16) too.
 * A head of zeros needs eps > 0.
 */
typedef struct {
  const int32_t *positions;
  const float *inv_freq;
  int32_t rot, interleaved;
  const void *q_weight, *k_weight;
  float eps;
} lb_rope;

/*
 * A paged cache: page i, head h, slot s holds dim keys (values) at
 * k (v) + i * page_stride + h * head_stride + s * slot_stride.  Heads before
 * slots inside a page is the usual order; slots before heads works as well.
 *   dtype      LB_F16 or LB_BF16.
 *   page_size  slots a page, a power of two from 8 to 65536.
 *   dim        a multiple of 8 up to LB_HEAD_MAX_DIM.  k and v are 16-byte aligned and
 *              the strides multiples of 8 elements; slot_stride <= 2^24.
 */
typedef struct {
  void *k, *v;
  int64_t page_stride, head_stride, slot_stride;
  int32_t pages, heads, page_size, dim;
  int32_t dtype;
} lb_cache;

/*
 * The sequences of a call.  Sequence i has the rows starts[i] to starts[i+1] - 1
 * of the call's tokens (none, one or many), and lens[i] keys in the cache, those
 * of the call's rows, its last, among them.  Its key j lies in page table[i][j /
 * page_size], slot j % page_size.  All int32 on the device, read by the kernels:
 * one captured graph serves every content.
 *   table      seqs rows of `columns` entries, table_stride apart.  Entries past a
 *              sequence's keys may hold anything.
 * Rows that belong to no sequence (before starts[0], from starts[seqs] on) are left
 * as they are in every output.  What the tables say wrongly cannot reach memory
 * outside the tensors: an entry that names no page, or a key past the last column,
 * stands for no key (it is not attended, and nothing is written for it), and rows
 * outside of the call's tokens are not computed.  A sequence with a negative length or
 * start, or with no row of the call, has none: what it would name is left as it is.
 * starts must not fall; where they do, rows may be left out or taken twice.
 * 1 <= seqs < 2^16, columns <= 2^24, columns x page_size < 2^30.
 */
typedef struct {
  const int32_t *starts, *lens, *table;
  int64_t table_stride;
  int32_t seqs, columns;
} lb_cache_batch;

/*
 * Head norm and rotation of queries and keys, dense to dense.
 *   k, k_out   may both be NULL (queries alone); q, q_out too.
 *   q_out, k_out  may be q and k themselves (same strides); otherwise they overlap no input.
 * Channels from rot on are normed only.
 */
lb_status littlebit_rope_fwd(const lb_heads *q, const lb_heads *k, const lb_rope *rope, int dtype,
                             int64_t tokens, int32_t dim, const lb_heads *q_out,
                             const lb_heads *k_out, void *stream);

/*
 * Its backward pass: from the gradients dq, dk of q_out and k_out (any of the two
 * pairs may be NULL) those of q, k and, in fp32 [dim], of the weights.
 *   q, k       the forward's inputs; NULL (with the weight) where there is no norm.
 *   dq_in, dk_in  may be dq and dk themselves (same strides).
 *   dq_weight, dk_weight  given exactly where the weights are.  They are sums over
 *              all tokens and heads in a fixed order: the same call gives the same bits.
 *   ws         littlebit_rope_bwd_workspace_bytes bytes, 16-byte aligned; 0 without norms.
 */
size_t littlebit_rope_bwd_workspace_bytes(int64_t tokens, int32_t heads, int32_t kv_heads, int32_t dim);

lb_status littlebit_rope_bwd(const lb_heads *dq, const lb_heads *dk, const lb_heads *q,
                             const lb_heads *k, const lb_rope *rope, int dtype, int64_t tokens,
                             int32_t dim, const lb_heads *dq_in, const lb_heads *dk_in,
                             float *dq_weight, float *dk_weight, void *ws, size_t ws_bytes,
                             void *stream);

/*
 * Keys and values of the call's rows into their sequences' pages, the keys normed and
 * rotated on the way, the queries beside them.
 *   k, v       tokens x cache->heads x cache->dim, of the cache's type.
 *   q, q_out   as for littlebit_rope_fwd, or both NULL.
 *   rope       NULL: keys and queries are stored as they are.
 * Two rows of a call that fall on one slot (sequences that share the page they end in)
 * leave values of either there, piece by piece.
 */
lb_status littlebit_cache_append(const lb_cache *cache, const lb_cache_batch *batch, int64_t tokens,
                                 const lb_heads *k, const lb_heads *v, const lb_heads *q,
                                 const lb_rope *rope, const lb_heads *q_out, void *stream);

/*
 * Attention over the cache.  Row t of a sequence with n rows and len keys, head h:
 *     out = sum_j p_j v_j,  p = softmax of scale * q . k_j over the keys j that the row sees,
 * with the keys and values of head h / (q->heads / cache->heads).  It sees every key
 * before its sequence's rows (j < len - n), and of the rows' own keys
 *   tree NULL  those up to its own (j <= len - n + t);
 *   tree       int64 [tokens]: those whose bit j - (len - n) is set in the row's word, so
 *              that each row of a tree of drafts names its ancestors and itself.  A
 *              sequence has at most LB_TREE_MAX rows then; keys of later ones are not seen.
 * What a row does not see has no part in its output, NaN and infinities in it included.  An
 * infinite value that it sees is infinite there, NaN where its score is -infinity, or so low that
 * the type or fp32 may hold no more of its probability.
 * A row that sees nothing has output 0 and lse -infinity.
 *   scale      finite, 1e30 at most in size; may be negative or 0.
 *   out        as q; overlaps no input.
 *   lse        fp32 tokens x q->heads, or NULL: the logarithm of the sum of exp(scale q . k_j).
 *   ws         littlebit_cache_attention_workspace_bytes(...) bytes (may be 0, then ws may be
 *              NULL), 16-byte aligned.
 * Scores, softmax and sums are in fp32.  The matrix units take probabilities and values in one
 * type, the cache's: where sequences have more than some 80 rows x heads of a group on average, each
 * probability is rounded to it for that product, by half a step (in fp16, whose smallest step is
 * a fixed one, those below 2^-21 of a row's largest by up to 2^-32 of that one); with fewer, what
 * the rounding leaves is multiplied too.  scale q . k_j is 10^8 at most in size.  The same call
 * gives the same bits.
 * tokens x q->heads <= 2^30, fewer where the grid holds no more.
 */
size_t littlebit_cache_attention_workspace_bytes(const lb_cache *cache, const lb_cache_batch *batch,
                                                 int64_t tokens, int32_t heads);

lb_status littlebit_cache_attention_fwd(const lb_cache *cache, const lb_cache_batch *batch,
                                        int64_t tokens, const lb_heads *q, const int64_t *tree,
                                        float scale, const lb_heads *out, float *lse, void *ws,
                                        size_t ws_bytes, void *stream);

/*
 * After a tree is verified: the keys and values of its accepted rows moved together.
 * For every sequence and j < columns with path[i][j] >= 0, the keys and values of the
 * sequence's row path[i][j] are copied to where those of its row j lie; all are read before
 * any is written (of one sequence: two sequences of a call must not share pages that hold
 * their rows).  With `lens` lowered to the keys before the rows plus the accepted ones,
 * the cache is that of a text which had the accepted tokens only.
 *   path       int32 [seqs][columns], contiguous; negative entries, and those that name no
 *              row of the sequence, move nothing.  1 <= columns <= LB_TREE_MAX.
 */
lb_status littlebit_cache_accept(const lb_cache *cache, const lb_cache_batch *batch,
                                 const int32_t *path, int32_t columns, void *stream);

/* Thread-local message for the most recent failing call of this library. */
const char *littlebit_attn_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* LITTLEBIT_ATTN_H */
