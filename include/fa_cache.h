/*
 * fa_cache.h -- C ABI of the GB300 (sm_103a) library's serving operators: a
 * paged key/value cache held in 8 bits, attention over it, eviction from it by
 * accumulated attention weight, and decoding with a tree of drafted tokens
 * (attention, verification, acceptance).  Statuses, error messages, streams and
 * the bounded-wait contract are those of fa.h.
 *
 * The cache.  Keys and values live in blocks ("pages") of `page` tokens; a
 * block of one K/V head is [page, D] 8-bit values with one fp32 scale, and
 *
 *   key = stored value * k_scale[block, head]        (v alike)
 *
 * Sequence b's token j is slot j % page of block table[b, j / page].  Every
 * table entry that a sequence's tokens need must lie in [0, P); the others are
 * never read (-1 is customary).  One block serves one sequence where a call
 * writes it (fa_cache_append, fa_cache_accept, fa_cache_evict); sequences that are only read
 * may share blocks.
 *
 * A length past the table (lens[b] > M * page), a negative one, or an entry
 * outside [0, P) that a sequence needs is not followed: the tokens behind it
 * are skipped (not written; not seen by attention; not moved by eviction) and
 * fa_sync_status() then reports FA_ERR_INVALID_ARGUMENT once.  (Attention takes a
 * length past the table as M * page, its rows' positions with it.)
 *
 * Memory: every pointer is caller-owned device memory on the current device;
 * nothing is allocated, and nothing is kept after the call's kernels have run.
 * Calls are asynchronous on `stream` and can be captured into a CUDA graph;
 * lengths are read on the device, so a replayed graph follows lengths that
 * changed.  Calls that may run at the same time need a workspace each.
 */
#ifndef FA_GB300_FA_CACHE_H
#define FA_GB300_FA_CACHE_H

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_CACHE_E4M3 = 0, /* fp8 e4m3 (no infinities, largest value 448) */
  FA_CACHE_INT8 = 1  /* signed integers, -127 .. 127 when written by fa_cache_append */
} fa_cache_kind;

typedef struct fa_cache {
  void* k; /* [P, H_kv, page, D], 8 bits each, any {block, head, token} strides */
  void* v;
  float* k_scale; /* [P, H_kv] contiguous, >= 0 */
  float* v_scale;
  long long k_strides[3]; /* {block, head, token}, bytes; multiples of 16 */
  long long v_strides[3];
  int P, H_kv, page, D; /* page 16, 32, 64 or 128; D 64, 128 or 256 */
  int kind;             /* fa_cache_kind */
} fa_cache;

/*
 * fa_cache_append -- write n new tokens of every sequence behind the tokens
 * that it holds: token t of sequence b goes to position lens[b] + t, for
 * t < n_new[b] (all n when n_new is NULL).
 *
 * A block that receives tokens gets the scale
 *
 *   s' = max(s, 2^e)   where it held tokens before,   2^e  where it did not,
 *   e  = the least integer >= -100 with  max |x| <= MAX * 2^e
 *
 * over the block's new finite values x (MAX 448 or 127); new values are
 * stored as round(x / s') (nearest even; infinities saturate; NaN stays NaN in
 * e4m3 and becomes 0 in int8), and the tokens that it held become
 * round(stored * (s / s')).  With power-of-two scales an e4m3 token that moves
 * to a larger scale keeps all its bits (but for values that underflow), so
 * growing a block again and again adds no error.
 *
 * k, v: [B, H_kv, n, D] in `dtype` (f32, bf16, f16), element strides {batch,
 * head, token}, unit inner stride, 16-byte aligned rows.
 * weights, positions (each may be NULL): [B, H_kv, W] contiguous; the new
 * slots get weight 0 and position seen[b] + t (lens[b] + t when seen is NULL).
 * lens and n_new are read, not changed.
 */
typedef struct fa_cache_append_args {
  fa_cache cache;
  const void* k;
  const void* v;
  long long k_strides[3];
  long long v_strides[3];
  const int* table; /* [B, M], row stride table_stride */
  long long table_stride;
  const int* lens;  /* [B]: tokens held before the call */
  const int* n_new; /* [B] or NULL */
  float* weights;
  int* positions;
  const int* seen; /* [B] or NULL */
  int B, n, M, W;
  int dtype;
  void* stream;
} fa_cache_append_args;

int fa_cache_append(const fa_cache_append_args* args);

/*
 * fa_cache_attn -- attention of n query rows of every sequence over its cached
 * tokens (the rows' own tokens appended before):
 *
 *   S_ij = scale * q[b,h,i,:] . key_j     (then softcap * tanh(S / softcap))
 *   row i of n_q[b] rows (n when n_q is NULL) stands at position
 *   p = lens[b] - n_q[b] + i and sees the keys j <= p (all j < lens[b] when
 *   causal is 0), of those j > p - window when window > 0
 *   O = softmax(S) V, L = the natural-log logsumexp of S
 *   weights[b, kvh, j] += sum over i and the heads of kvh's group of softmax(S)_ij
 *
 * A row that sees no key, and the rows i >= n_q[b] that pad a sequence, get
 * O = 0 and L = -inf and add no weight.  Keys that no row sees get weight
 * added 0.  Stored bytes behind lens[b] may be anything, NaN included.  (A NaN
 * or a +infinite score that a row sees makes that row's O and L NaN, and the
 * weights of the tokens that it sees, as the formula does; a row whose scores
 * are all -infinite counts as one that sees no key.
 * A NaN among the values of a token may also reach the rows of its sequence and
 * K/V head that see other tokens but not that one, where another row of the
 * call does: a weight of 0 times NaN is NaN.)
 *
 * q, o: [B, H_q, n, D] bf16 or fp16, element strides {batch, head, row}, unit
 * inner stride, 16-byte aligned; lse: fp32 contiguous [B, H_q, n]; weights:
 * NULL or fp32 contiguous [B, H_kv, W], W >= every lens[b] (tokens at W and
 * behind get none and set the status above).  Sums over rows and heads are
 * taken in a fixed order: results do not change from run to run.  The order
 * depends on how the work is shared out, so on the device's SM count and on
 * fa_set_max_ctas, which caps this call's thread blocks too (SMs, or pairs an SM
 * for few rows): results with another cap differ by fp32 rounding.
 * workspace: 256-byte aligned, fa_cache_attn_workspace_bytes(args) bytes.
 */
typedef struct fa_cache_attn_args {
  fa_cache cache;
  const void* q;
  void* o;
  float* lse;
  float* weights;
  long long q_strides[3];
  long long o_strides[3];
  const int* table;
  long long table_stride;
  const int* lens; /* [B]: tokens held, the query rows' own among them */
  const int* n_q;  /* [B] or NULL */
  int B, H_q, n, M, W;
  float scale;
  int causal;
  int window;
  float softcap;
  int dtype;
  void* workspace;
  long long workspace_bytes;
  void* stream;
} fa_cache_attn_args;

int fa_cache_attn(const fa_cache_attn_args* args);

/* Bytes of scratch fa_cache_attn needs (it depends on shapes alone); -1 (with
 * the message set) when the arguments are invalid. */
long long fa_cache_attn_workspace_bytes(const fa_cache_attn_args* args);

/*
 * fa_cache_attn_tree -- fa_cache_attn where the rows are the drafts of a tree:
 * row i of n_q[b] is a node, its token in slot base + i, base = lens[b] -
 * n_q[b] (all appended before, as any tokens), and tree[b, i] the row of its
 * parent, which is less than i; -1: the node follows the last token before the
 * drafts.  Then
 *
 *   depth(i) = depth(tree[b, i]) + 1, 0 for a node without parent
 *   row i stands at position base + depth(i) and sees the tokens before slot
 *   base, itself and the nodes above it; of these, with window > 0, those whose
 *   position is more than its own - window
 *
 * A chain (tree[b, i] = i - 1) is fa_cache_attn.  Rows need not have one root.
 * An entry that is no earlier row counts as -1 (entries of the rows i < n_q[b]
 * alone are read), and fa_sync_status() then reports FA_ERR_INVALID_ARGUMENT
 * once.  Scores, O, L, weights (of all rows; fa_cache_accept moves them with
 * their tokens), paddings and NaN as fa_cache_attn has them; `attn.causal` must
 * be set, and n at most 1024.
 * attn.workspace: 256-byte aligned, fa_cache_attn_tree_workspace_bytes(args) bytes.
 */
typedef struct fa_cache_attn_tree_args {
  fa_cache_attn_args attn;
  const int* tree;       /* [B, n] */
  long long tree_stride; /* between sequences; 0: one tree for all */
} fa_cache_attn_tree_args;

int fa_cache_attn_tree(const fa_cache_attn_tree_args* args);
long long fa_cache_attn_tree_workspace_bytes(const fa_cache_attn_tree_args* args);

/*
 * fa_verify_drafts -- which drafted tokens stay, so that what is kept, and the
 * token behind it, are distributed as the target's probabilities say.
 *
 * Node 0 of a sequence's n_q[b] nodes (n when n_q is NULL) is its last token,
 * which stays; node i > 0 is a draft of token tokens[b, i], behind its parent
 * tree[b, i] (as in fa_cache_attn_tree; nodes without parent but node 0 are
 * never reached).  p[b, i, :] are the target's probabilities behind node i,
 * q[b, i, :] those that node i's children were drawn from, independently and in
 * the order of their rows; with q NULL the children of a node are distinct
 * candidates chosen without chance.  From node 0 the path goes on as follows.
 * At its last node c, with r = p[c], Z = 1, for each child i in order, t its token:
 *
 *   u[b, i] * q[c, t] * Z < r[t]   (1 for q[c, t] where q is NULL):
 *       the path goes on at i; else
 *   r = max(r - Z q[c], 0), Z = sum of r   (q NULL: Z -= r[t], r[t] = 0)
 *
 * Where no child is left, or none was taken, the next token is the least t with
 * r[0] + .. + r[t] > u_next[b] * (r[0] + r[1] + ..).  If all of r is 0, p[c]
 * takes its place (and token 0, if that is 0 too).
 *
 * path[b, :] are the path's nodes, ascending, path[b, 0] = 0, then -1;
 * count[b] how many they are (node 0 among them); token[b] the next token.  A
 * sequence of no nodes gets count 0 and token -1.
 *
 * p, q: `dtype` (f32, bf16, f16), element strides {batch, node}, unit inner
 * stride; rows sum to 1 up to their rounding.  What is no positive finite
 * number counts as 0.  u, u_next: fp32 in [0, 1), the caller's random numbers.
 * Sums are taken in 48 bits and more, in a fixed order.
 * A tree entry out of range counts as -1, a token outside [0, V) is rejected
 * (its q is 0), n_q[b] outside [0, n] is cut, and fa_sync_status() then reports
 * FA_ERR_INVALID_ARGUMENT once.  n at most 1024, V at most 2^20.
 */
typedef struct fa_verify_drafts_args {
  const void* p; /* [B, n, V] */
  const void* q; /* [B, n, V] or NULL */
  long long p_strides[2];
  long long q_strides[2];
  const int* tokens;       /* [B, n] */
  long long tokens_stride; /* between sequences */
  const int* tree;         /* [B, n] */
  long long tree_stride;   /* between sequences; 0: one tree for all */
  const float* u;          /* [B, n] */
  long long u_stride;      /* between sequences */
  const float* u_next;     /* [B] */
  const int* n_q;          /* [B] or NULL */
  int* path;               /* [B, n] contiguous */
  int* count;              /* [B] */
  int* token;              /* [B] */
  int B, n, V;
  int dtype;
  void* stream;
} fa_verify_drafts_args;

int fa_verify_drafts(const fa_verify_drafts_args* args);

/*
 * fa_cache_accept -- of the n_q[b] drafts (n when n_q is NULL) that end the
 * lens[b] tokens of a sequence, those of a path become its next tokens, the
 * others are dropped: with base = lens[b] - n_q[b], the token in slot base +
 * path[b, i] moves to slot base + i, for i < count[b], and lens_out[b] = base +
 * count[b].  Paths ascend; fa_verify_drafts makes them.  For every layer's cache
 * alike, with the same path.
 *
 * A block that receives tokens gets the largest scale s' of the blocks that
 * its tokens come from (its own among them where tokens stay before those that
 * come); a token from a block of scale s becomes round(stored * (s / s')).
 * weights: NULL or fp32 contiguous [B, H_kv, W], moved along.  (A slot's position
 * is that of the path's token that it receives: fa_cache_append's numbers stay.)
 * Slots behind lens_out[b] keep what they held.
 * lens_out may be lens itself; it shares no other memory with the inputs.
 * A path that does not ascend, leaves [0, n_q[b]), or (lens[b] past the table)
 * reaches a draft that the table has no slot for, ends before that entry;
 * count[b] is cut to [0, n_q[b]]; a sequence with fewer tokens than drafts, or
 * n_q[b] outside [0, n], stays as it is; fa_sync_status() then reports
 * FA_ERR_INVALID_ARGUMENT once.  n at most 1024.
 */
typedef struct fa_cache_accept_args {
  fa_cache cache;
  const int* table; /* [B, M], row stride table_stride */
  long long table_stride;
  const int* lens; /* [B]: tokens held, the drafts among them */
  const int* n_q;  /* [B] or NULL */
  const int* path; /* [B, n], row stride path_stride */
  long long path_stride;
  const int* count; /* [B] */
  float* weights;
  int* lens_out; /* [B] */
  int B, n, M, W;
  void* stream;
} fa_cache_accept_args;

int fa_cache_accept(const fa_cache_accept_args* args);

/*
 * fa_cache_evict -- keep at most `keep` tokens of every sequence, chosen per
 * K/V head: the `recent` latest ones (positions > the head's largest position
 * - recent), then those with the largest accumulated weight, +infinity the
 * largest; ties go to the lowest slot, a NaN weight counts as -infinity.  A
 * sequence with no more than `keep` tokens keeps all.  The heads of a sequence
 * may keep different tokens; all keep equally many, so table and lens stay
 * common.
 *
 * into == NULL: in place.  Kept tokens in slots below `keep` stay where they
 * are; those at `keep` and behind move, in ascending order, into the slots
 * below `keep` that became free.  weights and positions move along.
 * into != NULL: the kept tokens are copied, in ascending slot order, to the
 * blocks of into [B, M_into] of the same cache (blocks that no sequence of
 * `table` uses); weights and positions go to weights_out, positions_out
 * [B, H_kv, W_out] (each may be NULL) and the sources stay as they were.
 *
 * A block that receives tokens gets the largest scale s' of the blocks that
 * its tokens come from (its own among them where tokens stay); a token from a
 * block of scale s becomes round(stored * (s / s')).
 * lens_out[b] = min(lens[b], keep); lens_out may be lens itself.
 * Slots behind lens_out[b] keep what they held.
 * workspace: 256-byte aligned, fa_cache_evict_workspace_bytes(args) bytes.
 */
typedef struct fa_cache_evict_args {
  fa_cache cache;
  const int* table;
  long long table_stride;
  const int* lens;
  float* weights; /* [B, H_kv, W] contiguous */
  int* positions; /* [B, H_kv, W] contiguous; may be NULL with `into`: a token's position is then its slot */
  const int* into;
  long long into_stride;
  float* weights_out;
  int* positions_out;
  int* lens_out; /* [B] */
  int B, M, W, M_into, W_out;
  int keep, recent;
  void* workspace;
  long long workspace_bytes;
  void* stream;
} fa_cache_evict_args;

int fa_cache_evict(const fa_cache_evict_args* args);
long long fa_cache_evict_workspace_bytes(const fa_cache_evict_args* args);

#ifdef __cplusplus
}
#endif

#endif /* FA_GB300_FA_CACHE_H */
