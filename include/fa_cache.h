/*
 * fa_cache.h -- C ABI of the GB300 (sm_103a) library's serving operators: a
 * paged key/value cache held in 8 bits, attention over it, and eviction from
 * it by accumulated attention weight.  Statuses, error messages, streams and
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
 * writes it (fa_cache_append, fa_cache_evict); sequences that are only read
 * may share blocks.
 *
 * A length past the table (lens[b] > M * page), a negative one, or an entry
 * outside [0, P) that a sequence needs is not followed: the tokens behind it
 * are skipped (not written; not seen by attention; not moved by eviction) and
 * fa_sync_status() then reports FA_ERR_INVALID_ARGUMENT once.
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
