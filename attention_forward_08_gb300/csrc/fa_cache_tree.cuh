// fa_cache_tree.cuh -- which tokens a draft of a tree sees (include/fa_cache.h,
// fa_cache_attn_tree): those before the drafts, itself, and the drafts above it;
// with a window, of these the latest `window`.
//
// Drafts are numbered in rows, parents before children, so that a node's line
// (itself and what is above it) as bits by row has its latest token highest.
// Lines are found by each block for itself: of up to 32 nodes, a lane a node,
// by doubling; of more, a thread a row, by walking up.
#pragma once

#include <climits>

#include "fa_cache_line.cuh"

namespace fa {

// A sequence's tree.  (By value: a walk that had its numbers behind a reference
// to the kernel's parameters fetched them again at each step, 15 us a call.)
struct TreeOf {
  const int* up;  // parents
  int n, window;
  unsigned int* status;
};
__device__ __forceinline__ TreeOf tree_of(const CacheAttnParams& a, int b) {
  return {a.tree + b * a.tree_stride, a.n, a.window, a.c.status};
}

// The row above `node` (-1: none).  An entry that is no earlier row counts as -1, and is told.
__device__ __forceinline__ int tree_parent(const TreeOf& t, int node) {
  const int up = __ldg(t.up + node);
  if (up >= node || up < -1) {
    atomicOr(t.status, kStatusBadIndex);
    return -1;
  }
  return up;
}

// How many drafts are above node i.
__device__ __forceinline__ int tree_depth(const TreeOf& t, int i) {
  int depth = 0;
#pragma unroll 1
  while ((i = tree_parent(t, i)) >= 0) ++depth;
  return depth;
}
// The first token before the drafts (the first of them in slot `base`) that a window shows a node.
__device__ __forceinline__ int tree_first(const TreeOf& t, int base, int depth) {
  return max(0, max(0, base + depth) - t.window + 1);
}

// Up to 32 nodes, by a whole warp, lane i with node i's parent: its line.
__device__ __forceinline__ uint32_t tree_lines(int up) {
  uint32_t line = 1u << (threadIdx.x & 31);
#pragma unroll
  for (int r = 0; r < 5; ++r) {  // lines of 1, 2, 4, .. 32 nodes; `up` is the node above the line
    const int from = up & 31;
    const uint32_t theirs = __shfl_sync(0xFFFFFFFFu, line, from);
    const int next = __shfl_sync(0xFFFFFFFFu, up, from);
    if (up >= 0) line |= theirs, up = next;
  }
  return line;
}
// Cuts a line to the window; returns the first token before the drafts that is seen.
__device__ __forceinline__ int tree_window(const TreeOf& t, int base, uint32_t& line) {
  if (t.window <= 0) return 0;
  const int first = tree_first(t, base, __popc(line) - 1);
#pragma unroll 1
  for (int more = __popc(line) - t.window; more > 0; --more) line &= line - 1;
  return first;
}
__device__ __forceinline__ bool tree_bit(uint32_t line, int i) { return (unsigned)i < 32u && ((line >> i) & 1u); }

// Any number of nodes, by a thread for itself: row i's line, cut to the window,
// as words kStride apart.
template <int kStride>
__device__ __noinline__ void tree_write_line(TreeOf t, int i, uint32_t* words) {
  for (int w = 0; w < (t.n + 31) / 32; ++w) words[w * kStride] = 0u;
  for (int n = t.window > 0 ? t.window : INT_MAX; i >= 0 && n > 0; --n) {
    words[(i >> 5) * kStride] |= 1u << (i & 31);
    i = tree_parent(t, i);
  }
}
// Bits `from` .. from + 31 of row i's line (from may be negative), by walking up;
__device__ __forceinline__ uint32_t tree_walk_here(const TreeOf& t, int i, int from) {
  uint32_t bits = 0u;
  for (int n = t.window > 0 ? t.window : INT_MAX; i >= from && i >= 0 && n > 0; --n) {
    if (i < from + 32) bits |= 1u << (i - from);
    i = tree_parent(t, i);
  }
  return bits;
}
// (a call, where it is rare and its registers would be another's)
__device__ inline __noinline__ uint32_t tree_walk(TreeOf t, int i, int from) { return tree_walk_here(t, i, from); }
// ... or of a line of n nodes that was written.
template <int kStride>
__device__ __forceinline__ uint32_t tree_read_line(const uint32_t* words, int n, int from) {
  const int w = from >> 5, most = (n + 31) / 32;
  const uint32_t lo = w >= 0 && w < most ? words[w * kStride] : 0u;
  const uint32_t hi = w >= -1 && w + 1 < most ? words[(w + 1) * kStride] : 0u;
  return __funnelshift_r(lo, hi, from & 31);
}

// Does row i of `rows` see the draft in row `node`?
__device__ inline __noinline__ bool tree_sees_draft(TreeOf t, int rows, int i, int node) {
  if (node < 0 || node > i || i >= rows) return false;
  int n = t.window > 0 ? t.window : INT_MAX;
  while (i > node && --n > 0) i = tree_parent(t, i);
  return i == node && n > 0;
}
// ... or any token of the cache?
__device__ __forceinline__ bool tree_sees(const TreeOf& t, const DecSeq& s, int i, int tok) {
  const int base = s.len - s.nq;
  if (tok >= base) return tree_sees_draft(t, s.nq, i, tok - base);
  return i < s.nq && (t.window <= 0 || tok >= tree_first(t, base, tree_depth(t, i)));
}

}  // namespace fa
