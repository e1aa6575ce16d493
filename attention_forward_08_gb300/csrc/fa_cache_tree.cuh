// fa_cache_tree.cuh -- which tokens a draft of a tree sees (include/fa_cache.h,
// fa_cache_attn_tree): those before the drafts, itself, and the drafts above it;
// with a window, of these the latest `window`.
//
// Drafts are numbered in rows, parents before children, so that a node's line
// (itself and what is above it) as bits by row has its latest token highest.
// Lines are found by each block for itself: of few rows, a lane a node, by
// doubling; of many, a thread a row, by walking up.
#pragma once

#include <climits>

#include "fa_cache_line.cuh"

namespace fa {

// The row above `node` (-1: none).  An entry that is no earlier row counts as -1, and is told.
__device__ __forceinline__ int tree_parent(const CacheAttnParams& a, int b, int node) {
  const int up = __ldg(a.tree + b * a.tree_stride + node);
  if (up >= node || up < -1) {
    flag_bad_index(a.c);
    return -1;
  }
  return up;
}

// How many drafts are above node i.
__device__ __forceinline__ int tree_depth(const CacheAttnParams& a, int b, int i) {
  int depth = 0;
#pragma unroll 1
  while ((i = tree_parent(a, b, i)) >= 0) ++depth;
  return depth;
}
// The first token before the drafts (the first of them in slot `base`) that a window shows a node.
__device__ __forceinline__ int tree_first(const CacheAttnParams& a, int base, int depth) {
  return max(0, max(0, base + depth) - a.window + 1);
}

// Up to 32 nodes, by a whole warp: lane i's line.
__device__ __forceinline__ uint32_t tree_lines(const CacheAttnParams& a, int b, int nodes) {
  const int lane = threadIdx.x & 31;
  int up = lane < nodes ? tree_parent(a, b, lane) : -1;
  uint32_t line = 1u << lane;
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
__device__ __forceinline__ int tree_window(const CacheAttnParams& a, int base, uint32_t& line) {
  if (a.window <= 0) return 0;
  const int first = tree_first(a, base, __popc(line) - 1);
#pragma unroll 1
  for (int more = __popc(line) - a.window; more > 0; --more) line &= line - 1;
  return first;
}
__device__ __forceinline__ bool tree_bit(uint32_t line, int i) { return (unsigned)i < 32u && ((line >> i) & 1u); }

// Any number of nodes, by a thread for itself: row i's line, cut to the window,
// as words kStride apart.
template <int kStride>
__device__ __noinline__ void tree_write_line(const CacheAttnParams& a, int b, int i, uint32_t* words) {
  for (int w = 0; w < (a.n + 31) / 32; ++w) words[w * kStride] = 0u;
  for (int n = a.window > 0 ? a.window : INT_MAX; i >= 0 && n > 0; --n) {
    words[(i >> 5) * kStride] |= 1u << (i & 31);
    i = tree_parent(a, b, i);
  }
}
// Bits `from` .. from + 31 of row i's line (from may be negative), by walking up;
__device__ inline __noinline__ uint32_t tree_walk(const CacheAttnParams& a, int b, int i, int from) {
  uint32_t bits = 0u;
  for (int n = a.window > 0 ? a.window : INT_MAX; i >= from && i >= 0 && n > 0; --n) {
    if (i < from + 32) bits |= 1u << (i - from);
    i = tree_parent(a, b, i);
  }
  return bits;
}
// ... or of a line of n nodes that was written.
template <int kStride>
__device__ __forceinline__ uint32_t tree_read_line(const uint32_t* words, int n, int from) {
  const int w = from >> 5, most = (n + 31) / 32;
  const uint32_t lo = w >= 0 && w < most ? words[w * kStride] : 0u;
  const uint32_t hi = w >= -1 && w + 1 < most ? words[(w + 1) * kStride] : 0u;
  return __funnelshift_r(lo, hi, from & 31);
}

// Does row i see the draft in slot `tok`?
__device__ inline __noinline__ bool tree_sees_draft(const CacheAttnParams& a, const DecSeq& s, int b, int i, int tok) {
  const int base = s.len - s.nq, node = tok - base;
  if (tok < base || node > i || i >= s.nq) return false;
  int n = a.window > 0 ? a.window : INT_MAX;
  while (i > node && --n > 0) i = tree_parent(a, b, i);
  return i == node && n > 0;
}
// ... or any token of the cache?
__device__ __forceinline__ bool tree_sees(const CacheAttnParams& a, const DecSeq& s, int b, int i, int tok) {
  const int base = s.len - s.nq;
  if (tok >= base) return tree_sees_draft(a, s, b, i, tok);
  return i < s.nq && (a.window <= 0 || tok >= tree_first(a, base, tree_depth(a, b, i)));
}

}  // namespace fa
