// fa_cache_line.cuh -- how the cache attention kernels share their work.
//
// A segment is a sequence, a K/V head and a group of C::kRows query rows
// (row r: query row r / group, head r % group of the group); its tiles are
// the C::kTile-token pieces of the cache that some of its rows see.  The tiles
// of all segments, in order, form one line, which is cut into equal parts, one
// for each thread block, wherever the cuts fall: sequences of any lengths load
// the machine evenly, and nothing is planned on the host, which does not know
// the lengths.  A thread block that holds a whole segment writes its output;
// the parts of a cut segment go to the workspace, and cache_join_kernel joins
// them.
#pragma once

#include <cuda.h>

#include "fa_cache_ops.cuh"
#include "fa_cache_ptx.cuh"

namespace fa {

constexpr float kDecLn2 = 0.6931471805599453f, kLog2eF = 1.4426950408889634f;
constexpr long long kDecDrainCycles = 1LL << 33;

// Weights in f16.  A row's reference r is set 2^lift below its largest weight so
// far, which is then 2^lift, and set again when one would be more than 2^14 (f16
// ends at 2^16; the rest is room for the rounding of an exponent).  A weight
// keeps all of its f16's 11 bits down to 2^-(14 + lift) of the largest, and is
// lost below 2^-(25 + lift).
constexpr float kDecMost = 14.0f;
constexpr float dec_unlift(int lift) { return 1.0f / (float)(1 << lift); }
// Has a row's largest score left the reference's range?  (The difference of
// two neighbours is exact; false where there is no score yet.)
__device__ __forceinline__ bool dec_grown(float top, float r) { return top - r > kDecMost; }
// The reference for `top`: rounded up, so that top - r is never above the lift.
template <class C>
__device__ __forceinline__ float dec_reference(float top) { return __fsub_ru(top, (float)C::kLift); }

struct DecParams {
  CacheAttnParams a;
  int rows, row_groups;   // rows of a K/V head; groups of kRows
  int max_ctas;
  float* part_o;          // [2 * max_ctas, kRows, D]
  float2* part_ml;        // [2 * max_ctas, kRows]: reference, sum
  float* scores;          // [B, H, M * page / 32, rows, 32]: scores in base 2, for the weights (or NULL)
};

struct DecSeq {
  int len, nq;
};
__device__ __forceinline__ DecSeq dec_seq(const CacheAttnParams& a, int b) {
  DecSeq s;
  const long long most = (long long)a.c.M * a.c.page;
  const int len = a.lens[b];
  s.len = len < 0 ? 0 : (int)min((long long)len, most);
  s.nq = a.n_q ? min(max(a.n_q[b], 0), a.n) : a.n;
  return s;
}

// Tokens that query rows i0 .. i1 see: [lo, hi), empty as {0, 0}.
__device__ __forceinline__ int2 dec_span(const CacheAttnParams& a, const DecSeq& s, int i0, int i1) {
  i1 = min(i1, s.nq - 1);
  if (i0 > i1) return make_int2(0, 0);
  const int p0 = s.len - s.nq + i0, p1 = s.len - s.nq + i1;
  const int hi = a.causal ? min(s.len, p1 + 1) : s.len;
  // (Where a call has more rows than tokens, the first stand before token 0: as
  // far as the window's begin goes, at 0, so that no window leaves 32 bits.)
  const int lo = a.window > 0 ? max(0, max(0, p0) - a.window + 1) : 0;
  return lo < hi ? make_int2(lo, hi) : make_int2(0, 0);
}
// ... and the query rows of row group rg.
template <class C>
__device__ __forceinline__ int2 dec_group_span(const DecParams& p, const DecSeq& s, int rg) {
  if (p.row_groups == 1) return dec_span(p.a, s, 0, p.a.n - 1);
  return dec_span(p.a, s, rg * C::kRows / p.a.group, (min(p.rows, (rg + 1) * C::kRows) - 1) / p.a.group);
}

// Tiles of one segment: at least one, so that empty rows are written too.
template <class C>
__device__ __forceinline__ int dec_tiles(const DecParams& p, const DecSeq& s, int rg) {
  const int2 v = dec_group_span<C>(p, s, rg);
  return max(1, (v.y + C::kTile - 1) / C::kTile - v.x / C::kTile);
}
// Tiles of a head's row groups 0 .. groups-1, by a whole warp (many groups).
template <class C>
__device__ __noinline__ int dec_many_groups(const DecParams& p, DecSeq s, int groups) {
  int n = 0;
#pragma unroll 1
  for (int rg = threadIdx.x & 31; rg < groups; rg += 32) n += dec_tiles<C>(p, s, rg);
  return __reduce_add_sync(0xFFFFFFFFu, n);
}

// A place on the line: a tile's segment.
struct DecPlace {
  int total, part;    // the line's length, and a thread block's part of it
  int b, h, rg;       // the segment: sequence, head, row group
  int seg0;           // its first tile
  DecSeq seq;
};
template <class C>
__device__ __forceinline__ int dec_part(const DecParams& p, int total);

// The place of the first tile of thread block `nth`.  Every warp finds it for
// itself, without a barrier; with one row group a head, up to 32 sequences
// take one load.  (The host keeps all counts below 2^31.)  False past the end.
template <class C>
__device__ __forceinline__ bool dec_find(const DecParams& p, int nth, DecPlace& at) {
  const int lane = threadIdx.x & 31, B = p.a.B, H = p.a.c.H;
  int mine = 0, total = 0, head = 0;
  if (p.row_groups == 1) {
#pragma unroll 1
    for (int i = lane; i < B; i += 32) {
      mine = dec_tiles<C>(p, dec_seq(p.a, i), 0) * H;
      total += mine;
    }
    total = __reduce_add_sync(0xFFFFFFFFu, total);
  } else {
#pragma unroll 1
    for (int i = 0; i < B; ++i) total += dec_many_groups<C>(p, dec_seq(p.a, i), p.row_groups) * H;
  }
  at.total = total;
  at.part = dec_part<C>(p, total);
  at.b = at.h = at.rg = at.seg0 = 0;
  if ((long long)at.part * nth >= total) return false;
  const int t = at.part * nth;
  int before = 0;
  if (p.row_groups == 1) {
#pragma unroll 1
    for (int base = 0;; base += 32) {
      if (B > 32) mine = base + lane < B ? dec_tiles<C>(p, dec_seq(p.a, base + lane), 0) * H : 0;
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += u;
      }
      upto += before;
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, t < upto);
      if (hit) {
        const int l = __ffs(hit) - 1;
        before = __shfl_sync(0xFFFFFFFFu, upto - mine, l);
        at.b = base + l;
        break;
      }
      before = __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
    at.seq = dec_seq(p.a, at.b);
    head = dec_tiles<C>(p, at.seq, 0);
  } else {
#pragma unroll 1
    for (;; ++at.b) {
      at.seq = dec_seq(p.a, at.b);
      head = dec_many_groups<C>(p, at.seq, p.row_groups);
      if (t < before + head * H) break;
      before += head * H;
    }
  }
  at.h = (int)((unsigned)(t - before) / (unsigned)head);
  at.seg0 = before + at.h * head;
  if (p.row_groups > 1) {
#pragma unroll 1
    for (int base = 0;; base += 32) {  // row groups, 32 at a time
      const int n = base + lane < p.row_groups ? dec_tiles<C>(p, at.seq, base + lane) : 0;
      int upto = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += u;
      }
      upto += at.seg0;
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, t < upto);
      if (hit) {
        const int l = __ffs(hit) - 1;
        at.seg0 = __shfl_sync(0xFFFFFFFFu, upto - n, l);
        at.rg = base + l;
        break;
      }
      at.seg0 = __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
  }
  return true;
}

// On to the segment behind one of `tiles` tiles.
__device__ __forceinline__ void dec_next(const DecParams& p, DecPlace& at, int tiles) {
  at.seg0 += tiles;
  if (++at.rg == p.row_groups) {
    at.rg = 0;
    if (++at.h == p.a.c.H) {
      at.h = 0;
      if (++at.b < p.a.B) at.seq = dec_seq(p.a, at.b);
    }
  }
}

// Tiles of one thread block's part of the line: an equal share of the grid's,
// and no less than kMinTiles (a shorter part's join costs more than its tiles),
// but for segments that are shorter themselves: each has a block then (one
// sequence of 128 tokens, 8 heads, D 128: 32 rows a K/V head 28.4 -> 14.6 us, 64
// rows 33.0 -> 14.5).
template <class C>
__device__ __forceinline__ int dec_part(const DecParams& p, int total) {
  const unsigned segments = (unsigned)p.a.B * p.a.c.H * p.row_groups;
  const int usual = (int)(((unsigned)total + segments - 1) / segments);
  return max(max(1, min(C::kMinTiles, usual)), (int)(((unsigned)total + p.max_ctas - 1) / (unsigned)p.max_ctas));
}

// A power of two that brings a query row whose largest entry is `top` into
// [2^9, 2^10), kept inside the normal numbers, and its inverse.
__device__ __forceinline__ void dec_row_scale(float top, float& up, float& down) {
  const int ex = min(max((int)(__float_as_uint(top) >> 23) - 127, -110), 127);
  up = __uint_as_float((uint32_t)(9 - ex + 127) << 23);
  down = __uint_as_float((uint32_t)(ex - 9 + 127) << 23);
}

// Four columns of one output row, and its L: `x` are sums of lifted weights,
// `sum` of weights as they are, both against the reference `top`.
template <class C>
__device__ __forceinline__ void dec_write(const CacheAttnParams& a, int b, int h, int row, int d, const float4& x,
                                          float top, float sum) {
  const int i = row / a.group, head = h * a.group + row % a.group;
  const float inv = rcp_approx(sum) * dec_unlift(C::kLift);
  uint2 y = make_uint2(0u, 0u);  // a row that sees nothing (another's NaN value may be in its x)
  if (sum != 0.0f) {             // (a NaN row stays one)
    y.x = C::kF16 ? pack_f16x2(x.x * inv, x.y * inv) : pack_bf16x2(x.x * inv, x.y * inv);
    y.y = C::kF16 ? pack_f16x2(x.z * inv, x.w * inv) : pack_bf16x2(x.z * inv, x.w * inv);
  }
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + b * a.os[0] + head * a.os[1] + i * a.os[2] + d) = y;
  if (d == 0) a.lse[((long long)b * a.Hq + head) * a.n + i] = sum == 0.0f ? -INFINITY : ((top + C::kLift) + lg2(sum)) * kDecLn2;
}

// The line's length, and the first tile (seg0) of sequence b; one row group.
template <class C>
__device__ __forceinline__ DecPlace dec_before(const DecParams& p, int b) {
  const int lane = threadIdx.x & 31;
  int all = 0, lower = 0;
#pragma unroll 1
  for (int i = lane; i < p.a.B; i += 32) {
    const int n = dec_tiles<C>(p, dec_seq(p.a, i), 0) * p.a.c.H;
    all += n;
    if (i < b) lower += n;
  }
  DecPlace at;
  at.total = __reduce_add_sync(0xFFFFFFFFu, all);
  at.part = dec_part<C>(p, at.total);
  at.b = b;
  at.h = at.rg = 0;
  at.seg0 = __reduce_add_sync(0xFFFFFFFFu, lower);
  return at;
}

// Joins the parts of a cut segment, by the block of the first cut inside it:
// four columns a thread.  Of few rows a block takes 512 / D (`piece` of the
// segment's), every fourth part a quarter of the block, whose sums are added in
// order (38 parts a segment: one sequence of 131071 tokens in all 57.7 us with
// one thread a column for all parts, 52.4 so); of many, four times as many.
constexpr int kJoinThreads = 512;
template <class C>
constexpr bool kJoinByParts = C::kRows <= 32;

template <class C>
__device__ __forceinline__ void join_parts(const DecParams& p, int piece, int cut) {
  const CacheAttnParams& a = p.a;
  constexpr int kRowsHere = 512 / C::kD;  // rows a quarter
  constexpr bool kByParts = kJoinByParts<C>;
  const int tid = threadIdx.x % 128, quarter = threadIdx.x / 128;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  DecPlace at;
  const bool in = dec_find<C>(p, cut, at);
  const int t = at.part * cut;
  const int r = (kByParts ? piece : piece * 4 + quarter) * kRowsHere + tid / (C::kD / 4), row = at.rg * C::kRows + r, d = tid % (C::kD / 4) * 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are written
  if (!in || at.seg0 == t || at.seg0 < t - at.part) return;
  const int c1 = (at.seg0 + dec_tiles<C>(p, at.seq, at.rg) - 1) / at.part;
  float top = -INFINITY, sum = 0.0f;
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](float2 ml, float4 y) {
    const float m2 = fmaxf(top, ml.x), z = m2 == -INFINITY ? 0.0f : m2;
    const float f = ex2(top - z), g = ex2(ml.x - z);
    top = m2;
    sum = fmaf(sum, f, ml.y * g);
    x.x = fmaf(x.x, f, y.x * g), x.y = fmaf(x.y, f, y.y * g), x.z = fmaf(x.z, f, y.z * g), x.w = fmaf(x.w, f, y.w * g);
  };
  if (row < p.rows) {
#pragma unroll 4
    for (int i = cut - 1 + (kByParts ? quarter : 0); i <= c1; i += kByParts ? 4 : 1) {
      const long long slot = (long long)(2 * i + (i == cut - 1)) * C::kRows + r;
      add(__ldcg(p.part_ml + slot), __ldcg(reinterpret_cast<const float4*>(p.part_o + slot * C::kD + d)));
    }
  }
  if constexpr (kByParts) {
    __shared__ float4 s_x[3][128];
    __shared__ float2 s_ml[3][128];
    if (quarter > 0) {
      s_x[quarter - 1][tid] = x;
      s_ml[quarter - 1][tid] = make_float2(top, sum);
    }
    __syncthreads();
    if (quarter > 0) return;
#pragma unroll
    for (int q = 0; q < 3; ++q) add(s_ml[q][tid], s_x[q][tid]);
  }
  if (row < p.rows) dec_write<C>(a, at.b, at.h, row, d, x, top, sum);
}
// Blocks of one cut: no more rows than a segment can have.
template <class C>
__host__ __device__ __forceinline__ int join_pieces(const DecParams& p) {
  const int rows = p.rows < C::kRows ? p.rows : C::kRows, here = 512 / C::kD * (kJoinByParts<C> ? 1 : 4);
  return (rows + here - 1) / here;
}
template <class C>
__global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(const __grid_constant__ DecParams p) {
  join_parts<C>(p, blockIdx.x, blockIdx.y + 1);
}

}  // namespace fa
