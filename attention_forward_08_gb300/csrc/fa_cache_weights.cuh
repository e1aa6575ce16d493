// fa_cache_weights.cuh -- the attention weight that every cached token got:
//
//   weights[b, kvh, j] += sum over rows r of the K/V head of 2^(s_rj - L2_r)
//
// with L2 the row's logsumexp in base 2, known once the attention itself has
// run.  Few rows: the attention leaves its scores, and cache_finish_kernel
// sums them up.  Many: a warp owns 32 tokens, holds their keys in registers,
// computes each score again and goes over the rows, 16 at a time (to keep the
// scores would take 4 bytes a row and token, while a key is 1 byte an element
// for all rows of its head); the query rows are brought into the tensor core's
// order once, by a small kernel before it, together with each row's two
// factors.  Either way sums stay in one thread, so that nothing is added twice
// or in an order that changes.
//
// Bound: the scores' way through L2 for few rows; the second reading of K and
// the tensor cores for many.
#pragma once

#include "fa_cache_decode.cuh"

namespace fa {

struct WeightParams {
  CacheAttnParams a;
  int rows, row_groups;  // rows of a K/V head, and groups of 16 of them
  uint32_t* q;           // [B, H, row group, k-step, lane, 4]: A operands
  float2* row;           // [B, H, row group * 16]: score to base 2 (without k_scale), L2 (+inf: a row that sees nothing)
};

// One warp a row (the grid has 16 warps a row group).
template <bool kF16, int kD>
__global__ void __launch_bounds__(256) cache_rows_kernel(const __grid_constant__ WeightParams p) {
  const CacheAttnParams& a = p.a;
  constexpr int kE = kD / 32;
  const int lane = threadIdx.x & 31, r = blockIdx.x * 8 + (threadIdx.x >> 5), h = blockIdx.y, b = blockIdx.z;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int i = r / a.group, head = h * a.group + r % a.group;
  const bool in = r < p.rows;
  float f[kE], up = 1.0f, down = 1.0f;
#pragma unroll
  for (int e = 0; e < kE; ++e) f[e] = 0.0f;
  if (in) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + b * a.qs[0] +
                                                          head * a.qs[1] + i * a.qs[2]) + lane * (kE / 2);
#pragma unroll
    for (int e = 0; e < kE; e += 2) {
      const uint32_t w = __ldg(q + e / 2);
      f[e] = half_bits_to_f32<kF16>(w);
      f[e + 1] = half_bits_to_f32<kF16>(w >> 16);
    }
  }
  if constexpr (!kF16) {
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) top = fmaxf(top, fabsf(f[e]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    dec_row_scale(top, up, down);
  }
  const long long bh = (long long)b * a.c.H + h;
  uint32_t* out = p.q + (bh * p.row_groups + (r >> 4)) * (kD / 16) * 128;
#pragma unroll
  for (int e = 0; e < kE; e += 2) out[dec_q_word<kD>(r & 15, lane * kE + e)] = pack_f16x2(f[e] * up, f[e + 1] * up);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // L is written
  if (lane == 0) {
    const float lse = in ? a.lse[((long long)b * a.Hq + head) * a.n + i] : -INFINITY;
    p.row[bh * p.row_groups * 16 + r] = make_float2(down, lse == -INFINITY ? INFINITY : lse * kLog2eF);
  }
}

// Of tokens tok0 .. + 31, those that row i of a tree sees.
__device__ __forceinline__ uint32_t weight_seen(const TreeOf& tree, const DecSeq& seq, int pos0, int i, int tok0) {
  if (i >= seq.nq) return 0u;
  const int from = tree.window > 0 ? min(max(tree_first(tree, pos0, tree_depth(tree, i)) - tok0, 0), 32) : 0;
  const int to = min(max(pos0 - tok0, 0), 32);
  uint32_t seen = from < to ? (0xFFFFFFFFu >> (32 - (to - from))) << from : 0u;
  if (to < 32) seen |= tree_walk_here(tree, i, tok0 - pos0);
  return seen;
}

template <int kKind, int kD, bool kTree>
__global__ void __launch_bounds__(128) cache_weights_kernel(const __grid_constant__ WeightParams p) {
  const CacheAttnParams& a = p.a;
  const CacheView& c = a.c;
  const int h = blockIdx.y, b = blockIdx.z, tok0 = (blockIdx.x * 4 + (threadIdx.x >> 5)) * 32;
  const long long bh = (long long)b * c.H + h;
  const DecSeq seq = dec_seq(a, b);
  const uint4* q = reinterpret_cast<const uint4*>(p.q) + bh * p.row_groups * (kD / 16) * 32;
  const float2* row = p.row + bh * p.row_groups * 16;
  constexpr int kK = kD / 16;  // k-steps
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // the query rows that see one of these tokens
  int i0 = 0, i1 = seq.nq - 1;
  const int pos0 = seq.len - seq.nq;
  if (a.causal) i0 = max(0, tok0 - pos0);
  if (!kTree && a.window > 0) i1 = (int)min((long long)i1, (long long)tok0 + 31 + a.window - 1 - pos0);
  // The first token that any row sees: blocks behind the window need not be there.
  const int lo = dec_span<kTree>(a, seq, 0, a.n - 1).x;
  const bool none = tok0 >= seq.len || tok0 + 31 < lo || i0 > i1;
  const int rg0 = i0 * a.group / 16, rg1 = (i1 * a.group + a.group - 1) / 16;

  // keys: lane (g, t) holds the bytes of token 8j + g that it multiplies
  uint32_t w[4][kK];
  float ks[2];
  bool here[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int tok = tok0 + 16 * half;
    int blk = -1;
    if (!none && tok < seq.len && tok + 15 >= lo) blk = checked_block(c, c.table, c.table_stride, b, tok >> c.page_log2);
    here[half] = blk >= 0;
    ks[half] = here[half] ? __ldg(c.k_scale + (long long)blk * c.H + h) : 0.0f;
#pragma unroll
    for (int j = 2 * half; j < 2 * half + 2; ++j) {
      const uint8_t* k = c.k + blk * c.ks[0] + h * c.ks[1] + (((tok0 + 8 * j) & (c.page - 1)) + g) * c.ks[2];
#pragma unroll
      for (int u = 0; u < kK / 4; ++u) {  // 16-byte units: t of the row (D 64), 2t and 2t + 1 of each 128 bytes
        const int at = kD == 64 ? 16 * t : 128 * (u / 2) + 32 * t + 16 * (u & 1);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (here[half]) v = __ldg(reinterpret_cast<const uint4*>(k + at));
        w[j][4 * u] = v.x, w[j][4 * u + 1] = v.y, w[j][4 * u + 2] = v.z, w[j][4 * u + 3] = v.w;
      }
    }
  }
  // The rows are there (every block waits, also one that has nothing to do: a
  // grid ends no earlier than the one before it).
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (none) return;
  const bool raw = a.cap_out == 0.0f;
  const TreeOf tree = tree_of(a, b);
  float sum[4][2] = {};
#pragma unroll 1
  for (int rg = rg0; rg <= rg1; ++rg) {
    float sc[4][4] = {};
#pragma unroll
    for (int kk = 0; kk < kK; ++kk) {
      const uint4 x = __ldcg(q + ((long long)rg * kK + kk) * 32 + lane);
      const uint32_t qa[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t b0, b1;
        to_f16x4<kKind>(w[j][kk], b0, b1);
        mma_f16(sc[j], qa, b0, b1);
      }
    }
    const float2 r0 = __ldcg(row + rg * 16 + g), r1 = __ldcg(row + rg * 16 + g + 8);
    const int ia = (rg * 16 + g) / a.group, ib = (rg * 16 + g + 8) / a.group;
    // Tokens that rows g and g + 8 see (a row that is none has L2 = +inf): from .x
    // to .y; of a tree's, bits from this lane's first token on.
    int2 va = make_int2(0, 0), vb = va;
    uint32_t sa = 0u, sb = 0u;
    if constexpr (kTree) {
      sa = weight_seen(tree, seq, pos0, ia, tok0) >> (2 * t), sb = weight_seen(tree, seq, pos0, ib, tok0) >> (2 * t);
      __syncwarp();  // (each lane has walked for itself; the next rows' products take whole warps)
    } else {
      va = dec_span(a, seq, ia, ia), vb = dec_span(a, seq, ib, ib);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 r = e < 2 ? r0 : r1;
        float s = sc[j][e];
        if (kTree && raw) {
          s = fmaf(s, ks[j >> 1] * (r.x * a.scale_log2), -r.y);
        } else {
          s *= ks[j >> 1] * r.x;
          s = raw ? s * a.scale_log2
                  : fmaf(-2.0f * a.cap_out, rcp_approx(ex2(s * a.cap_in * 2.8853900817779268f) + 1.0f), a.cap_out);
          s -= r.y;
        }
        bool seen;
        if constexpr (kTree) {
          seen = ((e < 2 ? sa : sb) >> (8 * j + (e & 1))) & 1u;
        } else {
          const int2 v = e < 2 ? va : vb;
          const int tok = tok0 + 8 * j + 2 * t + (e & 1);
          seen = tok >= v.x && tok < v.y;
        }
        if (seen) sum[j][e & 1] += ex2(s);
      }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum[j][e] += __shfl_xor_sync(0xFFFFFFFFu, sum[j][e], o);
    }
  if (g == 0) {
    float* out = a.weights + ((long long)b * c.H + h) * a.W;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tok = tok0 + 8 * j + 2 * t + e;
        if (tok >= seq.len || !here[j >> 1]) continue;
        if (tok >= a.W)
          flag_bad_index(c);
        else
          out[tok] += sum[j][e];
      }
  }
}

// Few rows (one row group of the decode kernel's): that kernel has left its
// scores, 4 bytes a row and token, and one kernel joins the parts of cut
// segments (its first `joins` blocks) and sums the weights, a thread a token.
// A block finds the rows' L where the parts say so: a few numbers a row.
constexpr int kFinishTokens = kJoinThreads;  // a block

template <class C>
__global__ void __launch_bounds__(kJoinThreads) cache_finish_kernel(const __grid_constant__ DecParams p, int joins, int chunks) {
  const CacheAttnParams& a = p.a;
  if ((int)blockIdx.x < joins) {
    const int pieces = join_pieces<C>(p);
    join_parts<C>(p, blockIdx.x % pieces, blockIdx.x / pieces + 1);
    return;
  }
  __shared__ float s_l2[C::kRows];
  const int nth = blockIdx.x - joins, tid = threadIdx.x;
  const int bh = nth / chunks, h = bh % a.c.H, b = bh / a.c.H, tok0 = nth % chunks * kFinishTokens;
  const DecSeq seq = dec_seq(a, b);
  const int2 span = dec_group_span<C>(p, seq, 0);
  const DecPlace at = dec_before<C>(p, b);
  const int tiles = dec_tiles<C>(p, seq, 0), u0 = at.seg0 + h * tiles, u1 = u0 + tiles;
  const int c0 = u0 / at.part, c1 = (u1 - 1) / at.part;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // scores, parts, and the L of whole segments are written
  if (tok0 >= span.y || tok0 + kFinishTokens <= span.x) return;
  if (tid < p.rows) {
    float l2;
    if (c0 == c1) {
      const int i = tid / a.group, head = h * a.group + tid % a.group;
      l2 = __ldcg(a.lse + ((long long)b * a.Hq + head) * a.n + i) * kLog2eF;
    } else {
      float top = -INFINITY, sum = 0.0f;
#pragma unroll 4
      for (int i = c0; i <= c1; ++i) {
        const float2 ml = __ldcg(p.part_ml + (long long)(2 * i + (i == c0)) * C::kRows + tid);
        const float m2 = fmaxf(top, ml.x), z = m2 == -INFINITY ? 0.0f : m2;
        sum = fmaf(sum, ex2(top - z), ml.y * ex2(ml.x - z));
        top = m2;
      }
      l2 = sum == 0.0f ? -INFINITY : (top + C::kLift) + lg2(sum);
    }
    s_l2[tid] = l2 == -INFINITY ? INFINITY : l2;  // (a row that sees nothing adds nothing)
  }
  __syncthreads();
  const float* scores = p.scores + (long long)bh * ((a.c.M * (a.c.page >> 4) + 1) / 2) * p.rows * 32;
  float* out = a.weights + (long long)bh * a.W;
  const int tok = tok0 + tid;
  if (tok < span.x || tok >= span.y) return;
  const float* s = scores + (long long)(tok >> 5) * p.rows * 32 + (tok & 31);
  float sum = 0.0f;
#pragma unroll 4
  for (int r = 0; r < p.rows; ++r) sum += ex2(__ldcg(s + r * 32) - s_l2[r]);
  if (sum != sum) {  // a NaN row among them: only for the tokens that it sees
    sum = 0.0f;
    for (int r = 0; r < p.rows; ++r) {
      bool seen;
      if constexpr (C::kTree) {
        seen = tree_sees(tree_of(a, b), seq, r / a.group, tok);
      } else {
        const int2 see = dec_span(a, seq, r / a.group, r / a.group);
        seen = tok >= see.x && tok < see.y;
      }
      if (seen) sum += ex2(__ldcg(s + r * 32) - s_l2[r]);
    }
  }
  if (tok < a.W)
    out[tok] += sum;
  else
    flag_bad_index(a.c);
}

}  // namespace fa
