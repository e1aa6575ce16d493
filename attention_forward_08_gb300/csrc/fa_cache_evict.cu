// fa_cache_evict.cu -- keep the heaviest and latest tokens (include/fa_cache.h).
//
// Two launches.  The first chooses: one thread block per sequence and head
// finds, digit by digit, the key of the last token that is kept (a radix
// selection: four passes over the weights, each counting one byte of those
// that match the bytes found so far), and writes for every slot below `keep`
// which slot's token ends there.  The second moves: one thread block per
// (sequence, head, receiving block of K or of V).
//
// In place, only tokens in slots at `keep` and behind move, and only into
// slots below `keep`: no slot is both read and written, so the moves need no
// order, and a decoding step that evicts one token moves one token, not a
// whole cache.
//
// Bound: memory.  Choosing reads 8 bytes a token and head (weight, position);
// moving reads and writes 2 * D bytes per moved token and head.
#include <climits>

#include "fa.h"
#include "fa_cache.h"
#include "fa_cache_ops.cuh"
#include "fa_device.h"

namespace fa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

// A weight as an unsigned key of the same order: -inf and NaN lowest, -0 as +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w != w ? -INFINITY : w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

__global__ void __launch_bounds__(kPlanThreads) cache_evict_plan_kernel(const EvictParams p) {
  const CacheView& c = p.c;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long bh = (long long)b * c.H + h;
  __shared__ int hist[256];
  __shared__ int part[kPlanWarps][4];
  __shared__ int s_max, s_digit, s_need;
  int n = checked_len(c, p.lens[b]);
  if (n > p.W) {
    if (tid == 0) flag_bad_index(c);
    n = p.W;
  }
  int* src = p.src + bh * p.keep;
  if (tid == 0) p.count[bh] = n <= p.keep ? (p.into ? n : -1 - n) : p.keep;
  if (n <= p.keep) {  // all stay (a copy takes them all, in order)
    if (p.into)
      for (int j = tid; j < n; j += kPlanThreads) src[j] = j;
    return;
  }
  const float* weight = p.weights + bh * p.W;
  const int* position = p.positions ? p.positions + bh * p.W : nullptr;
  if (tid == 0) s_max = INT_MIN;
  __syncthreads();
  if (p.recent > 0) {
    int most = position ? INT_MIN : n - 1;
    if (position)
      for (int j = tid; j < n; j += kPlanThreads) most = max(most, position[j]);
    atomicMax(&s_max, most);
  }
  __syncthreads();
  // Positions above the bound are kept first (long: the bound may lie below INT_MIN).
  const long long late = p.recent > 0 ? (long long)s_max - p.recent : LLONG_MAX;
  auto key_of = [&](int j) -> uint32_t {
    const long long pos = position ? position[j] : j;
    return weight_key(pos > late ? INFINITY : weight[j]);
  };
  uint32_t found = 0;  // the bytes found so far
  int need = p.keep;   // tokens still to take among those that match them
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
    for (int j = tid; j < n; j += kPlanThreads) {
      const uint32_t k = key_of(j);
      if ((k & mask) == found) atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {  // the digit at which the count from above reaches `need`
      int mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += hist[255 - (lane * 8 + i)];
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += t;
      }
      int before = upto - mine;
      if (before < need && upto >= need) {
        for (int i = 0; i < 8; ++i) {
          const int d = 255 - (lane * 8 + i);
          if (before + hist[d] >= need) {
            s_digit = d;
            s_need = need - before;
            break;
          }
          before += hist[d];
        }
      }
    }
    __syncthreads();
    found |= (uint32_t)s_digit << shift;
    need = s_need;
    __syncthreads();
  }
  // Kept: keys above `found`, and the first `need` slots whose key equals it.
  // Every warp owns a run of slots; a first sweep counts what lies before it.
  // In place, with `kept_lo` of the slots below `keep` kept: the slot j that
  // becomes free is hole number j - (kept slots before j), and a kept slot at
  // `keep` or behind is mover number (kept slots before it) - kept_lo; hole i
  // takes mover i.
  const int run = ((n + kPlanThreads - 1) / kPlanThreads) * 32;
  const int j0 = warp * run, j1 = min(n, j0 + run);
  int above = 0, equal = 0, above_lo = 0, equal_lo = 0;
  for (int j = j0 + lane; j < j1; j += 32) {
    const uint32_t k = key_of(j);
    const bool lo = j < p.keep;
    above += k > found;
    equal += k == found;
    above_lo += lo && k > found;
    equal_lo += lo && k == found;
  }
  above = warp_sum(above);
  equal = warp_sum(equal);
  above_lo = warp_sum(above_lo);
  equal_lo = warp_sum(equal_lo);
  if (lane == 0) part[warp][0] = above, part[warp][1] = equal, part[warp][2] = above_lo, part[warp][3] = equal_lo;
  __syncthreads();
  int eq = 0, kept_n = 0, kept_lo = 0, eq_lo = 0;
  for (int w = 0; w < kPlanWarps; ++w) {
    if (w < warp) {
      kept_n += part[w][0];
      eq += part[w][1];
    }
    kept_lo += part[w][2];
    eq_lo += part[w][3];
  }
  kept_n += min(eq, need);
  kept_lo += min(eq_lo, need);
  int* mover = p.mover + bh * p.keep;
  const uint32_t below = (1u << lane) - 1;
  for (int base = j0; base < j1; base += 32) {
    const int j = base + lane;
    const bool in = j < j1;
    const uint32_t k = in ? key_of(j) : 0;
    const uint32_t e = __ballot_sync(0xFFFFFFFFu, in && k == found);
    const bool kept = in && (k > found || (k == found && eq + __popc(e & below) < need));
    const uint32_t kb = __ballot_sync(0xFFFFFFFFu, kept);
    const int at = kept_n + __popc(kb & below);  // kept slots before j
    if (p.into) {
      if (kept) src[at] = j;
    } else if (in && j < p.keep) {
      src[j] = kept ? j : -1 - (j - at);
    } else if (kept) {
      mover[at - kept_lo] = j;
    }
    kept_n += __popc(kb);
    eq += __popc(e);
  }
  if (!p.into && tid < 2) {  // the block of slot `keep` may hold sources and be rescaled as a receiver
    const int blk = checked_block(c, c.table, c.table_stride, b, p.keep >> c.page_log2);
    p.edge[2 * bh + tid] = blk < 0 ? 0.0f : (tid ? c.v_scale : c.k_scale)[(long long)blk * c.H + h];
  }
}

// Moves the tokens of one receiving block.  A token's scale is that of the
// block it comes from; of the one source block that may itself receive (it
// holds slot `keep`) the scale from before the call is used.
template <int kKind>
__global__ void __launch_bounds__(256) cache_evict_move_kernel(const EvictParams p) {
  const CacheView& c = p.c;
  const int m = blockIdx.x, h = blockIdx.y % c.H, is_v = blockIdx.y / c.H, b = blockIdx.z, tid = threadIdx.x;
  const long long bh = (long long)b * c.H + h;
  const int count = p.count[bh];
  if (m == 0 && blockIdx.y == 0 && tid == 0) p.lens_out[b] = count < 0 ? -1 - count : count;
  const int j0 = m << c.page_log2;
  if (j0 >= count) return;
  const int tokens = min(c.page, count - j0);
  __shared__ int s_slot[128];
  __shared__ int s_block[128];
  __shared__ float s_scale[128];
  __shared__ float s_top[4];
  __shared__ int s_moves;
  const bool in_place = p.into == nullptr;
  if (tid == 0) s_moves = 0;
  __syncthreads();
  float* scales = is_v ? c.v_scale : c.k_scale;
  const int edge = p.keep >> c.page_log2;
  float top = 0.0f;
  if (tid < tokens) {
    int s = p.src[bh * p.keep + j0 + tid];
    if (s < 0) s = p.mover[bh * p.keep - 1 - s];
    s_slot[tid] = s;
    if (s != j0 + tid) s_moves = 1;
  }
  __syncthreads();
  if (in_place && !s_moves) return;
  if (tid < tokens) {
    const int s = s_slot[tid], mb = s >> c.page_log2;
    const int blk = checked_block(c, c.table, c.table_stride, b, mb);
    s_block[tid] = blk;
    float sc = 0.0f;
    if (blk >= 0) sc = in_place && mb == edge ? p.edge[2 * bh + is_v] : scales[(long long)blk * c.H + h];
    s_scale[tid] = sc;
    top = sc;
  }
  if (tid < 128) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if ((tid & 31) == 0) s_top[tid >> 5] = top;
  }
  __syncthreads();
  top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
  const int to = in_place ? checked_block(c, c.table, c.table_stride, b, m)
                          : checked_block(c, p.into, p.into_stride, b, m);
  if (to < 0) return;
  const long long* cs = is_v ? c.vs : c.ks;
  uint8_t* pool = is_v ? c.v : c.k;
  uint8_t* out = pool + to * cs[0] + h * cs[1];
  const int vd = c.D >> 4, vd_log2 = 31 - __clz(vd);  // 16-byte vectors a token
  for (int v = tid; v < tokens * vd; v += blockDim.x) {
    const int t = v >> vd_log2, at = (v & (vd - 1)) * 16, s = s_slot[t];
    if (s_block[t] < 0) continue;
    const float sc = s_scale[t];
    if (in_place && s == j0 + t && sc == top) continue;  // stays as it is
    uint4 w = *reinterpret_cast<const uint4*>(pool + s_block[t] * cs[0] + h * cs[1] + (s & (c.page - 1)) * cs[2] + at);
    if (sc != top) {
      const float ratio = __fdiv_rn(sc, top);
      uint32_t* u = &w.x;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float f[4];
        load8x4<kKind>(u[i], f);
        u[i] = round8x4<kKind>(__fmul_rn(f[0], ratio), __fmul_rn(f[1], ratio), __fmul_rn(f[2], ratio),
                               __fmul_rn(f[3], ratio));
      }
    }
    *reinterpret_cast<uint4*>(out + t * cs[2] + at) = w;
  }
  if (tid == 0) scales[(long long)to * c.H + h] = top;
  if (!is_v && tid < tokens) {
    const int s = s_slot[tid];
    float* w_out = in_place ? p.weights : p.weights_out;
    int* p_out = in_place ? p.positions : p.positions_out;
    const long long width = in_place ? p.W : p.W_out, at = bh * width + j0 + tid, from = bh * p.W + s;
    if (!in_place || s != j0 + tid) {
      if (w_out) w_out[at] = p.weights[from];
      if (p_out) p_out[at] = p.positions ? p.positions[from] : s;
    }
  }
}

}  // namespace

int launch_cache_evict(const EvictParams& p, int kind, const LaunchCtx& ctx) {
  cache_evict_plan_kernel<<<dim3((unsigned)p.c.H, (unsigned)p.B), kPlanThreads, 0, ctx.stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) {
    const dim3 grid((unsigned)((p.keep + p.c.page - 1) / p.c.page), (unsigned)(2 * p.c.H), (unsigned)p.B);
    if (kind == FA_CACHE_E4M3)
      cache_evict_move_kernel<kKindE4m3><<<grid, 256, 0, ctx.stream>>>(p);
    else
      cache_evict_move_kernel<kKindInt8><<<grid, 256, 0, ctx.stream>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) {
    set_error("cache eviction launch failed: %s", cudaGetErrorString(e));
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // namespace fa
