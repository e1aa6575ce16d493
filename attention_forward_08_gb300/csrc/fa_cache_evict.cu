// fa_cache_evict.cu -- keep the heaviest and latest tokens (include/fa_cache.h).
//
// The choice: one thread block per sequence and head finds, byte by byte, the
// key of the last token that is kept (a radix selection: four passes over the
// weights' keys, each counting one byte of those that match the bytes found so
// far; the keys stay in shared memory where they fit), and writes for every
// slot below `keep` which slot's token ends there.  A copy into other blocks
// then moves by a second launch, one thread block per (sequence, head,
// receiving block of K or of V).
//
// In place, only tokens in slots at `keep` and behind move, and only into
// slots below `keep`: no slot is both read and written, so the moves need no
// order, and a decoding step that evicts one token moves one token, not a
// whole cache.  They are few: the block that chose makes them itself, a warp a
// receiving block.
//
// Bound: memory.  Choosing reads 8 bytes a token and head (weight, position);
// moving reads and writes 2 * D bytes per moved token and head.
#include <algorithm>
#include <atomic>
#include <climits>

#include "fa.h"
#include "fa_cache.h"
#include "fa_cache_launch.cuh"
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

// Tokens whose keys fit shared memory (192 KB).
constexpr int kCachedKeys = 49152;

// Sixteen stored bytes of scale `from`, rounded to scale `to`.
template <int kKind>
__device__ __forceinline__ uint4 rescale16(uint4 w, float from, float to) {
  if (from == to) return w;
  const float ratio = __fdiv_rn(from, to);
  uint32_t* u = &w.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[4];
    load8x4<kKind>(u[i], f);
    u[i] = round8x4<kKind>(__fmul_rn(f[0], ratio), __fmul_rn(f[1], ratio), __fmul_rn(f[2], ratio), __fmul_rn(f[3], ratio));
  }
  return w;
}

template <int kKind>
__global__ void __launch_bounds__(kPlanThreads) cache_evict_plan_kernel(const EvictParams p, int cached) {
  const CacheView& c = p.c;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long bh = (long long)b * c.H + h;
  extern __shared__ uint32_t s_key[];
  __shared__ int hist[256];
  __shared__ int part[kPlanWarps][4];
  __shared__ int s_max, s_digit, s_need;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int n = checked_len(c, p.lens[b]);
  if (n > p.W) {
    if (tid == 0) flag_bad_index(c);
    n = p.W;
  }
  int* src = p.src + bh * p.keep;
  if (tid == 0) {
    p.count[bh] = min(n, p.keep);
    if (!p.into && p.lens_out != p.lens && h == 0) p.lens_out[b] = min(n, p.keep);
    s_max = INT_MIN;
  }
  if (n <= p.keep) {  // all stay (a copy takes them all, in order)
    if (p.into)
      for (int j = tid; j < n; j += kPlanThreads) src[j] = j;
    return;
  }
  const float* weight = p.weights + bh * p.W;
  const int* position = p.positions ? p.positions + bh * p.W : nullptr;
  __syncthreads();
  const bool in_smem = n <= cached;
  if (p.recent > 0 || in_smem) {
    int most = position ? INT_MIN : n - 1;
#pragma unroll 4
    for (int j = tid; j < n; j += kPlanThreads) {
      if (in_smem) s_key[j] = weight_key(weight[j]);
      if (p.recent > 0 && position) most = max(most, position[j]);
    }
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) atomicMax(&s_max, most);
  }
  if (tid < 256) hist[tid] = 0;
  __syncthreads();
  // Positions above the bound are kept first (long: the bound may lie below INT_MIN).
  const long long late = p.recent > 0 ? (long long)s_max - p.recent : LLONG_MAX;
  const uint32_t first = weight_key(INFINITY);
  auto key_of = [&](int j) -> uint32_t {
    const long long pos = p.recent > 0 && position ? position[j] : j;
    return pos > late ? first : weight_key(weight[j]);
  };
  uint32_t found = 0;  // the bytes found so far
  int need = p.keep;   // tokens still to take among those that match them
  for (int shift = 24; shift >= 0; shift -= 8) {
    const uint32_t mask = shift == 24 ? 0u : ~0u << (shift + 8);
    const int stop = (n + kPlanThreads - 1) / kPlanThreads * kPlanThreads;
#pragma unroll 4
    for (int j = tid; j < stop; j += kPlanThreads) {
      uint32_t k = 0;
      bool in = j < n;
      if (in) {
        if (!in_smem) {
          k = key_of(j);
        } else if (shift == 24) {
          k = s_key[j];
          if (p.recent > 0 && (position ? position[j] : j) > late) s_key[j] = k = first;
        } else {
          k = s_key[j];
        }
        in = (k & mask) == found;
      }
      // Weights crowd into few exponents: lanes that agree count once.
      const uint32_t live = __ballot_sync(0xFFFFFFFFu, in);
      if (in) {
        const int digit = (k >> shift) & 255;
        const uint32_t same = __match_any_sync(live, digit);
        if (__ffs(same) - 1 == lane) atomicAdd(&hist[digit], __popc(same));
      }
    }
    __syncthreads();
    if (warp == 0) {  // the digit at which the count from above reaches `need`
      int mine = 0, at[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += at[i] = hist[255 - (lane * 8 + i)];
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += t;
      }
      int before = upto - mine;
      if (before < need && upto >= need) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < need && before + at[i] >= need) {
            s_digit = 255 - (lane * 8 + i);
            s_need = need - before;
          }
          before += at[i];
        }
      }
    }
    __syncthreads();
    found |= (uint32_t)s_digit << shift;
    need = s_need;
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
  }
  auto key = [&](int j) -> uint32_t { return in_smem ? s_key[j] : key_of(j); };
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
    const uint32_t k = key(j);
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
    const uint32_t k = in ? key(j) : 0;
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
  if (p.into) return;
  // The moves in place.  The block of slot `keep` may hold sources and receive
  // as well: its scales from before.
  __shared__ float s_edge[2];
  if (tid < 2) {
    const int blk = checked_block(c, c.table, c.table_stride, b, p.keep >> c.page_log2);
    s_edge[tid] = blk < 0 ? 0.0f : (tid ? c.v_scale : c.k_scale)[(long long)blk * c.H + h];
  }
  __syncthreads();
  const int blocks = (p.keep + c.page - 1) >> c.page_log2;
  for (int m = warp; m < blocks; m += kPlanWarps) {
    const int m0 = m << c.page_log2, tokens = min(c.page, p.keep - m0);
    bool moves = false;
    for (int t = lane; t < tokens; t += 32) moves = moves || src[m0 + t] < 0;
    if (!__any_sync(0xFFFFFFFFu, moves)) continue;
    const int to = checked_block(c, c.table, c.table_stride, b, m);
    if (to < 0) continue;
#pragma unroll 1
    for (int is_v = 0; is_v < 2; ++is_v) {
      float* scales = is_v ? c.v_scale : c.k_scale;
      const float old = scales[(long long)to * c.H + h];
      float top = 0.0f;
      for (int t = lane; t < tokens; t += 32) {  // the largest scale of the blocks that the tokens come from
        const int s = src[m0 + t];
        float sc = old;
        if (s < 0) {
          const int blk = checked_block(c, c.table, c.table_stride, b, mover[-1 - s] >> c.page_log2);
          sc = blk < 0 ? 0.0f
               : mover[-1 - s] >> c.page_log2 == p.keep >> c.page_log2 ? s_edge[is_v]
                                                                         : scales[(long long)blk * c.H + h];
        }
        top = fmaxf(top, sc);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      const long long* cs = is_v ? c.vs : c.ks;
      uint8_t* pool = (is_v ? c.v : c.k) + h * cs[1];
      const int vd = c.D >> 4, vd_log2 = 31 - __clz(vd);  // 16-byte vectors a token
      for (int v = lane; v < tokens * vd; v += 32) {
        const int t = v >> vd_log2, at = (v & (vd - 1)) * 16, s = src[m0 + t];
        uint4* dst = reinterpret_cast<uint4*>(pool + to * cs[0] + t * cs[2] + at);
        if (s >= 0) {  // stays; rounded anew where the scale grows
          if (old != top) *dst = rescale16<kKind>(*dst, old, top);
          continue;
        }
        const int from = mover[-1 - s], fm = from >> c.page_log2;
        const int blk = checked_block(c, c.table, c.table_stride, b, fm);
        if (blk < 0) continue;
        const float sc = fm == p.keep >> c.page_log2 ? s_edge[is_v] : scales[(long long)blk * c.H + h];
        *dst = rescale16<kKind>(
            *reinterpret_cast<const uint4*>(pool + blk * cs[0] + (from & (c.page - 1)) * cs[2] + at), sc, top);
      }
      __syncwarp();
      if (lane == 0) scales[(long long)to * c.H + h] = top;
    }
    for (int t = lane; t < tokens; t += 32) {
      const int s = src[m0 + t];
      if (s >= 0) continue;
      p.weights[bh * p.W + m0 + t] = weight[mover[-1 - s]];
      p.positions[bh * p.W + m0 + t] = position[mover[-1 - s]];
    }
  }
}

// Copies the tokens of one receiving block, or (past them) the lengths.
template <int kKind>
__global__ void __launch_bounds__(256) cache_evict_copy_kernel(const EvictParams p) {
  const CacheView& c = p.c;
  const int m = blockIdx.x, h = blockIdx.y % c.H, is_v = blockIdx.y / c.H, b = blockIdx.z, tid = threadIdx.x;
  const long long bh = (long long)b * c.H + h;
  const int j0 = m << c.page_log2;
  __shared__ const uint8_t* s_from[128];
  __shared__ float s_scale[128];
  __shared__ float s_top[4];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the choice is made
  const int count = p.count[bh];
  if (m == 0 && blockIdx.y == 0 && tid == 0) p.lens_out[b] = count;
  if (j0 >= count) return;
  const int tokens = min(c.page, count - j0);
  float* scales = is_v ? c.v_scale : c.k_scale;
  const long long* cs = is_v ? c.vs : c.ks;
  uint8_t* pool = (is_v ? c.v : c.k) + h * cs[1];
  float top = 0.0f;
  if (tid < tokens) {
    const int s = p.src[bh * p.keep + j0 + tid];
    const int blk = checked_block(c, c.table, c.table_stride, b, s >> c.page_log2);
    s_from[tid] = blk >= 0 ? pool + blk * cs[0] + (s & (c.page - 1)) * cs[2] : nullptr;
    s_scale[tid] = top = blk >= 0 ? scales[(long long)blk * c.H + h] : 0.0f;
    if (!is_v) {
      const long long at = bh * p.W_out + j0 + tid, from = bh * p.W + s;
      if (p.weights_out) p.weights_out[at] = p.weights[from];
      if (p.positions_out) p.positions_out[at] = p.positions ? p.positions[from] : s;
    }
  }
  if (tid < 128) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if ((tid & 31) == 0) s_top[tid >> 5] = top;
  }
  __syncthreads();
  top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
  const int to = checked_block(c, p.into, p.into_stride, b, m);
  if (to < 0) return;
  uint8_t* out = pool + to * cs[0];
  const int vd = c.D >> 4, vd_log2 = 31 - __clz(vd);  // 16-byte vectors a token
#pragma unroll 4
  for (int v = tid; v < tokens * vd; v += 256) {
    const int t = v >> vd_log2, at = (v & (vd - 1)) * 16;
    if (!s_from[t]) continue;
    const uint4 w = *reinterpret_cast<const uint4*>(s_from[t] + at);
    *reinterpret_cast<uint4*>(out + t * cs[2] + at) = rescale16<kKind>(w, s_scale[t], top);
  }
  if (tid == 0) scales[(long long)to * c.H + h] = top;
}

// In place, and lens itself is to change: once every head has read it.
__global__ void cache_evict_lens_kernel(const EvictParams p) {
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (b < p.B) p.lens_out[b] = p.count[(long long)b * p.c.H];
}

template <int kKind>
int launch(const EvictParams& p, const LaunchCtx& ctx) {
  auto plan = cache_evict_plan_kernel<kKind>;
  static std::atomic<unsigned long long> configured{0};
  if (!allow_smem(plan, kCachedKeys * 4, ctx.dev, configured)) return FA_ERR_CUDA;
  // Shared memory for the keys that a head can have.
  const long long most = std::min((long long)p.c.M * p.c.page, (long long)p.W);
  const int cached = most <= kCachedKeys ? (int)most : kCachedKeys;
  plan<<<dim3((unsigned)p.c.H, (unsigned)p.B), kPlanThreads, (size_t)cached * 4, ctx.stream>>>(p, cached);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) {
    if (p.into)
      e = launch_after(cache_evict_copy_kernel<kKind>,
                       dim3((unsigned)((p.keep + p.c.page - 1) / p.c.page), (unsigned)(2 * p.c.H), (unsigned)p.B), 256,
                       ctx.stream, p);
    else if (p.lens_out == p.lens)
      e = launch_after(cache_evict_lens_kernel, dim3((unsigned)((p.B + 127) / 128)), 128, ctx.stream, p);
  }
  if (e != cudaSuccess) {
    set_error("cache eviction launch failed: %s", cudaGetErrorString(e));
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // namespace

int launch_cache_evict(const EvictParams& p, int kind, const LaunchCtx& ctx) {
  return kind == FA_CACHE_E4M3 ? launch<kKindE4m3>(p, ctx) : launch<kKindInt8>(p, ctx);
}

}  // namespace fa
