// fa_cache_evict.cu -- keep the heaviest and latest tokens (include/fa_cache.h).
//
// The choice: one thread block per sequence and head finds the key of the last
// token that is kept, and writes for every slot below `keep` which slot's token
// ends there.  Keys that are not protected are counted in 2048 classes that
// split their own range evenly, so that weights spread over the classes
// whatever their size (classes by leading bits would hold a few exponents, and
// their counters cost 15,000 cycles in atomics at 2049 tokens); the class in
// which the count from above reaches `keep` is settled by comparing its keys
// with one another where they are few, else split again (three times at most:
// 11 of 32 bits each).  The keys stay in shared memory where they fit.  A copy
// into other blocks then moves by a second launch, one thread block per
// (sequence, head, receiving block).
//
// In place, only tokens in slots at `keep` and behind move, and only into
// slots below `keep`: no slot is both read and written, so the moves need no
// order, and a decoding step that evicts one token moves one token, not a
// whole cache.  They are few: the block that chose makes them itself, a warp a
// receiving block.
//
// Bound: memory.  Choosing reads 8 bytes a token and head (weight, position);
// moving reads and writes 2 * D bytes per moved token and head.  Choosing is not
// near that: one block a head goes over its keys up to four times, each a
// barrier's latency apart (18 us for 64 heads of 16000 tokens).
#include <algorithm>
#include <atomic>
#include <climits>

#include "fa.h"
#include "fa_cache.h"
#include "fa_cache_launch.cuh"
#include "fa_cache_ops.cuh"
#include "fa_cache_rescale.cuh"
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

constexpr int kFewMoves = 1024;  // in place: lists in shared memory, else in the workspace
// Tokens whose keys fit shared memory (184 KB).
constexpr int kCachedKeys = 47104;

constexpr int kClasses = 2048, kFewKeys = 256;

struct PlanShared {
  int count[kClasses];
  uint32_t few[kFewKeys];
  int part[kPlanWarps][4];
  int hole[kFewMoves], mover[kFewMoves];
  int latest, n_few, total;
  uint32_t least, most, digit_over;  // range of the keys; the class found
  int over, inside;
  uint32_t found;
  int need;
  float edge[2];
};

// The choice for one head of n > keep tokens; kCached: the keys fit `s_key`.
// Returns the number of moves (in place), whose slots are in `s` if few, else
// in `src` and `mover`; of a copy, `src` is the answer.
template <bool kCached>
__device__ __forceinline__ int choose(const EvictParams& p, PlanShared& s, uint32_t* s_key, int n, const float* weight,
                                      const int* position, int* src, int* mover) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t first = ~0u;  // of protected tokens: above any weight's, +inf's too
  const int stop = (n + 31) & ~31;  // (whole warps stay together)
  for (int i = tid; i < kClasses; i += kPlanThreads) s.count[i] = 0;
  if (tid == 0) {
    s.latest = INT_MIN;
    s.n_few = s.total = 0;
    s.least = ~0u;
    s.most = 0u;
  }
  __syncthreads();
  if (kCached || p.recent > 0) {
    int most = position ? INT_MIN : n - 1;
#pragma unroll 4
    for (int j = tid; j < n; j += kPlanThreads) {
      if (kCached) s_key[j] = weight_key(weight[j]);
      if (p.recent > 0 && position) most = max(most, position[j]);
    }
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) atomicMax(&s.latest, most);
    __syncthreads();
  }
  // Positions above the bound are kept first (long: the bound may lie below INT_MIN).
  const long long late = p.recent > 0 ? (long long)s.latest - p.recent : LLONG_MAX;
  auto key_of = [&](int j) -> uint32_t {
    const long long pos = p.recent > 0 && position ? position[j] : j;
    return pos > late ? first : weight_key(weight[j]);
  };
  auto key = [&](int j) -> uint32_t { return kCached ? s_key[j] : key_of(j); };
  {  // protected tokens, and the others' range
    uint32_t least = ~0u, most = 0u;
    int sure = 0;
#pragma unroll 4
    for (int j = tid; j < n; j += kPlanThreads) {
      uint32_t k;
      if (kCached) {
        k = s_key[j];
        if (p.recent > 0 && (position ? position[j] : j) > late) s_key[j] = k = first;
      } else {
        k = key_of(j);
      }
      if (k == first) {
        ++sure;
      } else {
        least = min(least, k);
        most = max(most, k);
      }
    }
    least = __reduce_min_sync(0xFFFFFFFFu, least);
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    sure = __reduce_add_sync(0xFFFFFFFFu, sure);
    if (lane == 0) {
      atomicMin(&s.least, least);
      atomicMax(&s.most, most);
      atomicAdd(&s.total, sure);
    }
    __syncthreads();
  }
  // Kept: keys above `found`, and the first `need` slots whose key equals it.
  uint32_t found = first;
  int need = p.keep;
  if (s.total < p.keep) {
    uint32_t lo = s.least;                               // the key sought lies in lo .. lo + width
    int bits = 32 - __clz(s.most - lo), over = s.total;  // width < 2^bits; keys above the range
#pragma unroll 1
    while (true) {
      const int shift = max(bits - 11, 0);
      const uint32_t width = bits == 32 ? ~0u : (1u << bits) - 1u;
#pragma unroll 4
      for (int j = tid; j < stop; j += kPlanThreads) {
        const uint32_t k = j < n ? key(j) : first, at = (k - lo) >> shift;
        const bool in = k >= lo && k - lo <= width && k != first;
        // (ties crowd into a class: lanes that all agree count once)
        const uint32_t here = in ? at : ~0u, lead = __shfl_sync(0xFFFFFFFFu, here, 0);
        if (__all_sync(0xFFFFFFFFu, here == lead)) {
          if (lane == 0 && in) atomicAdd(&s.count[at], 32);
        } else if (in) {
          atomicAdd(&s.count[at], 1);
        }
      }
      __syncthreads();
      // The class at which the count from above reaches `keep`: two a thread.
      const int c1 = kClasses - 1 - 2 * tid, upper = s.count[c1], lower = s.count[c1 - 1];
      int upto = upper + lower;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += t;
      }
      if (lane == 31) s.part[warp][0] = upto;
      __syncthreads();
      s.count[c1] = s.count[c1 - 1] = 0;
      const int before = over + __reduce_add_sync(0xFFFFFFFFu, lane < warp ? s.part[lane][0] : 0) + upto - upper - lower;
      if (before < p.keep && before + upper + lower >= p.keep) {
        const bool second = before + upper < p.keep;
        s.digit_over = (uint32_t)(second ? c1 - 1 : c1);
        s.over = second ? before + upper : before;
        s.inside = second ? lower : upper;
      }
      __syncthreads();
      lo += s.digit_over << shift;
      over = s.over;
      const int inside = s.inside;
      bits = shift;
      if (bits == 0) {  // one key is left
        found = lo;
        need = p.keep - over;
        break;
      }
      if (inside <= kFewKeys) {  // compare its keys with one another
#pragma unroll 4
        for (int j = tid; j < n; j += kPlanThreads) {
          const uint32_t k = key(j);
          if (k >= lo && k != first && (k - lo) >> shift == 0u) s.few[atomicAdd(&s.n_few, 1)] = k;
        }
        __syncthreads();
        if (tid < inside) {
          const uint32_t k = s.few[tid];
          int above = 0, equal = 0;
          for (int i = 0; i < inside; ++i) {
            above += s.few[i] > k;
            equal += s.few[i] == k;
          }
          if (over + above < p.keep && over + above + equal >= p.keep) {  // (all that find it find the same)
            s.found = k;
            s.need = p.keep - over - above;
          }
        }
        __syncthreads();
        found = s.found;
        need = s.need;
        break;
      }
    }
  }
  // Every warp owns a run of slots; a first sweep counts what lies before it.
  // In place, with `kept_lo` of the slots below `keep` kept: the slot j that
  // becomes free is hole number j - (kept slots before j), and a kept slot at
  // `keep` or behind is mover number (kept slots before it) - kept_lo; hole i
  // takes mover i.
  const int run = ((n + kPlanThreads - 1) / kPlanThreads) * 32;
  const int j0 = warp * run, j1 = min(n, j0 + run);
  int above = 0, equal = 0, above_lo = 0, equal_lo = 0;
#pragma unroll 4
  for (int j = j0 + lane; j < j1; j += 32) {
    const uint32_t k = key(j);
    const int lo = j < p.keep ? 1 : 0, a = k > found ? 1 : 0, e = k == found ? 1 : 0;
    above += a;
    equal += e;
    above_lo += a & lo;
    equal_lo += e & lo;
  }
  above = __reduce_add_sync(0xFFFFFFFFu, above);
  equal = __reduce_add_sync(0xFFFFFFFFu, equal);
  above_lo = __reduce_add_sync(0xFFFFFFFFu, above_lo);
  equal_lo = __reduce_add_sync(0xFFFFFFFFu, equal_lo);
  if (lane == 0) *reinterpret_cast<int4*>(s.part[warp]) = make_int4(above, equal, above_lo, equal_lo);
  __syncthreads();
  const int4 their = *reinterpret_cast<const int4*>(s.part[lane]);
  int eq = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? their.y : 0);
  int kept_n = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? their.x : 0) + min(eq, need);
  const int kept_lo = __reduce_add_sync(0xFFFFFFFFu, their.z) + min(__reduce_add_sync(0xFFFFFFFFu, their.w), need);
  const int moves = p.keep - kept_lo;
  const bool few = moves <= kFewMoves;
  const uint32_t below = (1u << lane) - 1;
  for (int base = j0; base < j1; base += 128) {
    uint32_t k4[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) k4[u] = base + 32 * u + lane < j1 ? key(base + 32 * u + lane) : 0u;  // (0: below all)
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = base + 32 * u + lane;
      const bool in = j < j1;
      const uint32_t k = k4[u], e = __ballot_sync(0xFFFFFFFFu, in && k == found);
      const bool kept = in && (k > found || (k == found && eq + __popc(e & below) < need));
      const uint32_t kb = __ballot_sync(0xFFFFFFFFu, kept);
      const int at = kept_n + __popc(kb & below);  // kept slots before j
      if (p.into) {
        if (kept) src[at] = j;
      } else if (in && j < p.keep) {
        if (!kept) (few ? s.hole : src)[j - at] = j;
      } else if (kept) {
        (few ? s.mover : mover)[at - kept_lo] = j;
      }
      kept_n += __popc(kb);
      eq += __popc(e);
    }
  }
  return moves;
}

template <int kKind>
__global__ void __launch_bounds__(kPlanThreads) cache_evict_plan_kernel(const EvictParams p, int cached) {
  const CacheView& c = p.c;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long bh = (long long)b * c.H + h;
  extern __shared__ uint32_t s_key[];
  __shared__ __align__(16) PlanShared s;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int n = checked_len(c, p.lens[b]);
  if (n > p.W) {
    if (tid == 0) flag_bad_index(c);
    n = p.W;
  }
  int* src = p.src + bh * p.keep;
  int* mover = p.mover + bh * p.keep;
  if (tid == 0) {
    p.count[bh] = min(n, p.keep);
    if (!p.into && p.lens_out != p.lens && h == 0) p.lens_out[b] = min(n, p.keep);
  }
  if (n <= p.keep) {  // all stay (a copy takes them all, in order)
    if (p.into)
      for (int j = tid; j < n; j += kPlanThreads) src[j] = j;
    return;
  }
  const float* weight = p.weights + bh * p.W;
  const int* position = p.positions ? p.positions + bh * p.W : nullptr;
  const int moves = n <= cached ? choose<true>(p, s, s_key, n, weight, position, src, mover)
                                : choose<false>(p, s, s_key, n, weight, position, src, mover);
  if (p.into) return;
  // The moves in place.  The block of slot `keep` may hold sources and receive
  // as well: its scales from before.
  if (tid < 2) {
    const int blk = checked_block(c, c.table, c.table_stride, b, p.keep >> c.page_log2);
    s.edge[tid] = blk < 0 ? 0.0f : (tid ? c.v_scale : c.k_scale)[(long long)blk * c.H + h];
  }
  __syncthreads();
  const bool few = moves <= kFewMoves;
  auto hole_at = [&](int i) { return few ? s.hole[i] : src[i]; };
  auto mover_at = [&](int i) { return few ? s.mover[i] : mover[i]; };
  // A warp takes the moves into one block, of K or of V, from the first of them.
  for (int w = warp; w < 2 * moves; w += kPlanWarps) {
    const int i0 = w >> 1, is_v = w & 1, m = hole_at(i0) >> c.page_log2;
    if (i0 > 0 && hole_at(i0 - 1) >> c.page_log2 == m) continue;
    const int to = checked_block(c, c.table, c.table_stride, b, m);
    if (to < 0) continue;
    float* scales = is_v ? c.v_scale : c.k_scale;
    const float old = scales[(long long)to * c.H + h];
    // A mover's scale; of the block of slot `keep`, the one from before.
    auto scale_of = [&](int from, int& blk) -> float {
      const int fm = from >> c.page_log2;
      blk = checked_block(c, c.table, c.table_stride, b, fm);
      return blk < 0 ? 0.0f : fm == p.keep >> c.page_log2 ? s.edge[is_v] : scales[(long long)blk * c.H + h];
    };
    // The largest scale of the blocks that the block's tokens come from, its
    // own among them unless all its tokens are new.
    const int m0 = m << c.page_log2, tokens = min(c.page, p.keep - m0);
    int n = 0;  // moves into it
    float top = 0.0f;
    for (int base = i0;; base += 32) {
      const int i = base + lane;
      const bool here = i < moves && hole_at(i) >> c.page_log2 == m;
      int blk;
      if (here) top = fmaxf(top, scale_of(mover_at(i), blk));
      const int got = __popc(__ballot_sync(0xFFFFFFFFu, here));
      n += got;
      if (got < 32) break;
    }
    if (n < tokens) top = fmaxf(top, old);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    const long long* cs = is_v ? c.vs : c.ks;
    uint8_t* pool = (is_v ? c.v : c.k) + h * cs[1];
    uint8_t* out = pool + to * cs[0];
    const int vd = c.D >> 4, vd_log2 = 31 - __clz(vd);  // 16-byte vectors a token
    if (n < tokens && top != old) {  // what stays (and what is about to be overwritten) moves to the larger scale
      for (int v = lane; v < tokens * vd; v += 32) {
        uint4* at = reinterpret_cast<uint4*>(out + (v >> vd_log2) * cs[2] + (v & (vd - 1)) * 16);
        *at = rescale16<kKind>(*at, old, top);
      }
      __syncwarp();
    }
    for (int v = lane; v < n * vd; v += 32) {
      const int i = i0 + (v >> vd_log2), at = (v & (vd - 1)) * 16, from = mover_at(i);
      int blk;
      const float sc = scale_of(from, blk);
      if (blk < 0) continue;
      *reinterpret_cast<uint4*>(out + (hole_at(i) - m0) * cs[2] + at) = rescale16<kKind>(
          *reinterpret_cast<const uint4*>(pool + blk * cs[0] + (from & (c.page - 1)) * cs[2] + at), sc, top);
    }
    __syncwarp();
    if (lane == 0) scales[(long long)to * c.H + h] = top;
  }
  for (int i = tid; i < moves; i += kPlanThreads) {
    p.weights[bh * p.W + hole_at(i)] = weight[mover_at(i)];
    p.positions[bh * p.W + hole_at(i)] = position[mover_at(i)];
  }
}

// Copies the tokens of one receiving block, K and V.  Each token's bytes lie
// behind three loads (its slot, the block there, the scale), so that what
// counts is how many blocks wait at a time: 8 an SM, with one pair of vectors a
// thread in flight, 31.9 us for the whole eviction (8 x 16000 tokens, 8 heads of
// 128, keep 2048); 5 an SM with two pairs 34.7.
template <int kKind>
__global__ void __launch_bounds__(256, 8) cache_evict_copy_kernel(const EvictParams p) {
  const CacheView& c = p.c;
  const int m = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long bh = (long long)b * c.H + h;
  const int j0 = m << c.page_log2;
  __shared__ int s_blk[128], s_row[128];
  __shared__ float2 s_scale[128];
  __shared__ float2 s_top[4];
  const int to = m < p.M_into ? checked_block_quiet(c, p.into, p.into_stride, b, m) : -1;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the choice is made
  const int count = p.count[bh];
  if (m == 0 && h == 0 && tid == 0) p.lens_out[b] = count;
  if (j0 >= count) return;
  if (to < 0) {
    if (tid == 0) flag_bad_index(c);
    return;
  }
  const int tokens = min(c.page, count - j0);
  float2 top = make_float2(0.0f, 0.0f);
  int from = 0;
  if (tid < tokens) {
    from = p.src[bh * p.keep + j0 + tid];
    const int blk = checked_block(c, c.table, c.table_stride, b, from >> c.page_log2);
    s_blk[tid] = blk;
    s_row[tid] = from & (c.page - 1);
    if (blk >= 0) top = make_float2(c.k_scale[(long long)blk * c.H + h], c.v_scale[(long long)blk * c.H + h]);
    s_scale[tid] = top;
  }
  if (warp < 4) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      top.x = fmaxf(top.x, __shfl_xor_sync(0xFFFFFFFFu, top.x, o));
      top.y = fmaxf(top.y, __shfl_xor_sync(0xFFFFFFFFu, top.y, o));
    }
    if (lane == 0) s_top[warp] = top;
  }
  __syncthreads();
  top = s_top[0];
#pragma unroll
  for (int w = 1; w < 4; ++w) top = make_float2(fmaxf(top.x, s_top[w].x), fmaxf(top.y, s_top[w].y));
  const uint8_t *k_in = c.k + h * c.ks[1], *v_in = c.v + h * c.vs[1];
  uint8_t *k_out = c.k + to * c.ks[0] + h * c.ks[1], *v_out = c.v + to * c.vs[0] + h * c.vs[1];
  const int vd = c.D >> 4, vd_log2 = 31 - __clz(vd);  // 16-byte vectors a token
#pragma unroll 1
  for (int v = tid; v < tokens * vd; v += 256) {
    const int t = v >> vd_log2, at = (v & (vd - 1)) * 16;
    const long long blk = s_blk[t], row = s_row[t];
    if (blk < 0) continue;
    const uint4 x = *reinterpret_cast<const uint4*>(k_in + blk * c.ks[0] + row * c.ks[2] + at);
    const uint4 y = *reinterpret_cast<const uint4*>(v_in + blk * c.vs[0] + row * c.vs[2] + at);
    *reinterpret_cast<uint4*>(k_out + t * c.ks[2] + at) = rescale16<kKind>(x, s_scale[t].x, top.x);
    *reinterpret_cast<uint4*>(v_out + t * c.vs[2] + at) = rescale16<kKind>(y, s_scale[t].y, top.y);
  }
  if (tid == 0) {
    c.k_scale[(long long)to * c.H + h] = top.x;
    c.v_scale[(long long)to * c.H + h] = top.y;
  }
  if (tid < tokens) {
    const long long at = bh * p.W_out + j0 + tid, src = bh * p.W + from;
    if (p.weights_out) p.weights_out[at] = p.weights[src];
    if (p.positions_out) p.positions_out[at] = p.positions ? p.positions[src] : from;
  }
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
                       dim3((unsigned)((p.keep + p.c.page - 1) / p.c.page), (unsigned)p.c.H, (unsigned)p.B), 256,
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
