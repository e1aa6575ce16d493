// fa_cache_accept.cu -- the accepted drafts become a sequence's next tokens
// (include/fa_cache.h).
//
// An accepted path's tokens move down, in order: the one in slot base + path[i]
// to slot base + i <= base + path[i].  One thread block for K and one for V of
// each sequence and head goes over the receiving blocks in ascending order; it
// holds all that a block receives in registers before it writes there, so that
// a slot may give and receive in one block, and a later block's sources are
// never behind an earlier block's slots.
//
// Bound: latency; a block does one chain of loads (length and path, table,
// scales, bytes) a receiving cache block, and few tokens move.
#include "fa.h"
#include "fa_cache.h"
#include "fa_cache_launch.cuh"
#include "fa_cache_ops.cuh"
#include "fa_cache_rescale.cuh"
#include "fa_device.h"

namespace fa {
namespace {

constexpr int kAcceptThreads = 256;

struct Accepted {
  int held, base, count;  // tokens before the call; the first draft's slot; drafts that stay
};

// Sequence b's numbers, and its path in shared memory; the whole thread block.
// A path that does not ascend, or leaves the drafts, ends before that entry.
__device__ __forceinline__ Accepted accepted(const AcceptParams& p, int b, int* s_path, int* s_end) {
  Accepted r;
  r.held = checked_len(p.c, p.lens[b]);
  int nq = p.n_q ? p.n_q[b] : p.n, count = p.count[b];
  if (nq < 0 || nq > p.n || nq > r.held || count < 0 || count > nq) {
    if (threadIdx.x == 0) flag_bad_index(p.c);
    if (nq < 0 || nq > p.n || nq > r.held) {  // the drafts are not there: nothing is done
      r.base = r.held;
      r.count = 0;
      return r;
    }
    count = count < 0 ? 0 : nq;
  }
  r.base = r.held - nq;
  if (threadIdx.x == 0) *s_end = count;
  __syncthreads();
  const int* path = p.path + b * p.path_stride;
  for (int i = threadIdx.x; i < count; i += kAcceptThreads) {
    const int at = path[i];
    if (at >= nq || at <= (i ? path[i - 1] : -1)) atomicMin(s_end, i);
    s_path[i] = at;
  }
  __syncthreads();
  r.count = *s_end;
  if (r.count != count && threadIdx.x == 0) flag_bad_index(p.c);
  return r;
}

template <int kKind>
__global__ void __launch_bounds__(kAcceptThreads) cache_accept_kernel(const AcceptParams p) {
  const CacheView& c = p.c;
  const int is_v = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  extern __shared__ int s_path[];  // n
  __shared__ int s_end, s_first;
  __shared__ unsigned s_top;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Accepted a = accepted(p, b, s_path, &s_end);
  if (tid == 0) {
    s_first = a.count;
    if (is_v == 0 && h == 0 && p.lens_out != p.lens) p.lens_out[b] = a.base + a.count;
  }
  __syncthreads();
  for (int i = tid; i < a.count; i += kAcceptThreads)
    if (s_path[i] != i) atomicMin(&s_first, i);
  __syncthreads();
  const int first = s_first;
  if (first >= a.count) return;

  float* scales = is_v ? c.v_scale : c.k_scale;
  const long long* cs = is_v ? c.vs : c.ks;
  uint8_t* pool = (is_v ? c.v : c.k) + h * cs[1];
  const int vd = c.D >> 4, vd_log2 = 31 - __clz(vd);  // 16-byte vectors a token
  constexpr int kMost = 128 * 16 / kAcceptThreads;    // a thread's vectors of a receiving block
#pragma unroll 1
  for (int m = (a.base + first) >> c.page_log2; m <= (a.base + a.count - 1) >> c.page_log2; ++m) {
    const int m0 = m << c.page_log2, i0 = max(first, m0 - a.base), n = min(a.count, m0 + c.page - a.base) - i0;
    const int stay = a.base + i0 - m0;  // tokens of the block that stay in it, before those that come
    const int to = checked_block(c, c.table, c.table_stride, b, m);
    const float old = to < 0 ? 0.0f : scales[(long long)to * c.H + h];
    if (tid == 0) s_top = stay > 0 ? __float_as_uint(old) : 0u;  // (scales are >= 0: the order of bits)
    __syncthreads();
    // What comes, and its blocks' scales: read before anything is written.
    uint4 x[kMost];
    float from[kMost];
    bool comes[kMost];
#pragma unroll
    for (int u = 0; u < kMost; ++u) {
      const int v = tid + u * kAcceptThreads, i = v >> vd_log2;
      comes[u] = false;
      if (i < n && to >= 0) {
        const int slot = a.base + s_path[i0 + i];
        const int blk = checked_block(c, c.table, c.table_stride, b, slot >> c.page_log2);
        if (blk >= 0) {
          comes[u] = true;
          from[u] = scales[(long long)blk * c.H + h];
          x[u] = *reinterpret_cast<const uint4*>(pool + blk * cs[0] + (slot & (c.page - 1)) * cs[2] + (v & (vd - 1)) * 16);
          if ((v & (vd - 1)) == 0) atomicMax(&s_top, __float_as_uint(from[u]));
        }
      }
    }
    __syncthreads();
    const float top = __uint_as_float(s_top);
    if (to >= 0) {
      uint8_t* out = pool + to * cs[0];
      if (top != old) {
        for (int v = tid; v < stay * vd; v += kAcceptThreads) {
          uint4* at = reinterpret_cast<uint4*>(out + (v >> vd_log2) * cs[2] + (v & (vd - 1)) * 16);
          *at = rescale16<kKind>(*at, old, top);
        }
      }
#pragma unroll
      for (int u = 0; u < kMost; ++u) {
        const int v = tid + u * kAcceptThreads;
        if (comes[u])
          *reinterpret_cast<uint4*>(out + (stay + (v >> vd_log2)) * cs[2] + (v & (vd - 1)) * 16) =
              rescale16<kKind>(x[u], from[u], top);
      }
      if (tid == 0) scales[(long long)to * c.H + h] = top;
    }
    __syncthreads();
  }
  if (p.weights && is_v == 0) {
    float* w = p.weights + ((long long)b * c.H + h) * p.W;
    for (int i0 = first; i0 < a.count; i0 += kAcceptThreads) {
      const int i = i0 + tid, slot = i < a.count ? a.base + s_path[i] : 0;
      const bool in = i < a.count && slot < p.W;
      float x = 0.0f;
      if (in) x = w[slot];
      if (i < a.count && !in) flag_bad_index(c);
      __syncthreads();
      if (in) w[a.base + i] = x;
      __syncthreads();
    }
  }
}

// lens itself is to change: once every head has read it.
__global__ void __launch_bounds__(kAcceptThreads) cache_accept_lens_kernel(const AcceptParams p) {
  extern __shared__ int s_path[];
  __shared__ int s_end;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Accepted a = accepted(p, blockIdx.x, s_path, &s_end);
  __syncthreads();
  if (threadIdx.x == 0) p.lens_out[blockIdx.x] = a.base + a.count;
}

}  // namespace

int launch_cache_accept(const AcceptParams& p, int kind, const LaunchCtx& ctx) {
  const dim3 grid(2, (unsigned)p.c.H, (unsigned)p.B);
  const size_t smem = (size_t)p.n * 4;
  if (kind == FA_CACHE_E4M3)
    cache_accept_kernel<kKindE4m3><<<grid, kAcceptThreads, smem, ctx.stream>>>(p);
  else
    cache_accept_kernel<kKindInt8><<<grid, kAcceptThreads, smem, ctx.stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && p.lens_out == p.lens)
    e = launch_after_with(smem, cache_accept_lens_kernel, dim3((unsigned)p.B), kAcceptThreads, ctx.stream, p);
  if (e != cudaSuccess) {
    set_error("cache acceptance launch failed: %s", cudaGetErrorString(e));
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // namespace fa
