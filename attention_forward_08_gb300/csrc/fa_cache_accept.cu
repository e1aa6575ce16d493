// fa_cache_accept.cu -- the accepted drafts become a sequence's next tokens
// (include/fa_cache.h).
//
// An accepted path's tokens move down, in order: the one in slot base + path[i]
// to slot base + i <= base + path[i].  One thread block for K and one for V of
// each sequence and head reads all block numbers and scales first (no block's
// scale changes before the end), then moves 32 KB at a time in ascending order:
// into registers, and out when all of it is there.  A slot may so give and
// receive, and later sources are never behind earlier slots.
//
// Bound: latency; a chain of five loads (length and count, path, table, scales,
// bytes) and few tokens: 32 sequences of 16 drafts, 8 heads of 128, 7.1 us; 64 of 200,
// 8 heads of 256, blocks of 16, 13.1 us (26.8 a receiving block at a time).
#include "fa.h"
#include "fa_cache.h"
#include "fa_cache_launch.cuh"
#include "fa_cache_ops.cuh"
#include "fa_cache_rescale.cuh"
#include "fa_device.h"

namespace fa {
namespace {

constexpr int kAcceptThreads = 256, kAcceptMost = 8;  // 16-byte vectors that a thread moves at a time

struct Accepted {
  int held, base, count;  // tokens before the call; the first draft's slot; drafts that stay
};

// Sequence b's numbers, and its path in shared memory; the whole thread block.
// A path that does not ascend, or leaves the drafts, ends before that entry; so
// does one that reaches a draft behind the table, which nothing has stored.
__device__ __forceinline__ Accepted accepted(const AcceptParams& p, int b, int* s_path, int* s_end) {
  Accepted r;
  const int len = p.lens[b];
  r.held = checked_len(p.c, len);
  int nq = p.n_q ? p.n_q[b] : p.n, count = p.count[b];
  if (nq < 0 || nq > p.n || nq > len || count < 0 || count > nq) {
    if (threadIdx.x == 0) flag_bad_index(p.c);
    if (nq < 0 || nq > p.n || nq > len) {  // the drafts are not there: nothing is done
      r.base = r.held;
      r.count = 0;
      return r;
    }
    count = count < 0 ? 0 : nq;
  }
  r.base = min(len - nq, r.held);
  const int stored = r.held - r.base;  // drafts that the table has room for: all, but for a length past it
  if (threadIdx.x == 0) *s_end = count;
  __syncthreads();
  const int* path = p.path + b * p.path_stride;
  for (int i = threadIdx.x; i < count; i += kAcceptThreads) {
    const int at = path[i];
    if (at >= stored || at <= (i ? path[i - 1] : -1)) atomicMin(s_end, i);
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
  int* const s_from_block = s_path + p.n;  // the block that a draft comes from (-1: it does not come), its scale
  float* const s_from = reinterpret_cast<float*>(s_path + 2 * p.n);
  int* const s_to = s_path + 3 * p.n;  // the receiving blocks, from the first on, and their new scales
  unsigned* const s_top = reinterpret_cast<unsigned*>(s_path + 4 * p.n + 1);
  __shared__ int s_end, s_first;
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
  const int slot0 = a.base + first, m0 = slot0 >> c.page_log2, blocks = ((a.base + a.count - 1) >> c.page_log2) - m0 + 1;
  const int stay = slot0 & (c.page - 1);  // tokens of the first block that stay in it, before those that come
  // The receiving blocks, the sources, and the scales of both.
  float old = 0.0f;
  for (int m = tid; m < blocks; m += kAcceptThreads) {
    s_to[m] = checked_block(c, c.table, c.table_stride, b, m0 + m);
    s_top[m] = 0u;
  }
  if (stay > 0) {
    const int to = checked_block(c, c.table, c.table_stride, b, m0);
    old = to < 0 ? 0.0f : scales[(long long)to * c.H + h];
  }
  __syncthreads();
  for (int i = first + tid; i < a.count; i += kAcceptThreads) {
    const int blk = checked_block(c, c.table, c.table_stride, b, (a.base + s_path[i]) >> c.page_log2);
    const int m = ((a.base + i) >> c.page_log2) - m0;
    s_from_block[i] = s_to[m] < 0 ? -1 : blk;
    if (blk >= 0) {
      s_from[i] = scales[(long long)blk * c.H + h];
      atomicMax(s_top + m, __float_as_uint(s_from[i]));  // (scales are >= 0: the order of bits)
    }
  }
  if (tid == 0 && stay > 0) atomicMax(s_top, __float_as_uint(old));
  __syncthreads();
  if (stay > 0 && s_to[0] >= 0 && __uint_as_float(s_top[0]) != old) {
    uint8_t* out = pool + s_to[0] * cs[0];
    for (int v = tid; v < stay * vd; v += kAcceptThreads) {
      uint4* at = reinterpret_cast<uint4*>(out + (v >> vd_log2) * cs[2] + (v & (vd - 1)) * 16);
      *at = rescale16<kKind>(*at, old, __uint_as_float(s_top[0]));
    }
  }
#pragma unroll 1
  for (int v0 = first << vd_log2; v0 < a.count << vd_log2; v0 += kAcceptMost * kAcceptThreads) {
    uint4 x[kAcceptMost];
#pragma unroll
    for (int u = 0; u < kAcceptMost; ++u) {
      const int v = v0 + tid + u * kAcceptThreads, i = v >> vd_log2;
      if (i < a.count && s_from_block[i] >= 0)
        x[u] = *reinterpret_cast<const uint4*>(pool + s_from_block[i] * cs[0] + ((a.base + s_path[i]) & (c.page - 1)) * cs[2] +
                                               (v & (vd - 1)) * 16);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kAcceptMost; ++u) {
      const int v = v0 + tid + u * kAcceptThreads, i = v >> vd_log2, slot = a.base + i;
      if (i < a.count && s_from_block[i] >= 0) {
        const int m = (slot >> c.page_log2) - m0;
        *reinterpret_cast<uint4*>(pool + s_to[m] * cs[0] + (slot & (c.page - 1)) * cs[2] + (v & (vd - 1)) * 16) =
            rescale16<kKind>(x[u], s_from[i], __uint_as_float(s_top[m]));
      }
    }
  }
  for (int m = tid; m < blocks; m += kAcceptThreads)
    if (s_to[m] >= 0) scales[(long long)s_to[m] * c.H + h] = __uint_as_float(s_top[m]);
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
  const size_t smem = (size_t)p.n * 20 + 8, smem_lens = (size_t)p.n * 4;
  if (kind == FA_CACHE_E4M3)
    cache_accept_kernel<kKindE4m3><<<grid, kAcceptThreads, smem, ctx.stream>>>(p);
  else
    cache_accept_kernel<kKindInt8><<<grid, kAcceptThreads, smem, ctx.stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && p.lens_out == p.lens)
    e = launch_after_with(smem_lens, cache_accept_lens_kernel, dim3((unsigned)p.B), kAcceptThreads, ctx.stream, p);
  if (e != cudaSuccess) {
    set_error("cache acceptance launch failed: %s", cudaGetErrorString(e));
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // namespace fa
