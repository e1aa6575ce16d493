// fa_verify.cu -- which drafted tokens stay, and the token behind them
// (include/fa_cache.h, fa_verify_drafts).
//
// Mathematics.  At a node the children are tested in turn.  What the target's
// probabilities p leave after k rejected children, each drawn from q, is
//
//   r_0 = p,  r_k+1 = max(r_k - Z_k q, 0),  Z_0 = 1,  Z_k = sum r_k
//
// and since a value that reached 0 stays there, r_k = max(p - C_k q, 0) with
// C_k = Z_0 + .. + Z_k-1: a rejection costs one sum over the vocabulary and
// keeps no row.  Children of distinct candidates (no q) cost no sum at all:
// Z_k is 1 less what was rejected.
//
// A token is the least t whose cumulative sum passes u Z.  With a vocabulary of
// 10^5 two sums in 32 bits would disagree about t once in a hundred calls, so
// terms and partial sums are pairs of floats (48 bits; error-free sums and
// products), and 64 bits from a warp on: doubles for every term would take the
// few FP64 units ten times the memory's time.  All orders are fixed.
//
// Work.  A cluster of 8 blocks a sequence.  Tests need two numbers a node, which
// every block gathers for itself and walks over alike, so that decisions are
// not sent around; a pass over a row is shared out by contiguous segments, one
// a warp, whose sums go to all blocks (distributed shared memory).  The warp
// sums tell the segment in which the cumulative sum passes u Z; its block alone
// reads that again.
//
// Bound: latency (three dependent loads and two cluster barriers); then one row
// of p and q a sequence, and one more for each rejected draft that has a sibling.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa.h"
#include "fa_cache_params.h"
#include "fa_device.h"

namespace fa {
namespace {

constexpr int kVerThreads = 512, kVerWarps = kVerThreads / 32, kVerBlocks = 8, kVerSegs = kVerWarps * kVerBlocks;

__device__ __forceinline__ float ver_load(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ver_load(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
}
__device__ __forceinline__ float ver_load(const __half* p) { return __half2float(__ldg(p)); }
// (A probability that is none counts as 0.)
__device__ __forceinline__ float ver_prob(float x) { return x > 0.0f && x <= 3.402823466e38f ? x : 0.0f; }

__device__ __forceinline__ uint32_t ver_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void ver_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Writes x where `p` lies in block `rank` of the cluster.
__device__ __forceinline__ void ver_send(double* p, uint32_t rank, double x) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(at), "d"(x) : "memory");
}

// A sum of 48 bits: hi + lo.
struct Pair {
  float hi, lo;
};
// (intrinsics: nothing here may be contracted or reordered)
__device__ __forceinline__ void pair_add(Pair& a, float hi, float lo) {
  const float s = __fadd_rn(a.hi, hi), b = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, b)), __fsub_rn(hi, b));
  a.hi = s;
  a.lo = __fadd_rn(a.lo, __fadd_rn(e, lo));
}
// max(p - c q, 0).
__device__ __forceinline__ Pair ver_less(float p, float q, Pair c) {
  const float h = __fmul_rn(c.hi, q);
  const float e = __fmaf_rn(c.lo, q, __fmaf_rn(c.hi, q, -h));
  const float s = __fsub_rn(p, h), b = __fsub_rn(s, p);
  const float f = __fsub_rn(__fadd_rn(p, -__fsub_rn(s, b)), __fadd_rn(h, b));
  Pair r = {s, __fsub_rn(f, e)};
  if (!(__fadd_rn(r.hi, r.lo) > 0.0f)) r.hi = r.lo = 0.0f;
  return r;
}

__device__ __forceinline__ Pair ver_warp_sum(Pair x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(0xFFFFFFFFu, x.hi, o), lo = __shfl_xor_sync(0xFFFFFFFFu, x.lo, o);
    pair_add(x, hi, lo);
  }
  return x;
}
__device__ __forceinline__ double ver_upto(double x, int lane) {  // inclusive sum over the lanes
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Of values in order, a lane each: the first whose inclusive sum passes `rest`
// (the last that is not 0 where none does: u of 1, a rounding; -1: all are 0).
// What is left of `rest` before it.
__device__ __forceinline__ int ver_find(double x, int lane, double& rest) {
  const double upto = ver_upto(x, lane);
  const uint32_t some = __ballot_sync(0xFFFFFFFFu, x > 0.0), hit = __ballot_sync(0xFFFFFFFFu, x > 0.0 && upto > rest);
  if (!some) return -1;
  const int l = hit ? __ffs(hit) - 1 : 31 - __clz(some);
  rest = __shfl_sync(0xFFFFFFFFu, rest - (upto - x), l);
  return l;
}

struct VerShared {
  double sum[2][kVerSegs];  // of the segments, by pass & 1
  double part[kVerWarps];   // of a segment's pieces
  // Where the walk stands.
  int cur, next, count;     // the path's last node, the node to look at next, nodes of the path
  double c, z;              // r = max(p[cur] - c q[cur], 0), and its sum
  int ends, summed;         // no child is left; the last pass's sums are r's
  double total;
  // The segment that holds the token, and what is left of the sum sought there.
  int seg;
  double rest;
};

// What is left of a row.
template <class T>
struct VerRow {
  const T *p, *q;        // q: NULL where nothing is taken off
  Pair c;
  const uint32_t* gone;  // bit by entry - first: rejected candidates; or NULL
  int first;
  __device__ __forceinline__ Pair less(int e, float x, float y) const {
    x = ver_prob(x);
    if (q) return ver_less(x, ver_prob(y), c);
    if (gone && ((gone[(e - first) >> 5] >> ((e - first) & 31)) & 1u)) x = 0.0f;
    return {x, 0.0f};
  }
  // This lane's sum over entries e0 + lane, e0 + lane + 32, .. < e1.
  __device__ __forceinline__ Pair sum(int e0, int e1) const {
    Pair s = {0.0f, 0.0f};
#pragma unroll 1
    for (int e = e0 + (threadIdx.x & 31); e < e1; e += 32 * kAtOnce) {
      float x[kAtOnce], y[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) x[u] = e + 32 * u < e1 ? ver_load(p + e + 32 * u) : 0.0f;
      if (q) {
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) y[u] = e + 32 * u < e1 ? ver_load(q + e + 32 * u) : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const Pair r = less(min(e + 32 * u, e1 - 1), x[u], y[u]);
        pair_add(s, r.hi, r.lo);
      }
    }
    return s;
  }
  static constexpr int kAtOnce = 8;
};

template <class T>
__global__ void __launch_bounds__(kVerThreads) verify_kernel(const VerifyParams p) {
  extern __shared__ int s_nodes[];
  __shared__ VerShared s;
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // (met by the wait before the first pass)
  const int b = blockIdx.x / kVerBlocks, rank = (int)ver_rank(), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = p.n;
  int* s_tree = s_nodes;
  int* s_token = s_nodes + n;
  float* s_u = reinterpret_cast<float*>(s_nodes + 2 * n);
  float* s_p = reinterpret_cast<float*>(s_nodes + 3 * n);
  float* s_q = reinterpret_cast<float*>(s_nodes + 4 * n);
  uint32_t* s_gone = reinterpret_cast<uint32_t*>(s_nodes + 5 * n);  // a bit for each of this block's entries
  const int mine = kVerWarps * p.seg, first = rank * mine;          // entries of a block, and this one's first
  const T* const probs = static_cast<const T*>(p.p) + b * p.ps[0];
  const T* const drafts = p.q ? static_cast<const T*>(p.q) + b * p.qs[0] : nullptr;

  // The nodes, and the two numbers of each that its test needs.
  const int nodes = p.n_q ? min(max(p.n_q[b], 0), n) : n;
  bool bad = p.n_q && nodes != p.n_q[b];
  for (int i = tid; i < nodes; i += kVerThreads) {
    int up = p.tree[b * p.tree_stride + i], t = p.tokens[b * p.tokens_stride + i];
    if (up >= i || up < -1 || (i > 0 && (t < 0 || t >= p.V))) bad = true;
    if (up >= i || up < 0) up = -1;
    const bool there = up >= 0 && t >= 0 && t < p.V;
    s_tree[i] = up;
    s_token[i] = there ? t : -1;
    s_u[i] = p.u[b * p.u_stride + i];
    s_p[i] = there ? ver_prob(ver_load(probs + up * p.ps[1] + t)) : 0.0f;
    s_q[i] = there && drafts ? ver_prob(ver_load(drafts + up * p.qs[1] + t)) : 0.0f;
  }
  if (bad && rank == 0) atomicOr(p.status, kStatusBadIndex);
  if (!drafts)
    for (int w = tid; w < mine / 32; w += kVerThreads) s_gone[w] = 0u;
  int* const path = p.path + (long long)b * n;
  if (rank == 0)
    for (int i = tid; i < n; i += kVerThreads) path[i] = i == 0 && nodes > 0 ? 0 : -1;
  if (tid == 0) {
    s.cur = 0;
    s.next = s.count = 1;
    s.c = 0.0;
    s.z = 1.0;
    s.summed = 0;
  }
  __syncthreads();
  if (!drafts) {  // a candidate that a sibling before it has been: nothing is left of it
    for (int i = tid; i < nodes; i += kVerThreads) {
      bool again = false;
      for (int j = s_tree[i] + 1; j < i && s_tree[i] >= 0; ++j) again = again || (s_tree[j] == s_tree[i] && s_token[j] == s_token[i]);
      if (again) s_p[i] = 0.0f;
    }
    __syncthreads();
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (nodes == 0) {
    if (rank == 0 && tid == 0) p.count[b] = 0, p.token[b] = -1;
    return;
  }

  int passes = 0;
  VerRow<T> row;
  row.first = first;
  // The sums of all segments, and of the row; by the whole cluster.
  auto pass = [&](double c, const uint32_t* gone) {
    row.p = probs + s.cur * p.ps[1];
    row.q = drafts && c > 0.0 ? drafts + s.cur * p.qs[1] : nullptr;
    row.c.hi = (float)c;
    row.c.lo = (float)(c - (double)row.c.hi);
    row.gone = gone;
    double* const sums = s.sum[passes & 1];
    const int e0 = first + warp * p.seg;
    const Pair x = ver_warp_sum(row.sum(e0, min(e0 + p.seg, p.V)));
    if (lane < kVerBlocks) ver_send(sums + rank * kVerWarps + warp, (uint32_t)lane, (double)x.hi + (double)x.lo);
    ver_cluster_sync();
    ++passes;
    if (warp == 0) {
      double all = 0.0;
#pragma unroll
      for (int i = 0; i < kVerSegs / 32; ++i) all += sums[lane * (kVerSegs / 32) + i];
      all = __shfl_sync(0xFFFFFFFFu, ver_upto(all, lane), 31);
      if (lane == 0) s.total = all;
    }
    __syncthreads();
  };

  while (true) {
    if (warp == 0) {  // the walk, up to the path's end or to a sum that it needs
      int cur = s.cur, next = s.next, count = s.count, summed = s.summed;
      double c = s.c, z = summed ? s.total : s.z;
      bool ends = false;
      while (true) {
        int i = -1;
        for (int base = next & ~31; base < nodes; base += 32) {
          const int j = base + lane;
          const uint32_t hit = __ballot_sync(0xFFFFFFFFu, j >= next && j < nodes && s_tree[j] == cur);
          if (hit) {
            i = base + __ffs(hit) - 1;
            break;
          }
        }
        ends = i < 0;
        if (ends) break;
        next = i + 1;
        const double pi = (double)s_p[i], qi = drafts ? (double)s_q[i] : 1.0;
        const double r = drafts ? fmax(pi - c * qi, 0.0) : pi;
        if ((double)s_u[i] * qi * z < r) {
          if (rank == 0 && lane == 0) path[count] = i;
          ++count;
          cur = i;
          c = 0.0;
          z = 1.0;
          summed = 0;
        } else if (drafts) {
          c += z;
          break;
        } else {
          z -= r;
        }
      }
      __syncwarp();
      if (lane == 0) s.cur = cur, s.next = next, s.count = count, s.c = c, s.z = z, s.ends = ends, s.summed = ends ? summed : 1;
    }
    __syncthreads();
    if (s.ends) break;
    pass(s.c, nullptr);
  }
  if (!s.summed) {  // (the path ended with an accepted node, or there is no q)
    if (!drafts) {
      for (int j = s.cur + 1 + tid; j < nodes; j += kVerThreads) {
        const int e = s_token[j] - first;
        if (s_tree[j] == s.cur && s_token[j] >= 0 && e >= 0 && e < mine) atomicOr(s_gone + (e >> 5), 1u << (e & 31));
      }
      __syncthreads();
    }
    pass(s.c, drafts ? nullptr : s_gone);
  }
  if (s.total == 0.0) pass(0.0, nullptr);  // nothing is left: of p itself

  // The token: the segment, by every block; then, by that segment's block, the
  // piece of it and the entry.
  if (warp == 0) {
    const double* const sums = s.sum[(passes - 1) & 1];
    constexpr int kMine = kVerSegs / 32;
    const double u = (double)p.u_next[b];
    double rest = (u > 0.0 ? fmin(u, 1.0) : 0.0) * s.total, x = 0.0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) x += sums[lane * kMine + i];
    int seg = ver_find(x, lane, rest);
    if (seg >= 0) seg = seg * kMine + max(ver_find(lane < kMine ? sums[seg * kMine + lane] : 0.0, lane, rest), 0);
    if (lane == 0) s.seg = seg, s.rest = rest;
  }
  __syncthreads();
  const int seg = s.seg;
  if (rank == 0 && tid == 0) {
    p.count[b] = s.count;
    if (seg < 0) p.token[b] = 0;  // a row without any probability
  }
  if (seg < 0 || seg / kVerWarps != rank) return;
  const int piece = p.seg / kVerWarps, s0 = seg * p.seg, s1 = min(s0 + p.seg, p.V);
  const int p0 = s0 + warp * piece;
  const Pair x = ver_warp_sum(row.sum(p0, min(p0 + piece, s1)));
  if (lane == 0) s.part[warp] = (double)x.hi + (double)x.lo;
  __syncthreads();
  if (warp > 0) return;
  double rest = s.rest;
  const int at = max(ver_find(lane < kVerWarps ? s.part[lane] : 0.0, lane, rest), 0), end = min(s0 + (at + 1) * piece, s1);
  int token = 0;
#pragma unroll 1
  for (int e0 = s0 + at * piece; e0 < end; e0 += 32) {
    const int e = e0 + lane;
    Pair r = {0.0f, 0.0f};
    if (e < end) r = row.less(e, ver_load(row.p + e), row.q ? ver_load(row.q + e) : 0.0f);
    const double x = (double)r.hi + (double)r.lo, upto = ver_upto(x, lane);
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, x > 0.0), hit = __ballot_sync(0xFFFFFFFFu, x > 0.0 && upto > rest);
    if (some) token = e0 + 31 - __clz(some);
    if (hit) {
      token = e0 + __ffs(hit) - 1;
      break;
    }
    rest -= __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  if (lane == 0) p.token[b] = token;
}

template <class T>
cudaError_t launch(const VerifyParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * kVerBlocks));
  cfg.blockDim = dim3(kVerThreads);
  cfg.dynamicSmemBytes = (size_t)p.n * 20 + (p.q ? 0 : (size_t)kVerWarps * p.seg / 8);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = kVerBlocks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, p);
}

}  // namespace

int launch_verify(VerifyParams p, int dtype, const LaunchCtx& ctx) {
  p.seg = (p.V + kVerSegs * 32 - 1) / (kVerSegs * 32) * 32;
  const cudaError_t e = dtype == FA_DTYPE_F32    ? launch<float>(p, ctx.stream)
                        : dtype == FA_DTYPE_BF16 ? launch<__nv_bfloat16>(p, ctx.stream)
                                                 : launch<__half>(p, ctx.stream);
  if (e != cudaSuccess) {
    set_error("verification launch failed: %s", cudaGetErrorString(e));
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // namespace fa
