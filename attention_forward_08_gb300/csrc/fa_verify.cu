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
// terms and sums are pairs of floats (48 bits; error-free sums and products):
// doubles for every term would take the few FP64 units ten times the memory's
// time, and doubles for the walk and the sums of segments alone took half of a
// single sequence's (12.4 us).  All orders are fixed.
//
// Work.  A cluster of 2 to 8 blocks a sequence, as many as run at once (64
// sequences: 18.0 us with 4, 24 with 8, which take two turns).  Tests need two
// numbers a node, which every block gathers for itself and walks over alike, so that
// decisions are not sent around; a pass over a row is shared out by contiguous
// segments, one a warp, whose sums go to all blocks (distributed shared memory).
// These tell the segment in which the cumulative sum passes u Z; its block alone
// reads that again, a run of entries a thread.
//
// Bound: latency (three dependent loads and two cluster barriers: one sequence of 5
// nodes, 32000 entries, 9.2 us); then the sums' instructions, some 30 an entry of p
// and q (32 sequences of 16 nodes, 128001 bf16 entries, up to three passes one after
// the other, 29 us; of 17 nodes other draws, 27 us in bf16, 30 in fp16 and in fp32;
// 64 of 100000 bf16 entries without q, 18 us, 0.7 TB/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa.h"
#include "fa_cache_params.h"
#include "fa_device.h"

namespace fa {
namespace {

constexpr int kVerThreads = 512, kVerWarps = kVerThreads / 32, kVerMostBlocks = 8;
constexpr size_t kVerSmem = 45 * 1024;  // dynamic shared memory that needs no opting in

__device__ __forceinline__ float ver_load(const float* p) { return __ldg(p); }
__device__ __forceinline__ float ver_load(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
}
__device__ __forceinline__ float ver_load(const __half* p) { return __half2float(__ldg(p)); }
// (A probability that is none counts as 0.)
__device__ __forceinline__ float ver_prob(float x) { return __float_as_uint(x) < 0x7F800000u ? x : 0.0f; }

__device__ __forceinline__ uint32_t ver_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void ver_cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A number of 48 bits: hi + lo.
struct Pair {
  float hi, lo;
};
// Writes x where `p` lies in block `rank` of the cluster.
__device__ __forceinline__ void ver_send(Pair* p, uint32_t rank, Pair x) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;\n\tst.shared::cluster.f32 [%0 + 4], %2;" ::"r"(at), "f"(x.hi), "f"(x.lo)
               : "memory");
}

// (intrinsics: nothing here may be contracted or reordered)
__device__ __forceinline__ void pair_add(Pair& a, float hi, float lo) {
  const float s = __fadd_rn(a.hi, hi), b = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, b)), __fsub_rn(hi, b));
  a.hi = s;
  a.lo = __fadd_rn(a.lo, __fadd_rn(e, lo));
}
__device__ __forceinline__ Pair pair_sum(Pair a, Pair b) {  // normalised
  pair_add(a, b.hi, b.lo);
  const float s = __fadd_rn(a.hi, a.lo);
  return {s, __fsub_rn(a.lo, __fsub_rn(s, a.hi))};
}
__device__ __forceinline__ Pair pair_normal(Pair a) { return pair_sum(a, {0.0f, 0.0f}); }
__device__ __forceinline__ Pair pair_minus(Pair a, Pair b) { return pair_sum(a, {-b.hi, -b.lo}); }
__device__ __forceinline__ Pair pair_times(Pair a, float b) {
  const float h = __fmul_rn(a.hi, b);
  return pair_sum({h, 0.0f}, {__fmaf_rn(a.lo, b, __fmaf_rn(a.hi, b, -h)), 0.0f});
}
__device__ __forceinline__ bool pair_above(Pair a, Pair b) { return pair_minus(a, b).hi > 0.0f; }
// max(p - c q, 0).  (Not normalised: where p is within a step or two of c q, lo
// may be the larger part, and the sign is that of both.)
__device__ __forceinline__ Pair ver_less(float p, float q, Pair c) {
  const float h = __fmul_rn(c.hi, q);
  const float e = __fmaf_rn(c.lo, q, __fmaf_rn(c.hi, q, -h));
  const float s = __fsub_rn(p, h);
  const float f = __fsub_rn(__fsub_rn(p, s), h);  // (what s lost, where p > h; nothing where p is near h)
  const float lo = __fsub_rn(f, e);
  const bool some = __fadd_rn(s, lo) > 0.0f;
  return {some ? s : 0.0f, some ? lo : 0.0f};
}

__device__ __forceinline__ Pair ver_warp_sum(Pair x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(0xFFFFFFFFu, x.hi, o), lo = __shfl_xor_sync(0xFFFFFFFFu, x.lo, o);
    pair_add(x, hi, lo);
  }
  return x;
}
__device__ __forceinline__ Pair ver_lane(Pair x, int lane) {
  return {__shfl_sync(0xFFFFFFFFu, x.hi, lane), __shfl_sync(0xFFFFFFFFu, x.lo, lane)};
}
__device__ __forceinline__ Pair ver_upto(Pair x, int lane) {  // inclusive sum over the lanes
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const Pair y = {__shfl_up_sync(0xFFFFFFFFu, x.hi, o), __shfl_up_sync(0xFFFFFFFFu, x.lo, o)};
    if (lane >= o) x = pair_sum(x, y);
  }
  return x;
}

// Of values x in order, a lane each, `upto` their inclusive sums: the first whose
// sum passes `rest` (the last that is not 0 where none does: u of 1, a rounding;
// -1: all are 0).  What is left of `rest` before it.
__device__ __forceinline__ int ver_find(Pair x, Pair upto, Pair& rest) {
  const bool is = x.hi > 0.0f;
  const uint32_t some = __ballot_sync(0xFFFFFFFFu, is), hit = __ballot_sync(0xFFFFFFFFu, is && pair_above(upto, rest));
  if (!some) return -1;
  const int l = hit ? __ffs(hit) - 1 : 31 - __clz(some);
  const Pair before = ver_lane(upto, max(l - 1, 0));
  if (l > 0) rest = pair_minus(rest, before);
  return l;
}

struct VerShared {
  Pair sum[2][kVerWarps * kVerMostBlocks];  // of the segments, by pass & 1
  Pair part[kVerWarps];                     // of the chosen segment's pieces
  // What comes next: a pass over r = max(p[cur] - c q[cur], 0), without the
  // candidates below cur where `gone`; or the path's length, the segment that
  // holds the token, and what is left of the sum sought there.
  int ends, cur, gone, count, seg;
  Pair c, rest;
};

static_assert(kVerSmem + sizeof(VerShared) <= 48 * 1024, "shared memory");

// What is left of a row.
template <class T>
struct VerRow {
  const T *p, *q;        // q: NULL where nothing is taken off
  Pair c;
  const uint32_t* gone;  // bit by entry - first: rejected candidates; or NULL
  int first;
  __device__ __forceinline__ float left(int e, float x) const {
    return (gone[(e - first) >> 5] >> ((e - first) & 31)) & 1u ? 0.0f : x;
  }
  __device__ __forceinline__ Pair entry(int e) const {
    const float x = ver_prob(ver_load(p + e));
    if (q) return pair_normal(ver_less(x, ver_prob(ver_load(q + e)), c));
    return {gone ? left(e, x) : x, 0.0f};
  }
  // This lane's sum over entries e0 + lane, e0 + lane + 32, .. < e1.  (All are
  // asked for at once, into L2.)
  __device__ __forceinline__ Pair sum(int e0, int e1) const {
    const int lane = threadIdx.x & 31;
    constexpr int kLine = 128 / sizeof(T);
#pragma unroll 1
    for (int e = e0 + lane * kLine; e < e1; e += 32 * kLine) {
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p + e));
      if (q) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + e));
    }
    Pair s = {0.0f, 0.0f};
    if (q) {
      constexpr int kAtOnce = 8;
#pragma unroll 1
      for (int e = e0 + lane; e < e1; e += 32 * kAtOnce) {
        float x[kAtOnce], y[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) x[u] = e + 32 * u < e1 ? ver_load(p + e + 32 * u) : 0.0f;
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) y[u] = e + 32 * u < e1 ? ver_load(q + e + 32 * u) : 0.0f;
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
          const Pair r = ver_less(ver_prob(x[u]), ver_prob(y[u]), c);
          pair_add(s, r.hi, r.lo);
        }
      }
    } else {
      constexpr int kAtOnce = 16;
#pragma unroll 1
      for (int e = e0 + lane; e < e1; e += 32 * kAtOnce) {
        float x[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) x[u] = e + 32 * u < e1 ? ver_load(p + e + 32 * u) : 0.0f;
        if (gone) {
#pragma unroll
          for (int u = 0; u < kAtOnce; ++u) x[u] = left(min(e + 32 * u, e1 - 1), x[u]);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) pair_add(s, ver_prob(x[u]), 0.0f);
      }
    }
    return s;
  }
};

template <class T>
__global__ void __launch_bounds__(kVerThreads, 2) verify_kernel(const VerifyParams p) {
  extern __shared__ int s_nodes[];
  __shared__ VerShared s;
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // (met by the wait before the first pass)
  const int blocks = p.blocks, rank = (int)ver_rank(), b = blockIdx.x / blocks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = p.n;
  int* s_tree = s_nodes;
  int* s_token = s_nodes + n;
  float* s_u = reinterpret_cast<float*>(s_nodes + 2 * n);
  float* s_p = reinterpret_cast<float*>(s_nodes + 3 * n);
  float* s_q = reinterpret_cast<float*>(s_nodes + 4 * n);
  uint32_t* s_gone = reinterpret_cast<uint32_t*>(s_nodes + 5 * n);  // a bit for each of this block's entries
  const int first = rank * kVerWarps * p.seg;                       // the first of them
  const T* const probs = static_cast<const T*>(p.p) + b * p.ps[0];
  const T* const drafts = p.q ? static_cast<const T*>(p.q) + b * p.qs[0] : nullptr;

  // The nodes, and the two numbers of each that its test needs.
  const int told = p.n_q ? p.n_q[b] : n, nodes = min(max(told, 0), n);
  const float u_next = p.u_next[b];
  bool bad = nodes != told;
  for (int i = tid; i < n; i += kVerThreads) {
    int up = p.tree[b * p.tree_stride + i], t = p.tokens[b * p.tokens_stride + i];
    s_u[i] = p.u[b * p.u_stride + i];
    if (i < nodes && (up >= i || up < -1 || (i > 0 && (t < 0 || t >= p.V)))) bad = true;
    if (up >= i || up < 0) up = -1;
    const bool there = i < nodes && up >= 0 && t >= 0 && t < p.V;
    s_tree[i] = up;
    s_token[i] = there ? t : -1;
    s_p[i] = there ? ver_prob(ver_load(probs + up * p.ps[1] + t)) : 0.0f;
    s_q[i] = there && drafts ? ver_prob(ver_load(drafts + up * p.qs[1] + t)) : 0.0f;
  }
  if (bad && rank == 0) atomicOr(p.status, kStatusBadIndex);
  int* const path = p.path + (long long)b * n;
  if (rank == 0)
    for (int i = tid; i < n; i += kVerThreads) path[i] = i == 0 && nodes > 0 ? 0 : -1;
  __syncthreads();
  if (!drafts) {  // a candidate that a sibling before it has been: nothing is left of it
    const int each = max(kVerThreads / max(nodes, 1), 1), at = tid % each;  // threads a node
    for (int i = tid / each; i < nodes; i += kVerThreads / each) {
      if (s_token[i] < 0) continue;
      bool again = false;
#pragma unroll 1
      for (int j = s_tree[i] + 1 + at; j < i; j += each) again = again || (s_tree[j] == s_tree[i] && s_token[j] == s_token[i]);
      if (again) s_p[i] = 0.0f;
    }
    __syncthreads();
  }
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (nodes == 0) {
    if (rank == 0 && tid == 0) p.count[b] = 0, p.token[b] = -1;
    return;
  }

  VerRow<T> row;
  row.first = first;
  // Where the walk stands (warp 0): the path's last node, the node to look at
  // next, nodes of the path; c, and the sum of what is left; whether the path
  // has ended, the last pass's sums are those of what is left, and they are p's.
  int cur = 0, next = 1, count = 1;
  Pair c = {0.0f, 0.0f}, z = {1.0f, 0.0f};
  bool over = false, summed = false, bare = false;
  bool taken = false;  // the last pass was without rejected candidates
  const int per = (kVerWarps * blocks + 31) / 32;  // segments a lane
  Pair mine, upto;                                 // of its segments, and with the lanes before
#pragma unroll 1
  for (int passes = 0;; ++passes) {
    const Pair* const sums = s.sum[(passes - 1) & 1];  // (the last pass's)
    if (warp == 0) {
      if (passes > 0) {
        mine = {0.0f, 0.0f};
        for (int i = lane * per; i < min((lane + 1) * per, kVerWarps * blocks); ++i) mine = pair_sum(mine, sums[i]);
        upto = ver_upto(mine, lane);
        z = ver_lane(upto, 31);
      }
      // the walk, up to the path's end or to a sum that it needs
      bool gone = false, ends = false;
#pragma unroll 1
      while (!over) {
        int i = -1;
#pragma unroll 1
        for (int base = next & ~31; base < nodes; base += 32) {
          const int j = base + lane;
          const uint32_t hit = __ballot_sync(0xFFFFFFFFu, j >= next && j < nodes && s_tree[j] == cur);
          if (hit) {
            i = base + __ffs(hit) - 1;
            break;
          }
        }
        over = i < 0;
        if (over) break;
        next = i + 1;
        const float pi = s_p[i];
        Pair r = {pi, 0.0f}, least = pair_times(z, s_u[i]);
        if (drafts) {
          const Pair d = pair_sum(r, pair_times(c, -s_q[i]));
          r = d.hi > 0.0f ? d : Pair{0.0f, 0.0f};
          least = pair_times(least, s_q[i]);
        }
        if (pair_above(r, least)) {
          if (rank == 0 && lane == 0) path[count] = i;
          ++count;
          cur = i;
          c = {0.0f, 0.0f};
          z = {1.0f, 0.0f};
          summed = false;
        } else if (drafts) {
          c = pair_sum(c, z);
          summed = true;
          break;
        } else {
          z = pair_minus(z, r);
        }
      }
      if (over) {
        if (!summed) {  // (the path ended with an accepted node, or there is no q)
          gone = !drafts;
          summed = true;
        } else if (z.hi == 0.0f && !bare) {  // nothing is left: of p itself
          c = {0.0f, 0.0f};
          bare = true;
        } else {  // the segment that holds the token
          ends = true;
          Pair rest = pair_times(z, u_next > 0.0f ? fminf(u_next, 1.0f) : 0.0f);
          int seg = ver_find(mine, upto, rest);
          if (seg >= 0) {
            const int i = seg * per + lane;
            const Pair x = lane < per && i < kVerWarps * blocks ? sums[i] : Pair{0.0f, 0.0f};
            seg = seg * per + max(ver_find(x, ver_upto(x, lane), rest), 0);
          }
          if (lane == 0) s.seg = seg, s.rest = rest;
        }
      }
      if (lane == 0) s.ends = ends, s.cur = cur, s.gone = gone, s.count = count, s.c = c;
    }
    __syncthreads();
    if (s.ends) break;
    // The sums of all segments; by the whole cluster.
    const int e0 = first + warp * p.seg, e1 = min(e0 + p.seg, p.V);
    row.c = s.c;
    row.p = probs + s.cur * p.ps[1];
    row.q = drafts && row.c.hi > 0.0f ? drafts + s.cur * p.qs[1] : nullptr;
    row.gone = nullptr;
    taken = s.gone;
    if (taken) {  // (a warp's own bits)
      for (int w = lane; w < p.seg / 32; w += 32) s_gone[warp * (p.seg / 32) + w] = 0u;
      __syncwarp();
      bool some = false;
      for (int j = s.cur + 1 + lane; j < nodes; j += 32) {
        const int e = s_token[j];
        if (s_tree[j] != s.cur || e < e0 || e >= e1) continue;
        atomicOr(s_gone + ((e - first) >> 5), 1u << ((e - first) & 31));
        some = true;
      }
      __syncwarp();
      if (__any_sync(0xFFFFFFFFu, some)) row.gone = s_gone;
    }
    const Pair x = pair_normal(ver_warp_sum(row.sum(e0, e1)));
    if (lane < blocks) ver_send(&s.sum[passes & 1][rank * kVerWarps + warp], (uint32_t)lane, x);
    __syncwarp();  // (the barrier takes whole warps)
    ver_cluster_sync();
  }

  // The token: the chosen segment's block sums that again, a run of entries a
  // thread; the warp and then the lane in whose run the sum passes go over it.
  const int seg = s.seg;
  if (rank == 0 && tid == 0) {
    p.count[b] = s.count;
    if (seg < 0) p.token[b] = 0;  // a row without any probability
  }
  if (seg < 0 || seg / kVerWarps != rank) return;
  const int run = p.seg / kVerThreads + (p.seg % kVerThreads != 0), s1 = min((seg + 1) * p.seg, p.V);
  const int r0 = min(seg * p.seg + tid * run, s1), r1 = min(r0 + run, s1);
  row.gone = taken ? s_gone : nullptr;
  Pair x = {0.0f, 0.0f};
#pragma unroll 4
  for (int e = r0; e < r1; ++e) x = pair_sum(x, row.entry(e));
  const Pair upto_lane = ver_upto(x, lane);
  if (lane == 31) s.part[warp] = upto_lane;
  __syncthreads();
  Pair rest = s.rest;
  const Pair part = lane < kVerWarps ? s.part[lane] : Pair{0.0f, 0.0f};
  if (max(ver_find(part, ver_upto(part, lane), rest), 0) != warp) return;
  if (max(ver_find(x, upto_lane, rest), 0) != lane) return;
  int token = r0;
#pragma unroll 1
  for (int e = r0; e < r1; ++e) {
    const Pair r = row.entry(e);
    if (r.hi > 0.0f) {
      token = e;
      if (pair_above(r, rest)) break;
      rest = pair_minus(rest, r);
    }
  }
  p.token[b] = token;
}

template <class T>
cudaError_t launch(const VerifyParams& p, size_t smem, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * p.blocks));
  cfg.blockDim = dim3(kVerThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)p.blocks;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, p);
}

}  // namespace

int launch_verify(VerifyParams p, int dtype, const LaunchCtx& ctx) {
  const auto share = [&](int blocks) {
    const int segs = kVerWarps * blocks;
    p.blocks = blocks;
    p.seg = (p.V + segs * 32 - 1) / (segs * 32) * 32;
    return (size_t)p.n * 20 + (p.q ? 0 : (size_t)kVerWarps * p.seg / 8);
  };
  // Blocks a sequence: as many as run at once (two an SM), 2 to 8.
  int blocks = kVerMostBlocks;
  while (blocks > 2 && p.B * blocks > 2 * ctx.num_sms && share(blocks / 2) <= kVerSmem) blocks /= 2;
  const size_t smem = share(blocks);
  const cudaError_t e = dtype == FA_DTYPE_F32    ? launch<float>(p, smem, ctx.stream)
                        : dtype == FA_DTYPE_BF16 ? launch<__nv_bfloat16>(p, smem, ctx.stream)
                                                 : launch<__half>(p, smem, ctx.stream);
  if (e != cudaSuccess) {
    set_error("verification launch failed: %s", cudaGetErrorString(e));
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // namespace fa
