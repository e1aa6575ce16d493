// fa_cache_attn.cu -- attention over the 8-bit cache (include/fa_cache.h).
//
// The simplest form: one thread block per query row and head, one warp per
// key, an online softmax (running maximum, sum and output, base 2) per warp,
// and the warps joined at the end.  The accumulated weights take a second
// kernel, which computes each score again, one thread per key.
#include "fa.h"
#include "fa_cache.h"
#include "fa_cache_ops.cuh"
#include "fa_device.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

constexpr int kWarps = 4;
constexpr float kLn2f = 0.6931471805599453f;

template <bool kF16>
__device__ __forceinline__ float q_at(const CacheAttnParams& p, int b, int h, int i, int d) {
  const uint16_t u = static_cast<const uint16_t*>(p.q)[b * p.qs[0] + h * p.qs[1] + i * p.qs[2] + d];
  return half_bits_to_f32<kF16>(u);
}

__device__ __forceinline__ float cap_score(const CacheAttnParams& p, float s) {
  return p.cap_out > 0.0f ? p.cap_out * tanhf(s * p.cap_in) : s * p.scale_log2;
}

template <int kKind>
__device__ __forceinline__ float stored(const uint8_t* x) {
  float f[4];
  load8x4<kKind>(*x, f);
  return f[0];
}

template <int kKind, bool kF16>
__global__ void cache_attn_rows_kernel(const CacheAttnParams p) {
  const CacheView& c = p.c;
  const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int kvh = h / p.group, D = c.D;
  const int len = checked_len(c, p.lens[b]);
  const int nq = p.n_q ? min(max(p.n_q[b], 0), p.n) : p.n;
  const int pos = len - nq + i;
  const int hi = i >= nq ? 0 : (p.causal ? min(len, pos + 1) : len);
  const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  float m = -INFINITY, l = 0.0f, o[8] = {};
  for (int j = lo + warp; j < hi; j += kWarps) {
    const int blk = checked_block(c, c.table, c.table_stride, b, j >> c.page_log2);
    if (blk < 0) continue;
    const int slot = j & (c.page - 1);
    const uint8_t* k = c.k + blk * c.ks[0] + kvh * c.ks[1] + slot * c.ks[2];
    const uint8_t* v = c.v + blk * c.vs[0] + kvh * c.vs[1] + slot * c.vs[2];
    float s = 0.0f;
    for (int d = lane; d < D; d += 32) s += q_at<kF16>(p, b, h, i, d) * stored<kKind>(k + d);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, x);
    s = cap_score(p, s * c.k_scale[(long long)blk * c.H + kvh]);
    const float m2 = fmaxf(m, s), f = exp2f(m - m2), w = exp2f(s - m2), vs = c.v_scale[(long long)blk * c.H + kvh];
    m = m2;
    l = l * f + w;
    for (int e = 0; e < D / 32; ++e) o[e] = o[e] * f + w * vs * stored<kKind>(v + lane + 32 * e);
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][256];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  for (int e = 0; e < D / 32; ++e) so[warp][lane + 32 * e] = o[e];
  __syncthreads();
  float mx = -INFINITY, sum = 0.0f;
  for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm[w]);
  for (int w = 0; w < kWarps; ++w) sum += mx == -INFINITY ? 0.0f : sl[w] * exp2f(sm[w] - mx);
  for (int d = threadIdx.x; d < D; d += blockDim.x) {
    float x = 0.0f;
    for (int w = 0; w < kWarps; ++w) x += mx == -INFINITY ? 0.0f : so[w][d] * exp2f(sm[w] - mx);
    x = sum > 0.0f ? x / sum : 0.0f;
    const long long at = b * p.os[0] + h * p.os[1] + i * p.os[2] + d;
    if (kF16)
      static_cast<__half*>(p.o)[at] = __float2half_rn(x);
    else
      static_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(x);
  }
  if (threadIdx.x == 0)
    p.lse[((long long)b * p.Hq + h) * p.n + i] = sum > 0.0f ? (mx + log2f(sum)) * kLn2f : -INFINITY;
}

template <int kKind, bool kF16>
__global__ void cache_attn_weights_kernel(const CacheAttnParams p) {
  const CacheView& c = p.c;
  const int kvh = blockIdx.y, b = blockIdx.z, j = blockIdx.x * blockDim.x + threadIdx.x;
  const int len = checked_len(c, p.lens[b]);
  const int nq = p.n_q ? min(max(p.n_q[b], 0), p.n) : p.n;
  if (j >= len) return;
  if (j >= p.W) return flag_bad_index(c);
  const int blk = checked_block(c, c.table, c.table_stride, b, j >> c.page_log2);
  if (blk < 0) return;
  const uint8_t* k = c.k + blk * c.ks[0] + kvh * c.ks[1] + (j & (c.page - 1)) * c.ks[2];
  const float ks = c.k_scale[(long long)blk * c.H + kvh];
  float sum = 0.0f;
  for (int i = 0; i < nq; ++i) {
    const int pos = len - nq + i;
    if ((p.causal && j > pos) || (p.window > 0 && j <= pos - p.window)) continue;
    for (int g = 0; g < p.group; ++g) {
      const int h = kvh * p.group + g;
      float s = 0.0f;
      for (int d = 0; d < c.D; ++d) s += q_at<kF16>(p, b, h, i, d) * stored<kKind>(k + d);
      sum += exp2f(cap_score(p, s * ks) - p.lse[((long long)b * p.Hq + h) * p.n + i] * 1.4426950408889634f);
    }
  }
  p.weights[((long long)b * c.H + kvh) * p.W + j] += sum;
}

template <int kKind, bool kF16>
int launch(const CacheAttnParams& p, const LaunchCtx& ctx) {
  cache_attn_rows_kernel<kKind, kF16><<<dim3(p.n, p.Hq, p.B), 32 * kWarps, 0, ctx.stream>>>(p);
  if (p.weights)
    cache_attn_weights_kernel<kKind, kF16>
        <<<dim3((unsigned)(((long long)p.c.M * p.c.page + 127) / 128), p.c.H, p.B), 128, 0, ctx.stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("cache attention launch failed: %s", cudaGetErrorString(e));
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // namespace

int launch_cache_attn(const CacheAttnParams& p, int kind, int dtype, const LaunchCtx& ctx) {
  const bool f16 = dtype == FA_DTYPE_F16;
  if (kind == FA_CACHE_E4M3) return f16 ? launch<kKindE4m3, true>(p, ctx) : launch<kKindE4m3, false>(p, ctx);
  return f16 ? launch<kKindInt8, true>(p, ctx) : launch<kKindInt8, false>(p, ctx);
}

long long cache_attn_workspace(const CacheAttnParams&, int) { return 0; }

}  // namespace fa
