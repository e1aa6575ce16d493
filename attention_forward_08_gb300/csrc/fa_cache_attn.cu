// fa_cache_attn.cu -- attention over the 8-bit cache (include/fa_cache.h).
//
// Few rows and many rows alike run cache_decode_kernel (fa_cache_decode.cuh).
// The accumulated weights take a second kernel, which computes each score
// again, one thread per key.
#include "fa.h"
#include "fa_cache.h"
#include "fa_cache_ops.cuh"
#include "fa_cache_decode_launch.cuh"
#include "fa_device.h"
#include "fa_ptx.cuh"

namespace fa {
namespace {

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
  const int rc = p.c.D == 64    ? launch_decode_d64(p, kKind, kF16, ctx)
                 : p.c.D == 128 ? launch_decode_d128(p, kKind, kF16, ctx)
                                : launch_decode_d256(p, kKind, kF16, ctx);
  if (rc != FA_OK) return rc;
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

long long cache_attn_workspace(const CacheAttnParams& p, int num_sms) {
  return p.c.D == 64    ? decode_workspace_d<64>(p, num_sms)
         : p.c.D == 128 ? decode_workspace_d<128>(p, num_sms)
                        : decode_workspace_d<256>(p, num_sms);
}

}  // namespace fa
