// fa_cache_decode_launch.cuh -- host side of cache_decode_kernel for one head
// dim: tensor maps, grid, workspace.
#pragma once

#include <atomic>

#include "fa.h"
#include "fa_cache.h"
#include "fa_cache_decode.cuh"
#include "fa_cache_weights.cuh"
#include "fa_cache_maps.h"
#include "fa_device.h"

namespace fa {

template <class C>
long long decode_workspace(int num_sms) {
  const long long slots = 2LL * num_sms * C::kCtas * C::kRows;
  return slots * C::kD * 4 + slots * 8;
}

// Programmatic launch: the blocks come up while the kernel before ends, and
// wait for it (griddepcontrol.wait) before they read what it wrote.
template <class P>
cudaError_t launch_after(void (*kern)(P), dim3 grid, unsigned threads, cudaStream_t stream, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

// The accumulated weights, after the attention; workspace behind `used` bytes.
template <int kD>
long long weights_workspace(const CacheAttnParams& a) {
  const long long groups = (long long)a.B * a.c.H * ((a.n * (long long)a.group + 15) / 16);
  return a.weights ? groups * 16 * (kD * 2 + 8) : 0;
}
template <int kD>
int launch_weights(const CacheAttnParams& a, int kind, bool f16, long long used, const LaunchCtx& ctx) {
  WeightParams p;
  p.a = a;
  p.rows = a.n * a.group;
  p.row_groups = (p.rows + 15) / 16;
  p.q = reinterpret_cast<uint32_t*>(a.ws + used);
  p.row = reinterpret_cast<float2*>(a.ws + used + (long long)a.B * a.c.H * p.row_groups * 16 * kD * 2);
  const dim3 by_row((unsigned)(p.row_groups * 2), (unsigned)a.c.H, (unsigned)a.B);
  cudaError_t e = f16 ? launch_after(cache_rows_kernel<true, kD>, by_row, 256, ctx.stream, p)
                      : launch_after(cache_rows_kernel<false, kD>, by_row, 256, ctx.stream, p);
  if (e == cudaSuccess) {
    const long long tokens = (long long)a.c.M * a.c.page;
    const dim3 by_tile((unsigned)((tokens + 127) / 128), (unsigned)a.c.H, (unsigned)a.B);
    e = kind == FA_CACHE_E4M3 ? launch_after(cache_weights_kernel<kKindE4m3, kD>, by_tile, 128, ctx.stream, p)
                              : launch_after(cache_weights_kernel<kKindInt8, kD>, by_tile, 128, ctx.stream, p);
  }
  if (e != cudaSuccess) {
    set_error("cache weights launch failed: %s", cudaGetErrorString(e));
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

template <class C>
int launch_decode(const CacheAttnParams& a, const LaunchCtx& ctx) {
  CUtensorMap tk, tv;
  const int sub = a.c.page < C::kTile ? a.c.page : C::kTile;
  if (!encode_pool(&tk, a.c, false, sub) || !encode_pool(&tv, a.c, true, sub)) return FA_ERR_CUDA;
  auto kern = cache_decode_kernel<C>;
  static std::atomic<unsigned long long> configured{0};
  if (!((configured.load(std::memory_order_acquire) >> ctx.dev) & 1ull)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) {
      set_error("cudaFuncSetAttribute(max dynamic smem = %d): %s", C::kSmem, cudaGetErrorString(e));
      return FA_ERR_CUDA;
    }
    configured.fetch_or(1ull << ctx.dev, std::memory_order_release);
  }
  DecParams p;
  p.a = a;
  p.rows = a.n * a.group;
  p.row_groups = (p.rows + C::kRows - 1) / C::kRows;
  // The line's counts are 32-bit numbers.
  if ((double)a.B * a.c.H * p.row_groups * ((double)a.c.M * a.c.page / C::kTile + 1) >= 2147483648.0) {
    set_error("B * H_kv * row groups (%d) * table width (%d tokens) is beyond the kernel's index range", p.row_groups,
              a.c.M * a.c.page);
    return FA_ERR_UNSUPPORTED;
  }
  p.max_ctas = ctx.num_sms * C::kCtas;
  if (ctx.max_ctas > 0 && ctx.max_ctas < p.max_ctas) p.max_ctas = ctx.max_ctas;
  p.part_o = reinterpret_cast<float*>(a.ws);
  p.part_ml = reinterpret_cast<float2*>(a.ws + 2LL * p.max_ctas * C::kRows * C::kD * 4);
  kern<<<p.max_ctas, C::kThreads, C::kSmem, ctx.stream>>>(tk, tv, p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = launch_after(cache_join_kernel<C>, dim3((unsigned)(p.row_groups * (C::kRows * C::kD / 512)), (unsigned)a.c.H, (unsigned)a.B),
                     128, ctx.stream, p);
  if (e != cudaSuccess) {
    set_error("cache attention launch failed: %s", cudaGetErrorString(e));
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

// 32 rows a block where 16 would not hold them (and the registers do).
template <int kD, int kKind, bool kF16>
int launch_decode_rows(const CacheAttnParams& a, const LaunchCtx& ctx) {
  if constexpr (kD <= 128) {
    if (a.n * a.group > 16) return launch_decode<DecCfg<kKind, kF16, kD, 2>>(a, ctx);
  }
  return launch_decode<DecCfg<kKind, kF16, kD, 1>>(a, ctx);
}

// Workspace of the attention itself: the parts of cut segments.
template <int kD>
long long decode_workspace_d(const CacheAttnParams& a, int num_sms) {
  if constexpr (kD <= 128) {
    if (a.n * a.group > 16) return decode_workspace<DecCfg<0, false, kD, 2>>(num_sms);
  }
  return decode_workspace<DecCfg<0, false, kD, 1>>(num_sms);
}

template <int kD>
int launch_attn_d(const CacheAttnParams& a, int kind, bool f16, const LaunchCtx& ctx) {
  int rc;
  if (kind == FA_CACHE_E4M3)
    rc = f16 ? launch_decode_rows<kD, kKindE4m3, true>(a, ctx) : launch_decode_rows<kD, kKindE4m3, false>(a, ctx);
  else
    rc = f16 ? launch_decode_rows<kD, kKindInt8, true>(a, ctx) : launch_decode_rows<kD, kKindInt8, false>(a, ctx);
  if (rc != FA_OK || !a.weights) return rc;
  return launch_weights<kD>(a, kind, f16, decode_workspace_d<kD>(a, ctx.num_sms), ctx);
}

template <int kD>
long long attn_workspace_d(const CacheAttnParams& a, int num_sms) {
  return decode_workspace_d<kD>(a, num_sms) + weights_workspace<kD>(a);
}

}  // namespace fa
