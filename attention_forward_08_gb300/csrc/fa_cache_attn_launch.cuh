// fa_cache_attn_launch.cuh -- host side of the cache attention kernels for one head
// dim: tensor maps, grid, workspace.
#pragma once

#include <atomic>

#include "fa.h"
#include "fa_cache.h"
#include "fa_cache_decode.cuh"
#include "fa_cache_launch.cuh"
#include "fa_cache_prompt.cuh"
#include "fa_cache_weights.cuh"
#include "fa_cache_maps.h"
#include "fa_device.h"

namespace fa {

// The parts of cut segments: two a thread block.
template <class C>
long long line_workspace(int max_ctas) {
  const long long slots = 2LL * max_ctas * C::kRows;
  return slots * C::kD * 4 + slots * 8;
}

// The line's parameters; false (and the message) beyond its 32-bit counts.
template <class C>
bool line_params(DecParams& p, const CacheAttnParams& a, int max_ctas, const LaunchCtx& ctx) {
  p.a = a;
  p.rows = a.n * a.group;
  p.row_groups = (p.rows + C::kRows - 1) / C::kRows;
  if ((double)a.B * a.c.H * p.row_groups * ((double)a.c.M * a.c.page / C::kTile + 2) >= 2147483648.0) {
    set_error("B * H_kv * row groups (%d) * table width (%d tokens) is beyond the kernel's index range", p.row_groups,
              a.c.M * a.c.page);
    return false;
  }
  p.part_o = reinterpret_cast<float*>(a.ws);
  p.part_ml = reinterpret_cast<float2*>(a.ws + 2LL * max_ctas * C::kRows * C::kD * 4);
  p.scores = nullptr;
  p.max_ctas = ctx.max_ctas > 0 && ctx.max_ctas < max_ctas ? ctx.max_ctas : max_ctas;
  return true;
}

// Rows of a K/V head behind which a call is a prompt's: what the decode kernel
// holds at once.  (Several such groups, each reading every key, lose from the
// second on: 4 sequences of 8192 tokens, 8 heads, D 64: 48 rows 56.0 us against
// 51.4, 128 rows 74.5 against 49.2; D 128: 69.9 against 57.6 and 102.6 against
// 58.2; D 256: 32 rows 78.4 against 77.9, 128 rows 194 against 97.  Just below:
// D 128, 32 rows 37.0 us here, 55.3 there.)
template <int kD>
constexpr int kPromptRows = kD <= 128 ? 32 : 16;

// With weights, the decode kernel keeps its scores, unless a wide table would
// make them large (they take 4 bytes a row for every token that the table could
// hold; the keys are then read twice).  16 sequences of up to 4096 tokens, H
// 32/8, D 128: 33.6 us kept, 46 us read twice.
constexpr long long kMostScores = 256LL << 20;
inline long long score_bytes(const CacheAttnParams& a) {
  return (long long)a.B * a.c.H * (((long long)a.c.M * a.c.page + 31) / 32) * a.n * a.group * 128;
}
template <int kD>
bool keep_scores(const CacheAttnParams& a) {
  return a.weights && (long long)a.n * a.group <= kPromptRows<kD> &&
         (double)a.B * a.c.H * a.c.M * a.c.page * a.n * a.group * 4 <= (double)kMostScores;
}

// Workspace of the accumulated weights, behind the attention's own.
template <int kD>
long long weights_workspace(const CacheAttnParams& a) {
  if (!a.weights) return 0;
  if (keep_scores<kD>(a)) return score_bytes(a);
  const long long groups = (long long)a.B * a.c.H * ((a.n * (long long)a.group + 15) / 16);
  return groups * 16 * (kD * 2 + 8);
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
  CUtensorMap tk{}, tv{};
  if constexpr (C::kTma) {
    const int rows = a.c.page < C::kTile ? a.c.page : C::kTile;
    if (!encode_pool(&tk, a.c, false, rows) || !encode_pool(&tv, a.c, true, rows)) return FA_ERR_CUDA;
  }
  auto kern = cache_decode_kernel<C>;
  static std::atomic<unsigned long long> configured{0};
  DecParams p;
  if (!allow_smem(kern, C::kSmem, ctx.dev, configured)) return FA_ERR_CUDA;
  if (!line_params<C>(p, a, ctx.num_sms * C::kCtas, ctx)) return FA_ERR_UNSUPPORTED;
  if (keep_scores<C::kD>(a)) p.scores = reinterpret_cast<float*>(a.ws + line_workspace<C>(ctx.num_sms * C::kCtas));
  kern<<<p.max_ctas, C::kThreads, C::kSmem, ctx.stream>>>(tk, tv, p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && p.scores) {
    const int joins = (p.max_ctas - 1) * join_pieces<C>(p);
    const long long chunks = ((long long)a.c.M * a.c.page + kFinishTokens - 1) / kFinishTokens;
    if (chunks * a.c.H * a.B > 0x7fffffffLL - joins) {
      set_error("B * H_kv * table width (%lld tokens) is beyond the weights' index range", (long long)a.c.M * a.c.page);
      return FA_ERR_UNSUPPORTED;
    }
    e = launch_after(cache_finish_kernel<C>, dim3((unsigned)(joins + chunks * a.c.H * a.B)), kJoinThreads, ctx.stream, p,
                     joins, (int)chunks);
  } else if (e == cudaSuccess && p.max_ctas > 1) {
    e = launch_after(cache_join_kernel<C>, dim3((unsigned)join_pieces<C>(p), (unsigned)p.max_ctas - 1), kJoinThreads,
                     ctx.stream, p);
  }
  if (e != cudaSuccess) {
    set_error("cache attention launch failed: %s", cudaGetErrorString(e));
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

template <class C>
int launch_prompt(const CacheAttnParams& a, const LaunchCtx& ctx) {
  auto kern = cache_prompt_kernel<C>;
  static std::atomic<unsigned long long> configured{0};
  if (!((configured.load(std::memory_order_acquire) >> ctx.dev) & 1ull)) {
    // The register split inside the kernel assumes 128 a thread at launch; a
    // smaller allocation would make its increases wait forever.
    cudaFuncAttributes attr;
    const cudaError_t e = cudaFuncGetAttributes(&attr, kern);
    if (e != cudaSuccess || attr.numRegs != 128) {
      set_error("kernel register count %d differs from the 128 its register split assumes",
                e == cudaSuccess ? attr.numRegs : -1);
      return FA_ERR_CUDA;
    }
  }
  DecParams p;
  if (!allow_smem(kern, C::kSmem, ctx.dev, configured)) return FA_ERR_CUDA;
  if (!line_params<C>(p, a, ctx.num_sms, ctx)) return FA_ERR_UNSUPPORTED;
  kern<<<p.max_ctas, C::kThreads, C::kSmem, ctx.stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && p.max_ctas > 1)
    e = launch_after(cache_join_kernel<C>, dim3((unsigned)join_pieces<C>(p), (unsigned)p.max_ctas - 1), kJoinThreads,
                     ctx.stream, p);
  if (e != cudaSuccess) {
    set_error("cache attention launch failed: %s", cudaGetErrorString(e));
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

// Which kernel: by the rows of a K/V head.  Up to 16 (the decoding step), 32
// where the registers hold them; else the tensor memory kernel, which always
// computes 128 * kTiles rows.
enum class AttnPlan { kRows16, kRows32, kPrompt };
template <int kD>
AttnPlan attn_plan(const CacheAttnParams& a) {
  const long long rows = (long long)a.n * a.group;
  if (rows > kPromptRows<kD>) return AttnPlan::kPrompt;
  return kD <= 128 && rows > 16 ? AttnPlan::kRows32 : AttnPlan::kRows16;
}

template <int kD>
long long plan_workspace(const CacheAttnParams& a, int num_sms) {
  switch (attn_plan<kD>(a)) {
    case AttnPlan::kPrompt: return line_workspace<PromptCfg<0, false, kD, 16, true>>(num_sms);
    case AttnPlan::kRows32:
      if constexpr (kD <= 128) return line_workspace<DecCfg<0, false, kD, 2, true>>(num_sms * DecCfg<0, false, kD, 2, true>::kCtas);
    default: return line_workspace<DecCfg<0, false, kD, 1, true>>(num_sms * DecCfg<0, false, kD, 1, true>::kCtas);
  }
}

// TMA where a box holds 4 KB and more.  (Blocks of 16 tokens of D 64, int8, 75 MB
// of cache: 36.1 us with boxes of 1 KB, 32.3 with cp.async.  Blocks of 64 of D 128,
// 361 MB: 67.6 us with boxes of 4 KB, 83.7 with cp.async.)
template <int kD, int kKind, bool kF16, int kMT>
int launch_decode_by(const CacheAttnParams& a, const LaunchCtx& ctx) {
  if constexpr (kD >= 128) {
    if (a.c.page >= 32) return launch_decode<DecCfg<kKind, kF16, kD, kMT, true>>(a, ctx);
  }
  return launch_decode<DecCfg<kKind, kF16, kD, kMT, false>>(a, ctx);
}

template <int kD, int kKind, bool kF16>
int launch_plan(const CacheAttnParams& a, const LaunchCtx& ctx) {
  switch (attn_plan<kD>(a)) {
    case AttnPlan::kPrompt:
      if (a.cap_out == 0.0f && a.scale_log2 > 0.0f)
        return a.c.page >= 64 ? launch_prompt<PromptCfg<kKind, kF16, kD, 64, true>>(a, ctx)
                              : launch_prompt<PromptCfg<kKind, kF16, kD, 16, true>>(a, ctx);
      return launch_prompt<PromptCfg<kKind, kF16, kD, 16, false>>(a, ctx);
    case AttnPlan::kRows32:
      if constexpr (kD <= 128) return launch_decode_by<kD, kKind, kF16, 2>(a, ctx);
    default: return launch_decode_by<kD, kKind, kF16, 1>(a, ctx);
  }
}

template <int kD>
int launch_attn_d(const CacheAttnParams& a, int kind, bool f16, const LaunchCtx& ctx) {
  int rc;
  if (kind == FA_CACHE_E4M3)
    rc = f16 ? launch_plan<kD, kKindE4m3, true>(a, ctx) : launch_plan<kD, kKindE4m3, false>(a, ctx);
  else
    rc = f16 ? launch_plan<kD, kKindInt8, true>(a, ctx) : launch_plan<kD, kKindInt8, false>(a, ctx);
  if (rc != FA_OK || !a.weights || keep_scores<kD>(a)) return rc;
  return launch_weights<kD>(a, kind, f16, plan_workspace<kD>(a, ctx.num_sms), ctx);
}

template <int kD>
long long attn_workspace_d(const CacheAttnParams& a, int num_sms) {
  return plan_workspace<kD>(a, num_sms) + weights_workspace<kD>(a);
}

}  // namespace fa
