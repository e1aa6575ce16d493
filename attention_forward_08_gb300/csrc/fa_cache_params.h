// fa_cache_params.h -- parameter blocks of the 8-bit cache kernels (by value,
// as kernel arguments) and the host functions that launch them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_device.h"
#include "fa_params.h"

namespace fa {

// Pools, scales and the page table, as fa_cache.h describes them.
struct CacheView {
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  long long ks[3], vs[3];  // byte strides: block, head, token
  int P, H, page, D;
  int page_log2;
  const int* table;
  long long table_stride;
  int M;
  unsigned int* status;
};

struct AppendParams {
  CacheView c;
  const void *k, *v;
  long long ks[3], vs[3];  // element strides: batch, head, token
  const int *lens, *n_new, *seen;
  float* weights;
  int* positions;
  int B, n, W;
  int spans;  // blocks that n tokens can touch
};

struct CacheAttnParams {
  CacheView c;
  const void* q;
  void* o;
  float* lse;
  float* weights;
  long long qs[3], os[3];  // element strides: batch, head, row
  const int *lens, *n_q;
  const int* tree;         // [B, n], row stride tree_stride: the rows' parents; NULL: each row follows the one before
  long long tree_stride;
  int B, Hq, group, n, W;
  int causal, window;
  float scale_log2;             // scale * log2(e)
  float cap_in, cap_out;        // softcap: scale / cap and cap * log2(e); cap_out 0: off
  long long timeout_cycles;
  uint8_t* ws;                  // workspace
};

struct EvictParams {
  CacheView c;
  const int* lens;
  float* weights;
  int* positions;
  const int* into;
  long long into_stride;
  float* weights_out;
  int* positions_out;
  int* lens_out;
  int B, W, M_into, W_out;
  int keep, recent;
  // Workspace: what the choice tells the moves.
  int* src;         // [B, H, keep]: a copy: the slot whose token ends in slot j; in place: the receiving slots, in order
  int* mover;       // [B, H, keep]: in place: kept slots at `keep` and behind, in order
  int* count;       // [B, H]: tokens kept
};

constexpr int kMostDrafts = 1024;  // nodes of a sequence's tree

struct AcceptParams {
  CacheView c;
  const int *lens, *n_q;
  const int* path;  // [B, n], row stride path_stride
  long long path_stride;
  const int* count;
  float* weights;
  int* lens_out;
  int B, n, W;
};

struct VerifyParams {
  const void *p, *q;              // probabilities; q may be NULL
  long long ps[2], qs[2];         // element strides: batch, row
  const int *tokens, *tree;
  long long tokens_stride, tree_stride;
  const float *u, *u_next;
  long long u_stride;
  const int* n_q;
  int *path, *count, *token;      // path [B, n] contiguous
  int B, n, V;
  int blocks, seg;                // blocks a sequence, vocabulary entries a warp (set by the launch)
  unsigned int* status;
};

struct LaunchCtx {
  cudaStream_t stream;
  int num_sms;
  int dev;
  int max_ctas;  // 0: no cap (fa_set_max_ctas)
};

int launch_cache_append(const AppendParams& p, int kind, int dtype, const LaunchCtx& ctx);
// One head dim each (fa_cache_attn_d*.cu).
int launch_cache_attn_d64(const CacheAttnParams& p, int kind, bool f16, const LaunchCtx& ctx);
int launch_cache_attn_d128(const CacheAttnParams& p, int kind, bool f16, const LaunchCtx& ctx);
int launch_cache_attn_d256(const CacheAttnParams& p, int kind, bool f16, const LaunchCtx& ctx);
int launch_cache_tree_d64(const CacheAttnParams& p, int kind, bool f16, const LaunchCtx& ctx);  // (fa_cache_tree_d*.cu)
int launch_cache_tree_d128(const CacheAttnParams& p, int kind, bool f16, const LaunchCtx& ctx);
int launch_cache_tree_d256(const CacheAttnParams& p, int kind, bool f16, const LaunchCtx& ctx);
long long cache_attn_workspace_d64(const CacheAttnParams& p, int num_sms);
long long cache_attn_workspace_d128(const CacheAttnParams& p, int num_sms);
long long cache_attn_workspace_d256(const CacheAttnParams& p, int num_sms);
int launch_cache_evict(const EvictParams& p, int kind, const LaunchCtx& ctx);
int launch_cache_accept(const AcceptParams& p, int kind, const LaunchCtx& ctx);
int launch_verify(VerifyParams p, int dtype, const LaunchCtx& ctx);

}  // namespace fa
