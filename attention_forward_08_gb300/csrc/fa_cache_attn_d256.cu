// Cache attention, head dim 256.
#include "fa_cache_attn_launch.cuh"

namespace fa {
int launch_cache_attn_d256(const CacheAttnParams& a, int kind, bool f16, const LaunchCtx& ctx) {
  return launch_attn_d<256, false>(a, kind, f16, ctx);
}
long long cache_attn_workspace_d256(const CacheAttnParams& a, int num_sms) { return attn_workspace_d<256>(a, num_sms); }
}  // namespace fa
