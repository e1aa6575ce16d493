// Cache attention, head dim 256.
#include "fa_cache_attn_launch.cuh"

namespace fa {
int launch_cache_tree_d256(const CacheAttnParams& a, int kind, bool f16, const LaunchCtx& ctx) {
  return launch_attn_d<256, true>(a, kind, f16, ctx);
}
}  // namespace fa
