// Few-row cache attention, head dim 64.
#include "fa_cache_decode_launch.cuh"

namespace fa {
int launch_decode_d64(const CacheAttnParams& a, int kind, bool f16, const LaunchCtx& ctx) {
  return launch_decode_d<64>(a, kind, f16, ctx);
}
}  // namespace fa
