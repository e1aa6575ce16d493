// Few-row cache attention, head dim 128.
#include "fa_cache_decode_launch.cuh"

namespace fa {
int launch_decode_d128(const CacheAttnParams& a, int kind, bool f16, const LaunchCtx& ctx) {
  return launch_decode_d<128>(a, kind, f16, ctx);
}
}  // namespace fa
