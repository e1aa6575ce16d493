// fa_cache_rescale.cuh -- stored bytes brought to another block's scale.
#pragma once

#include "fa_cache_ops.cuh"

namespace fa {

// Sixteen stored bytes of scale `from`, rounded to scale `to`.
template <int kKind>
__device__ __forceinline__ uint4 rescale16(uint4 w, float from, float to) {
  if (from == to) return w;
  const float ratio = __fdiv_rn(from, to);
  uint32_t* u = &w.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[4];
    load8x4<kKind>(u[i], f);
    u[i] = round8x4<kKind>(__fmul_rn(f[0], ratio), __fmul_rn(f[1], ratio), __fmul_rn(f[2], ratio), __fmul_rn(f[3], ratio));
  }
  return w;
}

}  // namespace fa
