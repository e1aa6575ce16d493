// fa_cache_maps.h -- the tensor map of a cache pool.
#pragma once

#include <cuda.h>

#include "fa_cache_params.h"
#include "fa_device.h"

namespace fa {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn get_encode_tiled();  // defined in fa_api.cu

// K or V as {D, page, H, P} bytes, tiled as {min(D, 128), rows, 1, 1}, swizzled
// over the whole row of a tile (128 bytes; 64 for D = 64).
inline bool encode_pool(CUtensorMap* map, const CacheView& c, bool v, int rows) {
  const long long* s = v ? c.vs : c.ks;
  cuuint64_t dims[4] = {(cuuint64_t)c.D, (cuuint64_t)c.page, (cuuint64_t)c.H, (cuuint64_t)c.P};
  // A stride of an extent-1 dimension is never used; give it a legal value.
  cuuint64_t strides[3] = {(cuuint64_t)s[2], (cuuint64_t)(c.H > 1 ? s[1] : 16), (cuuint64_t)(c.P > 1 ? s[0] : 16)};
  cuuint32_t box[4] = {(cuuint32_t)(c.D < 128 ? c.D : 128), (cuuint32_t)rows, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) {
    set_error("cuTensorMapEncodeTiled is not available from the CUDA driver");
    return false;
  }
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, v ? c.v : c.k, dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, c.D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled (cache pool) failed (CUresult %d)", (int)r);
    return false;
  }
  return true;
}

}  // namespace fa
