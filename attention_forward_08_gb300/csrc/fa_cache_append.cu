// fa_cache_append.cu -- new tokens into the 8-bit cache (include/fa_cache.h).
//
// One thread block owns one cache block of one head, of K or of V: its scale
// depends on all of its new values, and nobody else writes it.  It reads its
// new values once into registers (at most 8 vectors of 8 elements a thread),
// takes their largest magnitude, and stores them rounded.  Tokens that the
// block held are read only when its scale grows.
//
// Bound: memory.  Each new element is read once (2 bytes, or 4) and written
// once (1 byte): 2 x 4096 tokens, 8 heads of 128, bf16: 12.9 us, 3.9 TB/s.  A
// decoding step's few tokens take 2.9 us, a launch and one load's latency.
#include "fa.h"
#include "fa_cache.h"
#include "fa_cache_ops.cuh"
#include "fa_device.h"

namespace fa {
namespace {

constexpr int kMaxVec = 8;  // vectors (8 elements) a thread holds

// Eight elements of the input as fp32.
template <int kDtype>
struct Vec8 {
  uint4 w[kDtype == FA_DTYPE_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, long long elem) {
    if constexpr (kDtype == FA_DTYPE_F32) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(base) + elem);
      w[0] = __ldg(p);
      w[1] = __ldg(p + 1);
    } else {
      w[0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + elem));
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (kDtype == FA_DTYPE_F32) {
      const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
    } else {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (kDtype == FA_DTYPE_BF16) {
          f[2 * i] = __uint_as_float(u[i] << 16);
          f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        } else {
          const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
          f[2 * i] = t.x;
          f[2 * i + 1] = t.y;
        }
      }
    }
  }
};

template <int kKind, int kDtype>
__global__ void __launch_bounds__(512) cache_append_kernel(const AppendParams p) {
  const CacheView& c = p.c;
  const int h = blockIdx.y % c.H, is_v = blockIdx.y / c.H, b = blockIdx.z, tid = threadIdx.x;
  const int n = p.n_new ? min(max(p.n_new[b], 0), p.n) : p.n;
  const int len0 = p.lens[b];
  if (len0 < 0) {
    if (tid == 0) flag_bad_index(c);
    return;
  }
  const long long end = (long long)len0 + n;  // one past the last new position
  const long long m = (len0 >> c.page_log2) + (long long)blockIdx.x, first = m << c.page_log2;
  if (n == 0 || first >= end) return;
  if (m >= c.M) {
    if (tid == 0) flag_bad_index(c);
    return;
  }
  const int block = checked_block(c, c.table, c.table_stride, b, (int)m);
  if (block < 0) return;
  const int held = (int)max(0LL, len0 - first);             // tokens the block held
  const int last = (int)min((long long)c.page, end - first);  // one past its last new slot
  const int t0 = (int)(first + held - len0);                // its first new token's index among the new ones

  const long long* is = is_v ? p.vs : p.ks;
  const void* in = is_v ? p.v : p.k;
  const long long in0 = b * is[0] + h * is[1] + (long long)t0 * is[2];
  const long long* cs = is_v ? c.vs : c.ks;
  uint8_t* out = (is_v ? c.v : c.k) + block * cs[0] + h * cs[1] + held * cs[2];
  float* scale_at = (is_v ? c.v_scale : c.k_scale) + (long long)block * c.H + h;

  const int vd = c.D >> 3;  // vectors a token (a power of two)
  const int vd_log2 = 31 - __clz(vd);
  const int nv = (last - held) * vd;
  Vec8<kDtype> x[kMaxVec];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kMaxVec; ++i) {
    const int v = tid + i * blockDim.x;
    if (v < nv) x[i].load(in, in0 + (long long)(v >> vd_log2) * is[2] + (v & (vd - 1)) * 8);
  }
#pragma unroll
  for (int i = 0; i < kMaxVec; ++i) {
    if (tid + i * (int)blockDim.x < nv) {
      float f[8];
      x[i].get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float a = fabsf(f[e]);
        amax = fmaxf(amax, a < INFINITY ? a : 0.0f);  // infinities and NaN set no scale
      }
    }
  }
  __shared__ float part[16];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if ((tid & 31) == 0) part[tid >> 5] = amax;
  __syncthreads();
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) amax = fmaxf(amax, part[w]);

  const float old = held > 0 ? *scale_at : 0.0f;
  const float s = fmaxf(old, pow2_scale<kKind>(amax));
  __syncthreads();  // everybody has read the old scale
  if (tid == 0) *scale_at = s;
  // x / s; where s is a power of two with a normal inverse (always, but for a
  // caller's own scales), x times its inverse is the same number.
  const uint32_t s_bits = __float_as_uint(s);
  const bool pow2 = (s_bits & 0x7FFFFFu) == 0u && s_bits - 0x00800000u < 0x7E000000u;
  const float inv = __uint_as_float(0x7F000000u - s_bits);
#pragma unroll
  for (int i = 0; i < kMaxVec; ++i) {
    const int v = tid + i * blockDim.x;
    if (v < nv) {
      float f[8];
      x[i].get(f);
      if (pow2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= inv;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __fdiv_rn(f[e], s);
      }
      uint2 r;
      r.x = round8x4<kKind>(f[0], f[1], f[2], f[3]);
      r.y = round8x4<kKind>(f[4], f[5], f[6], f[7]);
      *reinterpret_cast<uint2*>(out + (v >> vd_log2) * cs[2] + (v & (vd - 1)) * 8) = r;
    }
  }
  if (held > 0 && s > old) {  // the tokens it held move to the larger scale
    const float ratio = __fdiv_rn(old, s);
    uint8_t* base = out - held * cs[2];
    for (int v = tid; v < held * vd; v += blockDim.x) {
      uint2* at = reinterpret_cast<uint2*>(base + (v >> vd_log2) * cs[2] + (v & (vd - 1)) * 8);
      const uint2 w = *at;
      float lo[4], hi[4];
      load8x4<kKind>(w.x, lo);
      load8x4<kKind>(w.y, hi);
#pragma unroll
      for (int e = 0; e < 4; ++e) lo[e] = __fmul_rn(lo[e], ratio), hi[e] = __fmul_rn(hi[e], ratio);
      *at = make_uint2(round8x4<kKind>(lo[0], lo[1], lo[2], lo[3]), round8x4<kKind>(hi[0], hi[1], hi[2], hi[3]));
    }
  }
  if (!is_v && (p.weights || p.positions)) {
    for (int t = held + tid; t < last; t += blockDim.x) {
      const long long pos = first + t;
      if (pos >= p.W) {
        flag_bad_index(c);
        break;
      }
      const long long at = ((long long)b * c.H + h) * p.W + pos;
      if (p.weights) p.weights[at] = 0.0f;
      if (p.positions) p.positions[at] = (p.seen ? p.seen[b] : len0) + (int)(pos - len0);
    }
  }
}

template <int kKind, int kDtype>
int launch(const AppendParams& p, const LaunchCtx& ctx) {
  // As many threads as leave each at most kMaxVec vectors of a block's tokens
  // (page * D <= 32768 elements: 512 threads), at least one warp.
  const int vecs = min(p.c.page, p.n) * (p.c.D / 8);
  int threads = 32;
  while (threads * kMaxVec < vecs || (threads < 128 && threads < vecs)) threads *= 2;
  const dim3 grid((unsigned)p.spans, (unsigned)(2 * p.c.H), (unsigned)p.B);
  cache_append_kernel<kKind, kDtype><<<grid, threads, 0, ctx.stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error("cache append launch failed: %s", cudaGetErrorString(e));
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

template <int kKind>
int launch_kind(const AppendParams& p, int dtype, const LaunchCtx& ctx) {
  return dtype == FA_DTYPE_F32    ? launch<kKind, FA_DTYPE_F32>(p, ctx)
         : dtype == FA_DTYPE_BF16 ? launch<kKind, FA_DTYPE_BF16>(p, ctx)
                                  : launch<kKind, FA_DTYPE_F16>(p, ctx);
}

}  // namespace

int launch_cache_append(const AppendParams& p, int kind, int dtype, const LaunchCtx& ctx) {
  return kind == FA_CACHE_E4M3 ? launch_kind<kKindE4m3>(p, dtype, ctx) : launch_kind<kKindInt8>(p, dtype, ctx);
}

}  // namespace fa
