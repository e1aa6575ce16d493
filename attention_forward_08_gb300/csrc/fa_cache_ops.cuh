// fa_cache_ops.cuh -- device helpers of the 8-bit cache kernels: the stored
// types, table look-ups that check their entry, and power-of-two scales.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "fa_cache_params.h"

namespace fa {

constexpr int kKindE4m3 = 0, kKindInt8 = 1;

// Two stored bytes (low 16 bits) -> f16x2, exact for both kinds.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

// Four stored bytes -> two f16x2 (bytes 0, 1 and bytes 2, 3), exact.  int8: a
// byte u = x + 128 in the low mantissa bits of 1024 is the number 1024 + u.
template <int kKind>
__device__ __forceinline__ void to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (kKind == kKindE4m3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 ha = __hsub2(*reinterpret_cast<__half2*>(&a), off), hb = __hsub2(*reinterpret_cast<__half2*>(&b), off);
    lo = *reinterpret_cast<uint32_t*>(&ha);
    hi = *reinterpret_cast<uint32_t*>(&hb);
  }
}

// Round to the stored type, to nearest even.  e4m3 saturates infinities and
// keeps NaN; int8 clamps to +-127 and stores NaN as 0.
template <int kKind>
__device__ __forceinline__ uint32_t round8x4(float a, float b, float c, float d) {
  if constexpr (kKind == kKindE4m3) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\tmov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
  } else {
    auto one = [](float x) -> uint32_t {
      return (x != x ? 0u : (uint32_t)__float2int_rn(fminf(fmaxf(x, -127.0f), 127.0f))) & 0xFFu;
    };
    return one(a) | (one(b) << 8) | (one(c) << 16) | (one(d) << 24);
  }
}

// Four stored bytes -> fp32.
template <int kKind>
__device__ __forceinline__ void load8x4(uint32_t w, float (&f)[4]) {
  if constexpr (kKind == kKindE4m3) {
    const uint32_t lo = e4m3x2_to_f16x2(w & 0xFFFFu), hi = e4m3x2_to_f16x2(w >> 16);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(w >> (8 * i));
  }
}

// The least power of two s >= 2^-100 with amax <= MAX * s (amax finite, >= 0):
// with amax = m * 2^e and MAX = m0 * 2^e0 (m, m0 in [1, 2)) it is 2^(e - e0),
// once more where m > m0.  The comparison is on the bits: nothing is rounded.
template <int kKind>
__device__ __forceinline__ float pow2_scale(float amax) {
  constexpr uint32_t kM0 = kKind == kKindE4m3 ? 0x600000u : 0x7E0000u;  // 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6
  constexpr int kE0 = kKind == kKindE4m3 ? 8 : 6;
  const uint32_t bits = __float_as_uint(amax);
  const int e = (int)(bits >> 23) - 127 - kE0 + ((bits & 0x7FFFFFu) > kM0 ? 1 : 0);
  return __uint_as_float((uint32_t)(max(e, -100) + 127) << 23);  // amax 0 and denormals: 2^-100
}

__device__ __forceinline__ void flag_bad_index(const CacheView& c) { atomicOr(c.status, kStatusBadIndex); }

// Tokens that sequence b holds, kept inside the table.
__device__ __forceinline__ int checked_len(const CacheView& c, int len) {
  const long long most = (long long)c.M * c.page;
  if (len < 0 || len > most) {
    flag_bad_index(c);
    return len < 0 ? 0 : (int)most;
  }
  return len;
}

// A table's entry, or -1 for one out of range: without telling, or telling.
__device__ __forceinline__ int checked_block_quiet(const CacheView& c, const int* table, long long stride, int b, int m) {
  const int at = table[b * stride + m];
  return at < 0 || at >= c.P ? -1 : at;
}
// The block of sequence b's tokens m * page ..
__device__ __forceinline__ int checked_block(const CacheView& c, const int* table, long long stride, int b, int m) {
  const int at = table[b * stride + m];
  if (at < 0 || at >= c.P) {
    flag_bad_index(c);
    return -1;
  }
  return at;
}

}  // namespace fa
