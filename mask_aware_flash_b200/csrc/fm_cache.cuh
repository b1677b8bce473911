// The 8-bit number format of the paged K/V cache: the scale rule and the conversions, shared by the
// kernels that write a cache (fm_cache.cu) and the one that reads it (fm_cache_attn.cu).
#pragma once

#include <cuda_fp16.h>

#include "fm_common.cuh"

namespace fm {

constexpr int kPage = FM_CACHE_PAGE;
constexpr int kMaxCacheB = 65535;  // sequences: a grid dimension

// Host checks of a cache's shape and pointers (fm_cache.cu).
fm_status check_cache(const fm_kv_cache* c);

template <bool E4M3>
__device__ __forceinline__ float code_max() { return E4M3 ? 448.f : 127.f; }

// The smallest power of two s >= 2^-126 with Qmax * s >= amax (0 for 0).  With amax = m 2^k, 1 <= m < 2,
// and Qmax = M 2^K: s = 2^(k - K), or twice that where m > M.  (Subnormal amax: the lower bound.)
template <bool E4M3>
__device__ __forceinline__ float scale_rule(float amax) {
  constexpr uint32_t kM = E4M3 ? 0x600000u : 0x7E0000u;  // mantissa fields of 448 and of 127
  constexpr int kK = E4M3 ? 8 : 6;
  if (!(amax > 0.f)) return 0.f;
  const uint32_t bits = __float_as_uint(amax);
  const int e = (int)(bits >> 23) - 127 - kK + ((bits & 0x7FFFFFu) > kM ? 1 : 0);
  return __uint_as_float((uint32_t)(max(e, -126) + 127) << 23);
}

// |x| where x is finite, else 0
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

// Four values (already divided by their scale) -> four codes, the first in the low byte.  Rounded to
// nearest even, as both formats hold no more: half a step of the block's scale (int8) or half a unit of
// e4m3's 4-bit significand.  kSafe: any values; otherwise finite ones within the format's range (the values
// of a block without infinities and NaN, whose scale the rule above gives).  int8 in range: adding 1.5 * 2^23
// rounds to an integer whose two's complement low byte is the low byte of the sum's word.
template <bool E4M3, bool kSafe>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  float x[4] = {a, b, c, d};
  if constexpr (kSafe) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = x[i] == x[i] ? x[i] : 0.f;
      x[i] = fminf(fmaxf(x[i], -code_max<E4M3>()), code_max<E4M3>());
    }
  }
  if constexpr (E4M3) {
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
    return r;
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(x[i] + 12582912.f);
    return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
  }
}

// Four codes as two packed fp16 pairs (exact: both formats' values have at most 8 significant bits).
// int8: code ^ 0x80 is code + 128 in [0, 255]; put under the exponent byte 0x64 it is the fp16 number
// 1024 + 128 + code, and subtracting 1152 leaves the code.
template <bool E4M3>
__device__ __forceinline__ void decode4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E4M3) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    const uint32_t x = w ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    const __half2 ha = __hsub2(*reinterpret_cast<__half2*>(&a), bias), hb = __hsub2(*reinterpret_cast<__half2*>(&b), bias);
    lo = *reinterpret_cast<const uint32_t*>(&ha);
    hi = *reinterpret_cast<const uint32_t*>(&hb);
  }
}
template <bool E4M3>
__device__ __forceinline__ void decode4f(uint32_t w, float (&x)[4]) {
  uint32_t lo, hi;
  decode4<E4M3>(w, lo, hi);
  const float2 a = __half22float2(*reinterpret_cast<__half2*>(&lo)), b = __half22float2(*reinterpret_cast<__half2*>(&hi));
  x[0] = a.x;
  x[1] = a.y;
  x[2] = b.x;
  x[3] = b.y;
}

}  // namespace fm
