// Codes of 8 bits with a power of two as their scale: what a value becomes, and back.
//
// The scale of some values with largest magnitude m is 2^e, e >= -126 the smallest
// with m <= top * 2^e. Multiplying by 2^e or 2^-e is exact (but for results that are
// subnormal in FP32), so a code is x rounded once, to the nearest, ties to even,
// and a larger scale for codes is the same step again. A magnitude's float bits carry both
// parts of the choice: the exponent, and whether the fraction is above top's own.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_internal.h"

namespace tfx {

constexpr uint32_t kInfBits = 0x7f800000u;  // from here on: infinities and NaN
constexpr float kLeastScale = 1.1754943508222875e-38f;  // 2^-126

// top = (1 + kFraction / 2^23) * 2^kPlace
template <int Store>
struct Code;
template <>
struct Code<TFX_STORE_I8> {
  static constexpr int kPlace = 6;
  static constexpr uint32_t kFraction = 0x7e0000u;  // 127 = 1.984375 * 2^6
};
template <>
struct Code<TFX_STORE_E4M3> {
  static constexpr int kPlace = 8;
  static constexpr uint32_t kFraction = 0x600000u;  // 448 = 1.75 * 2^8
};

// The scale that magnitudes of up to the float with these bits need; NaN where it is not finite.
template <int Store>
__device__ __forceinline__ float scale_for(uint32_t bits) {
  if (bits >= kInfBits) return __uint_as_float(0x7fc00000u);
  const int e = (int)(bits >> 23) - Code<Store>::kPlace + ((bits & 0x7fffffu) > Code<Store>::kFraction);
  return __uint_as_float((uint32_t)max(e, 1) << 23);  // at least 2^-126
}
// 1 / scale, for powers of two of at least 2^-126 and at most 2^126; NaN of a NaN.
__device__ __forceinline__ float inverse_of(float scale) {
  return __uint_as_float(scale == scale ? 0x7f000000u - __float_as_uint(scale) : 0x7fc00000u);
}
// A NaN stays.
__device__ __forceinline__ float larger_scale(float a, float b) { return a != a || a > b ? a : b; }

// Codes of four values times inv, which is a power of two and brings them into the codes'
// range; NaN becomes any code. For I8, one rounded operation adds 1.5 * 2^23, which leaves the
// nearest whole number, ties to even, in the low bits (the conversion instruction runs at an
// eighth of its rate).
template <int Store>
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d, float inv);
template <>
__device__ __forceinline__ uint32_t code4<TFX_STORE_I8>(float a, float b, float c, float d, float inv) {
  const float by = 12582912.f;
  const uint32_t lo = __byte_perm(__float_as_uint(__fmaf_rn(a, inv, by)), __float_as_uint(__fmaf_rn(b, inv, by)), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(__fmaf_rn(c, inv, by)), __float_as_uint(__fmaf_rn(d, inv, by)), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}
template <>
__device__ __forceinline__ uint32_t code4<TFX_STORE_E4M3>(float a, float b, float c, float d, float inv) {
  uint32_t r;
  asm("{ .reg .b16 lo, hi; cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1; cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3; mov.b32 %0, {lo, hi}; }"
      : "=r"(r)
      : "f"(a * inv), "f"(b * inv), "f"(c * inv), "f"(d * inv));
  return r;
}

// The four codes of a word as FP16: bytes (0, 1) and (2, 3), or (0, 2) and (1, 3).
template <int Store, bool Split>
__device__ __forceinline__ void halves(uint32_t w, uint32_t& a, uint32_t& b) {
  if constexpr (Store == TFX_STORE_I8) {
    // 0x64xx is 1024 + xx
    w ^= 0x80808080u;
    const uint32_t x = __byte_perm(w, 0x64646464u, Split ? 0x4240 : 0x4140);
    const uint32_t y = __byte_perm(w, 0x64646464u, Split ? 0x4341 : 0x4342);
    const __half2 by = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 p = __hsub2(*reinterpret_cast<const __half2*>(&x), by);
    const __half2 q = __hsub2(*reinterpret_cast<const __half2*>(&y), by);
    a = *reinterpret_cast<const uint32_t*>(&p);
    b = *reinterpret_cast<const uint32_t*>(&q);
  } else {
    if (Split) w = __byte_perm(w, 0, 0x3120);
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.rn.f16x2.e4m3x2 %0, lo; cvt.rn.f16x2.e4m3x2 %1, hi; }"
        : "=r"(a), "=r"(b)
        : "r"(w));
  }
}

// log2 of a scale, NaN of a NaN.
__device__ __forceinline__ float log2_scale(float s) {
  return s == s ? (float)((int)(__float_as_uint(s) >> 23) - 127) : s;
}

// Values of the four codes in a word.
template <int Store>
__device__ __forceinline__ void values4(uint32_t w, float (&x)[4]) {
  uint32_t a, b;
  halves<Store, false>(w, a, b);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&a)), g = __half22float2(*reinterpret_cast<const __half2*>(&b));
  x[0] = f.x;
  x[1] = f.y;
  x[2] = g.x;
  x[3] = g.y;
}

// BF16 values whose largest magnitude has the bits `top`: the power of two that brings it to
// [2^14, 2^15), where FP16 holds them exactly but for those 2^28 times smaller; at most 2^126.
__device__ __forceinline__ float brings_up(uint32_t top) { return __uint_as_float((268u - max(top >> 7, 15u)) << 23); }

__device__ __forceinline__ float2 pair_to_float(uint32_t w, __half) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ float2 pair_to_float(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

}  // namespace tfx
