// asp_kv8.cuh -- values held in 8 bits: codes, scales and their conversions.
//
// A value is code * scale with one scale per block of tokens, KV head and side.
// E4M3 codes (1-4-3, largest 448) and I8 codes (integers in [-127, 127]) both fit
// fp16 exactly, so a pair of codes becomes an fp16x2 matrix operand without
// rounding and the scales stay outside the products.
#pragma once

#include <cuda_fp16.h>

#include "asp_common.cuh"

namespace asp {

struct CodeE4M3 {
  // packed magnitudes of four codes, and whether one of them is NaN
  __device__ __forceinline__ static uint32_t mag4(uint32_t w) { return w & 0x7f7f7f7fu; }
  static constexpr uint32_t kNanMag = 0x7fu;
  __device__ __forceinline__ static float mag_value(uint32_t m) {   // of one magnitude
    const uint32_t h = pair(m, 0);
    return __half2float(__ushort_as_half((unsigned short)h));
  }
  // four codes times a power of two f in [2^-24, 2^15], encoded again: every product that is
  // not exact in fp16 rounds to the code 0 either way
  __device__ __forceinline__ static uint32_t rescale4(uint32_t w, __half2 f) {
    const uint32_t a = pair(w, 0), b = pair(w, 1);
    const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&a), f);
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&b), f);
    unsigned short lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(lo) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(hi) : "r"(*reinterpret_cast<const uint32_t*>(&y)));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  }
  // frexp mantissa of the largest code, 448 = 0.875 * 2^9: the fraction bits above
  // which a value needs the next power of two, and the exponent it is taken off
  static constexpr uint32_t kTopFrac = 0x600000u;
  static constexpr int kShift = 9;
  static constexpr float kMax = 448.f;
  // two codes (low, high byte) -> fp16x2 (low, high half), exact
  __device__ __forceinline__ static uint32_t pair(uint32_t w, int half) {
    uint32_t r;
    const unsigned short h = (unsigned short)(half ? (w >> 16) : w);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
    return r;
  }
  // what pair() takes: the codes as stored
  __device__ __forceinline__ static uint32_t prep(uint32_t w) { return w; }
  __device__ __forceinline__ static uint32_t encode4(float a, float b, float c, float d) {
    unsigned short lo, hi;   // nearest code, ties to even, infinities to +-448, NaN to NaN
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  }
};

struct CodeI8 {
  __device__ __forceinline__ static uint32_t mag4(uint32_t w) { return __vabs4(w); }
  static constexpr uint32_t kNanMag = 0x1ffu;   // none
  __device__ __forceinline__ static float mag_value(uint32_t m) { return (float)m; }
  // as above; 1536 + x rounds x to an integer, whose low byte is then the code's
  __device__ __forceinline__ static uint32_t rescale4(uint32_t w, __half2 f) {
    const uint32_t p = prep(w), a = pair(p, 0), b = pair(p, 1), m = 0x66006600u;
    const __half2 x = __hfma2(*reinterpret_cast<const __half2*>(&a), f, *reinterpret_cast<const __half2*>(&m));
    const __half2 y = __hfma2(*reinterpret_cast<const __half2*>(&b), f, *reinterpret_cast<const __half2*>(&m));
    return __byte_perm(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y), 0x6420);
  }
  static constexpr uint32_t kTopFrac = 0x7e0000u;   // 127 = 0.9921875 * 2^7
  static constexpr int kShift = 7;
  static constexpr float kMax = 127.f;
  // The biased byte u = code + 128 below the fp16 pattern 0x6400 is 1024 + u; less 1152
  // it is the code, exact.
  __device__ __forceinline__ static uint32_t prep(uint32_t w) { return w ^ 0x80808080u; }
  __device__ __forceinline__ static uint32_t pair(uint32_t w, int half) {
    const uint32_t b = __byte_perm(w, 0x64646464u, half ? 0x4342 : 0x4140);
    const uint32_t off = 0x64806480u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&b), *reinterpret_cast<const __half2*>(&off));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  __device__ __forceinline__ static uint32_t code(float x) {   // NaN converts to 0
    const int i = __float2int_rn(x);
    return (uint32_t)(i < -127 ? -127 : (i > 127 ? 127 : i)) & 0xffu;
  }
  __device__ __forceinline__ static uint32_t encode4(float a, float b, float c, float d) {
    return code(a) | (code(b) << 8) | (code(c) << 16) | (code(d) << 24);
  }
};

// Four codes of a word as fp32.
template <typename CT>
__device__ __forceinline__ void decode4(uint32_t w, float (&v)[4]) {
  const uint32_t p = CT::prep(w);
  const uint32_t a = CT::pair(p, 0), b = CT::pair(p, 1);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
  v[0] = x.x;
  v[1] = x.y;
  v[2] = y.x;
  v[3] = y.y;
}

constexpr int kMinScaleExp = -100;

// Exponent of the smallest power of two s >= 2^-100 with amax <= qmax * s; amax given
// by its bits (finite, sign cleared).
template <typename CT>
__device__ __forceinline__ int scale_exp(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 127 + 1 - CT::kShift + ((amax_bits & 0x7fffffu) > CT::kTopFrac ? 1 : 0);
  return e < kMinScaleExp ? kMinScaleExp : e;
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // -126..127

// |x| bits, 0 for an infinity or NaN (`bad` is then set, where given)
__device__ __forceinline__ uint32_t finite_abs(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}
__device__ __forceinline__ uint32_t finite_abs(float x, bool& bad) {
  bad |= (__float_as_uint(x) & 0x7fffffffu) >= 0x7f800000u;
  return finite_abs(x);
}

}  // namespace asp
