// w4_quant.cuh — codes of fp16 / bf16 values: exact steps shared by the per-token
// quantizer (w4_quant.cu) and the key-value cache's writer (w4_cache.cu).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace w4 {
namespace {

template <typename T>
__device__ __forceinline__ float2 pair_f32(uint32_t v);
template <>
__device__ __forceinline__ float2 pair_f32<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <>
__device__ __forceinline__ float2 pair_f32<__nv_bfloat16>(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}
template <typename T>
__device__ __forceinline__ float one_f32(T x);
template <>
__device__ __forceinline__ float one_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float one_f32<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}

// Running maximum of |x| over pairs of 16-bit values, kept packed: the
// maximum is exact in the input type, so it is taken there (one instruction
// per pair) and converted to fp32 once per thread.
template <typename T>
struct Pair16;
template <>
struct Pair16<__half> {
  using P = __half2;
  static __device__ __forceinline__ P zero() { return __float2half2_rn(0.f); }
  static __device__ __forceinline__ P amax(P m, uint32_t v) {
    return __hmax2(m, __habs2(*reinterpret_cast<const __half2*>(&v)));
  }
  static __device__ __forceinline__ float to_f32(P m) {
    return fmaxf(__low2float(m), __high2float(m));
  }
};
template <>
struct Pair16<__nv_bfloat16> {
  using P = __nv_bfloat162;
  static __device__ __forceinline__ P zero() { return __float2bfloat162_rn(0.f); }
  static __device__ __forceinline__ P amax(P m, uint32_t v) {
    return __hmax2(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&v)));
  }
  static __device__ __forceinline__ float to_f32(P m) {
    return fmaxf(__low2float(m), __high2float(m));
  }
};
template <typename T>
__device__ __forceinline__ typename Pair16<T>::P amax8(typename Pair16<T>::P m, const uint4& v) {
  m = Pair16<T>::amax(m, v.x);
  m = Pair16<T>::amax(m, v.y);
  m = Pair16<T>::amax(m, v.z);
  return Pair16<T>::amax(m, v.w);
}

// int8 codes without a division per element: with r = 1/s rounded once to
// fp32, the product p = fl(x * r) differs from fl(x / s) by at most
// |x / s| * (2^-23 + 2^-24 + 2^-47) < 2.3e-5 for |x / s| <= 127 + 2^-16; so
// when p is farther than 2^-15 from every half-integer, both round to the
// same integer (ties to even only matter exactly at a half-integer), and
// only the few quotients that close are divided exactly.  (s below 2^-128
// makes r infinite: then every code takes the division.)

// fast: r = 1/s is finite (s below 2^-128 takes the division everywhere)
__device__ __forceinline__ float code_s8_fast(float x, float s, float r, bool fast) {
  const float p = x * r;
  const float d = fabsf(p - truncf(p));  // distance above the integer toward zero
  float q = (!fast || fabsf(d - 0.5f) <= 0x1p-15f) ? rintf(__fdiv_rn(x, s)) : rintf(p);
  return fminf(fmaxf(q, -127.f), 127.f);
}

// The eight int8 codes of f[] (|f| <= amax, so every code is within
// [-127, 127]), rounded to nearest even, as t[e] = code + 1.5 * 2^23: adding
// that constant to a value of magnitude below 2^22 rounds it to an integer
// (nearest even, the FADD's own rounding) held in the low mantissa bits, so
// the low byte of t's bit pattern is the two's-complement code and t - 1.5 *
// 2^23 its exact value.  Codes come from the products p with r; a product
// whose distance to the nearest integer is 0.5 - 2^-15 or more (within
// 2^-15 of a half-integer), or any product when r is not finite, is replaced
// by the code of the exact quotient, in a branch taken for few vectors.
constexpr float kRoundMagic = 12582912.f;  // 1.5 * 2^23
__device__ __forceinline__ void codes8_s8(const float (&f)[8], float s, float r, bool fast,
                                          float (&t)[8]) {
  // explicitly rounded operations: none may be fused or reassociated
  float dmax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float p = __fmul_rn(f[e], r);
    t[e] = __fadd_rn(p, kRoundMagic);
    dmax = fmaxf(dmax, fabsf(__fsub_rn(p, __fsub_rn(t[e], kRoundMagic))));
  }
  if (!fast || dmax >= 0.5f - 0x1p-15f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float p = __fmul_rn(f[e], r);
      if (!fast || fabsf(__fsub_rn(p, __fsub_rn(t[e], kRoundMagic))) >= 0.5f - 0x1p-15f)
        t[e] = __fadd_rn(__fdiv_rn(f[e], s), kRoundMagic);
    }
  }
}

// Low bytes of four ints, in order, in one word.
__device__ __forceinline__ uint32_t pack4_s8(int a, int b, int c, int d) {
  uint32_t lo, hi, r;
  asm("prmt.b32 %0, %1, %2, 0x0040;" : "=r"(lo) : "r"(a), "r"(b));
  asm("prmt.b32 %0, %1, %2, 0x0040;" : "=r"(hi) : "r"(c), "r"(d));
  asm("prmt.b32 %0, %1, %2, 0x5410;" : "=r"(r) : "r"(lo), "r"(hi));
  return r;
}

// E4M3 byte of the correctly rounded quotient x / s: nearest-even,
// saturated at 448
__device__ __forceinline__ uint32_t code_e4m3(float x, float s) {
  uint16_t e2;
  const float v = __fdiv_rn(x, s);
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e2) : "f"(0.f), "f"(v));
  return e2 & 0xFFu;
}

}  // namespace
}  // namespace w4
