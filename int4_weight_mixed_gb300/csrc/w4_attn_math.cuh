// w4_attn_math.cuh — what the attention kernels compute with: codes as 16-bit
// values, exponentials.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace w4 {
namespace {

// A row's running maximum moves only when the maximum grows by more than this
// (log2), so that sums are seldom rescaled (a published method): probabilities
// relative to it reach 2^8 (2^9 in the kernel that rounds it to a whole number).
// They enter the product with the values 2^7 (2^6) times as large, up to 2^15: fp16
// then holds half a step of 2^-11 of a probability down to 2^-20 of the row's largest
// one, and 2^-31 of that one below.
constexpr float kSlack = 8.f;
constexpr int kDecLift = 7, kTcLift = 6;
// log2 vs of a key that is none: far below any score, and still a number.
constexpr float kNoKey = -0x1p120f;
// Where its logarithm is taken, a value's scale counts as this at least (the
// cache's writer makes none smaller but 0) ...
constexpr float kLeastScale = 0x1p-100f;
// ... and that of a row of zeros, which weighs in a row's sum alone, as this.  A p
// below 2^-126 is lost from the sum, so it must not lie too far below the other
// values' scales; nor above them, or theirs would leave fp16.
constexpr float kZeroScale = 0x1p-60f;

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// A value's scale, as it counts in exponents.  (A NaN is dealt with elsewhere.)
__device__ __forceinline__ float counted(float vs) {
  return vs > 0.f ? fmaxf(vs, kLeastScale) : kZeroScale;
}

// Four codes as two pairs of fp16.  int8: 1024 + (code + 128) by its bits, less
// 1152, exactly.
template <bool E4M3>
__device__ __forceinline__ void codes4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E4M3) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    const uint32_t x = w ^ 0x80808080u;
    const __half2 c = __half2half2(__ushort_as_half(0x6480));  // 1152
    const uint32_t a = prmt(x, 0x64646464u, 0x4140), b = prmt(x, 0x64646464u, 0x4342);
    const __half2 ha = __hsub2(*reinterpret_cast<const __half2*>(&a), c);
    const __half2 hb = __hsub2(*reinterpret_cast<const __half2*>(&b), c);
    lo = *reinterpret_cast<const uint32_t*>(&ha);
    hi = *reinterpret_cast<const uint32_t*>(&hb);
  }
}

// The same as bf16, times 2^-8, exactly: so products with queries, which bf16 lets be
// as large as fp32's largest number, leave fp32 2^8 later.  int8: with the code's low
// seven bits u and sign bit s, code = (128 + u) - (128 + 128 s), and bf16 holds
// (128 + u) 2^-8 as 0x3F00 | u, (128 + 128 s) 2^-8 as 0x3F00 | s << 7.  E4M3: the
// code's exponent and mantissa at bf16's place are the value times 2^-120, subnormals
// too.
constexpr float kBf16Code = 0x1p-8f;
template <bool E4M3>
__device__ __forceinline__ void codes4_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E4M3) {
    const __nv_bfloat162 up = __bfloat162bfloat162(__ushort_as_bfloat16(0x7780));  // 2^112
    const uint32_t a = prmt(w, 0u, 0x1404), b = prmt(w, 0u, 0x3424);
    const uint32_t x = (a & 0x80008000u) | (a >> 4 & 0x07F007F0u);
    const uint32_t y = (b & 0x80008000u) | (b >> 4 & 0x07F007F0u);
    const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&x), up);
    const __nv_bfloat162 q = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&y), up);
    lo = *reinterpret_cast<const uint32_t*>(&p);
    hi = *reinterpret_cast<const uint32_t*>(&q);
  } else {
    const uint32_t a = prmt(w, 0x3F3F3F3Fu, 0x4140), b = prmt(w, 0x3F3F3F3Fu, 0x4342);
    const uint32_t au = a & 0xFF7FFF7Fu, as = a & 0xFF80FF80u;
    const uint32_t bu = b & 0xFF7FFF7Fu, bs = b & 0xFF80FF80u;
    const __nv_bfloat162 p = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&au),
                                     *reinterpret_cast<const __nv_bfloat162*>(&as));
    const __nv_bfloat162 q = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&bu),
                                     *reinterpret_cast<const __nv_bfloat162*>(&bs));
    lo = *reinterpret_cast<const uint32_t*>(&p);
    hi = *reinterpret_cast<const uint32_t*>(&q);
  }
}

// Two fp32 operations at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 w, x, y;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// The largest of three (a NaN counts as none).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

}  // namespace
}  // namespace w4
