#pragma once
// w4_epilogue.cuh — the output step shared by every GEMM engine.
//
//   W4A16: out[m][n] = round_T(sum + bias[n])            (T = fp16 / bf16)
//   W4A8 : out[m][n] = fp16_rn((float)acc * s_tok[m] * s_ch[n] + bias[n])
//          or the raw int32 accumulator (no scales, no bias); with fp8
//          activations acc is the fp32 sum of the exact products
//
// The sum is the fp32 (W4A16) or exact int32 (W4A8) result of the product;
// the products by the per-token and per-channel scales are taken left to
// right in fp32 (vLLM PR #6547 "Enable Dynamic Per Token fp8": per-token x
// per-channel scales applied in the epilogue); the optional bias [N], of the
// output type, is added in fp32 before the single rounding to the output
// type (the vLLM "rdna_hybrid_w4a16" page adds the layer bias to the GEMM
// result, _rdna_hybrid_w4a16_apply_impl).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "w4_internal.h"

namespace w4 {

template <typename T>
__device__ __forceinline__ float ep_f32(T x);
template <>
__device__ __forceinline__ float ep_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float ep_f32<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T ep_round(float x);
template <>
__device__ __forceinline__ __half ep_round<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 ep_round<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// Store output element (m, n) (both in range): vf is the fp32 sum (W4A16),
// vi the int32 accumulator (W4A8).
template <int MODE>
__device__ __forceinline__ void store_out(const TcArgs& args, int64_t m, int64_t n, float vf,
                                          int32_t vi) {
  const int64_t o = m * args.N + n;
  if constexpr (MODE == kW4A8F8) {  // fp32 sum of the exact E4M3 x int4 products
    float r = vf * args.s_tok[m] * args.s_ch[n];
    if (args.bias) r += ep_f32(static_cast<const __half*>(args.bias)[n]);
    static_cast<__half*>(args.out)[o] = __float2half_rn(r);
  } else if constexpr (MODE == kW4A8) {
    if (args.out_s32) {
      static_cast<int32_t*>(args.out)[o] = vi;
      return;
    }
    float r = static_cast<float>(vi) * args.s_tok[m] * args.s_ch[n];
    if (args.bias) r += ep_f32(static_cast<const __half*>(args.bias)[n]);
    static_cast<__half*>(args.out)[o] = __float2half_rn(r);
  } else {
    using T16 = typename std::conditional<MODE == kW4A16_F16, __half, __nv_bfloat16>::type;
    if (args.bias) vf += ep_f32(static_cast<const T16*>(args.bias)[n]);
    static_cast<T16*>(args.out)[o] = ep_round<T16>(vf);
  }
}

// ---------------------------------------------------------------------------
// A product with an epilogue of its own (EpArgs).  v is the fp32 value above
// before its rounding (sum, scales, bias):
//
//   plain: out[m][n] = round(act(v[m][n]) + residual[m][n])
//   gated: out[m][j] = round(act(v[m][2j]) * v[m][2j+1] + residual[m][j])
//
// everything in fp32 with one rounding at the end; the steps around act are
// explicitly rounded, so that every schedule takes the same sums to the same
// bits.  The residual is read
// (from L2: another grid may just have written it) by the thread that
// writes the same element of out, so the two may be one array.

// v of element (m, n), in range
template <int MODE>
__device__ __forceinline__ float ep_value(const EpArgs& args, int64_t m, int64_t n, float vf,
                                          int32_t vi) {
  if constexpr (MODE == kW4A8 || MODE == kW4A8F8) {
    float r = __fmul_rn(__fmul_rn(MODE == kW4A8F8 ? vf : static_cast<float>(vi), args.s_tok[m]),
                        args.s_ch[n]);
    if (args.bias) r = __fadd_rn(r, ep_f32(static_cast<const __half*>(args.bias)[n]));
    return r;
  } else {
    using T16 = typename std::conditional<MODE == kW4A16_F16, __half, __nv_bfloat16>::type;
    if (args.bias) vf = __fadd_rn(vf, ep_f32(static_cast<const T16*>(args.bias)[n]));
    return vf;
  }
}

// GELU, v * (1 + erf(v / sqrt 2)) / 2 = max(v, 0) - q with
//   q = |v| erfc(|v| / sqrt 2) / 2 = |v| t P(t) e^(-v^2 / 2),
//   t = 1 / (1 + |v| / (2 sqrt 2)),
// so that the tail keeps its relative accuracy.  P is a polynomial of degree 8
// fitted by linear programming on 5500 points to erfc(z) e^(z^2) / (2 t) over
// z = |v| / sqrt 2 in [0, 14]; with its coefficients rounded to fp32 it has
// relative error 1.81 * 2^-24 there.  The whole is within (2 v^2 + 12) 2^-24 of
// GELU.  (E4M3 1024 x 8192 x 21760 with bias 155 us; 162 with erfcf.)
__device__ __forceinline__ float ep_gelu(float v) {
  const float a = fabsf(v);
  const float t = __fdividef(1.f, fmaf(0.35355339f, a, 1.f));
  float p = -0.0301823653f;
  p = fmaf(p, t, 0.145287484f);
  p = fmaf(p, t, -0.249470085f);
  p = fmaf(p, t, 0.145345181f);
  p = fmaf(p, t, -0.0173700731f);
  p = fmaf(p, t, 0.102930456f);
  p = fmaf(p, t, 0.121185437f);
  p = fmaf(p, t, 0.141233012f);
  p = fmaf(p, t, 0.141040921f);
  float e;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(v * v * -0.72134752f));
  const float q = a * t * p * e;
  return fmaxf(v, 0.f) - (a >= 100.f ? 0.f : q);  // (infinities: q is 0; NaN stays)
}

// act(v).  The logistic and the tanh go through one exponential; each is
// exact to a few units of fp32, far below the output's 11 or 8 bits.  (The
// fast division gives 0 for a quotient by more than 2^126: SiLU and the tanh
// form reach 0 at -87, where they are below 1e-36.)
__device__ __forceinline__ float ep_act(float v, int act) {
  switch (act) {
    case kActRelu: return v > 0.f ? v : (v != v ? v : 0.f);
    case kActSilu: return __fdividef(v, 1.f + __expf(-v));
    case kActGelu: return ep_gelu(v);
    case kActGeluTanh: {  // (1 + tanh(u)) / 2 = 1 / (1 + e^-2u)
      const float u2 = 1.5957691f * fmaf(0.044715f * v * v, v, v);
      return __fdividef(v, 1.f + __expf(-u2));
    }
    default: return v;
  }
}

// act of each of n values: one branch for all of them
template <int N>
__device__ __forceinline__ void ep_act_n(float (&v)[N], int act) {
  switch (act) {
#define W4_ACT_CASE(A)                              \
  case A:                                           \
    _Pragma("unroll") for (int i = 0; i < N; ++i) { \
      v[i] = ep_act(v[i], A);                       \
    }                                               \
    break;
    W4_ACT_CASE(kActRelu)
    W4_ACT_CASE(kActSilu)
    W4_ACT_CASE(kActGelu)
    W4_ACT_CASE(kActGeluTanh)
#undef W4_ACT_CASE
    default: break;
  }
}

// output element o = m * columns + column from its value before the residual
template <int MODE>
__device__ __forceinline__ float ep_residual(const EpArgs& args, int64_t o) {
  using T16 = typename std::conditional<MODE == kW4A16_BF16, __nv_bfloat16, __half>::type;
  if (!args.residual) return 0.f;
  const unsigned short b = __ldcg(static_cast<const unsigned short*>(args.residual) + o);
  return ep_f32(*reinterpret_cast<const T16*>(&b));
}
template <int MODE>
__device__ __forceinline__ void ep_store(const EpArgs& args, int64_t o, float r) {
  using T16 = typename std::conditional<MODE == kW4A16_BF16, __nv_bfloat16, __half>::type;
  static_cast<T16*>(args.out)[o] = ep_round<T16>(r);
}

// Where column n of row m goes: its element of out (gated: its pair's)
__device__ __forceinline__ int64_t ep_offset(const EpArgs& args, int64_t m, int64_t n) {
  return args.gated ? m * (args.N >> 1) + (n >> 1) : m * args.N + n;
}
// The residual that element (m, n) takes, to be asked for before the sums
// are ready; nothing for a product without an epilogue of its own.  A grid
// that may run beside the one that wrote the residual waits for it first
// (ep_wait, by every thread that reads it).
template <int MODE>
__device__ __forceinline__ float ep_side(const TcArgs&, int64_t, int64_t, bool) { return 0.f; }
template <int MODE>
__device__ __forceinline__ float ep_side(const EpArgs& args, int64_t m, int64_t n, bool ok) {
  return ok ? ep_residual<MODE>(args, ep_offset(args, m, n)) : 0.f;
}
__device__ __forceinline__ void ep_wait(const TcArgs&) {}
__device__ __forceinline__ void ep_wait(const EpArgs&) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The output step of one element per lane, for both kinds of arguments: `ok`
// says whether (m, n) is in range, `side` is ep_side of it.  Lanes whose
// indexes differ in bit XOR hold the columns n and n ^ 1 of the same row, and
// all lanes of `mask` call it together.
template <int MODE, int XOR>
__device__ __forceinline__ void store_lane(const TcArgs& args, int64_t m, int64_t n, bool ok,
                                           float vf, int32_t vi, float, unsigned) {
  if (ok) store_out<MODE>(args, m, n, vf, vi);
}
template <int MODE, int XOR>
__device__ __forceinline__ void store_lane(const EpArgs& args, int64_t m, int64_t n, bool ok,
                                           float vf, int32_t vi, float side, unsigned mask) {
  float v = ok ? ep_value<MODE>(args, m, n, vf, vi) : 0.f;
  bool mine = ok;
  if (args.gated) {
    const float up = __shfl_xor_sync(mask, v, XOR);
    mine = ok && !(n & 1);
    if (mine) v = __fmul_rn(ep_act(v, args.act), up);
  } else {
    v = ep_act(v, args.act);
  }
  if (mine) ep_store<MODE>(args, ep_offset(args, m, n), __fadd_rn(v, side));
}

// ------------------------------------------- eight rows by 32 columns a warp
// The tensor-core schedules hand a warp eight rows of 32 columns, a column a
// lane.  Here the block is transposed by shuffles, so that lane l has row
// l % 8 and the eight columns from 8 * (l / 8): the residual is one 16-byte
// load and out one 16-byte store a lane (8 bytes each when gated, whose pairs
// then lie in one lane), where a column a lane takes eight 2-byte ones (E4M3
// 1024 x 8192 x 21760 with a residual: 207 us with those, 155 with these; 143
// without an epilogue).  The arrays are 16-byte aligned, N is a multiple of 8.

// The residual of a lane's eight columns (gated: of its four pairs)
template <int MODE>
__device__ __forceinline__ uint4 ep_side8(const EpArgs& args, int64_t m0, int64_t n0) {
  const int lane = threadIdx.x & 31;
  const int64_t m = m0 + (lane & 7), n = n0 + (lane >> 3) * 8;
  uint4 r = make_uint4(0u, 0u, 0u, 0u);
  if (!args.residual || m >= args.M || n >= args.N) return r;
  const unsigned short* p =
      static_cast<const unsigned short*>(args.residual) + ep_offset(args, m, n);
  if (args.gated) {
    const uint2 h = __ldcg(reinterpret_cast<const uint2*>(p));
    r.x = h.x;
    r.y = h.y;
  } else {
    r = __ldcg(reinterpret_cast<const uint4*>(p));
  }
  return r;
}

template <typename T16>
__device__ __forceinline__ float2 ep_pair(uint32_t w) {
  return make_float2(ep_f32(reinterpret_cast<const T16*>(&w)[0]),
                     ep_f32(reinterpret_cast<const T16*>(&w)[1]));
}
template <typename T16>
__device__ __forceinline__ uint32_t ep_pack(float a, float b) {
  T16 h[2] = {ep_round<T16>(a), ep_round<T16>(b)};
  return *reinterpret_cast<const uint32_t*>(h);
}

// d: the sums (fp32 bits, or int32) of rows m0..m0+7 of column n0 + lane, n0
// a multiple of 32.  side: ep_side8.
template <int MODE>
__device__ __forceinline__ void store_block8(const EpArgs& args, int64_t m0, int64_t n0,
                                             const uint32_t (&d)[8], const uint4& side) {
  using T16 = typename std::conditional<MODE == kW4A16_BF16, __nv_bfloat16, __half>::type;
  const int lane = threadIdx.x & 31;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = MODE == kW4A8 ? static_cast<float>(static_cast<int32_t>(d[i])) : __uint_as_float(d[i]);
#pragma unroll
  for (int s = 1; s < 8; s *= 2) {
    const bool up = lane & s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i & s) continue;
      const float got = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i | s], s);
      if (up) v[i] = got;
      else v[i | s] = got;
    }
  }
  const int64_t m = m0 + (lane & 7), n = n0 + (lane >> 3) * 8;
  if (m >= args.M || n >= args.N) return;
  if constexpr (MODE == kW4A8 || MODE == kW4A8F8) {
    const float st = args.s_tok[m];
    const float4 a = *reinterpret_cast<const float4*>(args.s_ch + n);
    const float4 b = *reinterpret_cast<const float4*>(args.s_ch + n + 4);
    const float sc[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(__fmul_rn(v[e], st), sc[e]);
  }
  if (args.bias) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const T16*>(args.bias) + n);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = ep_pair<T16>(u[i]);
      v[2 * i] = __fadd_rn(v[2 * i], p.x);
      v[2 * i + 1] = __fadd_rn(v[2 * i + 1], p.y);
    }
  }
  const uint32_t r[4] = {side.x, side.y, side.z, side.w};
  uint32_t o[4];
  if (args.gated) {
    float g[4] = {v[0], v[2], v[4], v[6]};
    ep_act_n(g, args.act);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 p = ep_pair<T16>(r[i]);
      o[i] = ep_pack<T16>(__fadd_rn(__fmul_rn(g[2 * i], v[4 * i + 1]), p.x),
                          __fadd_rn(__fmul_rn(g[2 * i + 1], v[4 * i + 3]), p.y));
    }
    o[2] = o[3] = 0u;
  } else {
    ep_act_n(v, args.act);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = ep_pair<T16>(r[i]);
      o[i] = ep_pack<T16>(__fadd_rn(v[2 * i], p.x), __fadd_rn(v[2 * i + 1], p.y));
    }
  }
  T16* const out = static_cast<T16*>(args.out) + ep_offset(args, m, n);
  if (args.gated) *reinterpret_cast<uint2*>(out) = make_uint2(o[0], o[1]);
  else *reinterpret_cast<uint4*>(out) = make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace w4
