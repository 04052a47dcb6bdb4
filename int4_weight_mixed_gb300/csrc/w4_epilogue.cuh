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
// everything in fp32 with one rounding at the end.  The residual is read
// (from L2: another grid may just have written it) by the thread that
// writes the same element of out, so the two may be one array.

// v of element (m, n), in range
template <int MODE>
__device__ __forceinline__ float ep_value(const EpArgs& args, int64_t m, int64_t n, float vf,
                                          int32_t vi) {
  if constexpr (MODE == kW4A8 || MODE == kW4A8F8) {
    float r = (MODE == kW4A8F8 ? vf : static_cast<float>(vi)) * args.s_tok[m] * args.s_ch[n];
    if (args.bias) r += ep_f32(static_cast<const __half*>(args.bias)[n]);
    return r;
  } else {
    using T16 = typename std::conditional<MODE == kW4A16_F16, __half, __nv_bfloat16>::type;
    if (args.bias) vf += ep_f32(static_cast<const T16*>(args.bias)[n]);
    return vf;
  }
}

// act(v).  The logistic and the tanh go through one exponential; each is
// exact to a few units of fp32, far below the output's 11 or 8 bits.
__device__ __forceinline__ float ep_act(float v, int act) {
  switch (act) {
    case kActRelu: return v > 0.f ? v : (v != v ? v : 0.f);
    case kActSilu: return v / (1.f + __expf(-v));
    case kActGelu: return 0.5f * v * erfcf(v * -0.70710678f);  // exact in the tail too
    case kActGeluTanh: {  // (1 + tanh(u)) / 2 = 1 / (1 + e^-2u)
      const float u2 = 1.5957691f * fmaf(0.044715f * v * v, v, v);
      return v / (1.f + __expf(-u2));
    }
    default: return v;
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

// The output step of one element per lane, for both kinds of arguments: `ok`
// says whether (m, n) is in range.  Lanes whose indexes differ in bit XOR
// hold the columns n and n ^ 1 of the same row, and all lanes of `mask` call
// it together.
template <int MODE, int XOR>
__device__ __forceinline__ void store_lane(const TcArgs& args, int64_t m, int64_t n, bool ok,
                                           float vf, int32_t vi, unsigned) {
  if (ok) store_out<MODE>(args, m, n, vf, vi);
}
template <int MODE, int XOR>
__device__ __forceinline__ void store_lane(const EpArgs& args, int64_t m, int64_t n, bool ok,
                                           float vf, int32_t vi, unsigned mask) {
  const float v = ok ? ep_value<MODE>(args, m, n, vf, vi) : 0.f;
  if (args.gated) {
    const float up = __shfl_xor_sync(mask, v, XOR);
    if (ok && !(n & 1)) {
      const int64_t o = m * (args.N >> 1) + (n >> 1);
      ep_store<MODE>(args, o, ep_act(v, args.act) * up + ep_residual<MODE>(args, o));
    }
  } else if (ok) {
    const int64_t o = m * args.N + n;
    ep_store<MODE>(args, o, ep_act(v, args.act) + ep_residual<MODE>(args, o));
  }
}

// The output step of eight rows m0..m0+7 of column n, one column per lane of
// a full warp (the lanes cover 32 columns from a multiple of 32): d holds the
// sums (fp32 bits, or int32).  Gated: even lanes take the first four rows of
// their pair of columns, odd lanes the last four, so all lanes work and each
// stored row covers 32 contiguous bytes.
template <int MODE>
__device__ __forceinline__ void store_block8(const EpArgs& args, int64_t m0, int64_t n,
                                             const uint32_t (&d)[8]) {
  const bool col = n < args.N;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = col && m0 + i < args.M ? ep_value<MODE>(args, m0 + i, n, __uint_as_float(d[i]),
                                                   static_cast<int32_t>(d[i]))
                                  : 0.f;
  if (args.gated) {
    const bool odd = n & 1;
    const int64_t cols = args.N >> 1, mh = m0 + (odd ? 4 : 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[4 + i], 1);
      const float gate = odd ? other : v[i], up = odd ? v[4 + i] : other;
      if (!col || mh + i >= args.M) continue;
      const int64_t o = (mh + i) * cols + (n >> 1);
      ep_store<MODE>(args, o, ep_act(gate, args.act) * up + ep_residual<MODE>(args, o));
    }
  } else {
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      r[i] = col && m0 + i < args.M ? ep_residual<MODE>(args, (m0 + i) * args.N + n) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col && m0 + i < args.M)
        ep_store<MODE>(args, (m0 + i) * args.N + n, ep_act(v[i], args.act) + r[i]);
  }
}

}  // namespace w4
