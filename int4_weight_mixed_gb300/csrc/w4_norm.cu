// w4_norm.cu — root-mean-square norm of the rows that feed a product, with
// the residual stream's addition before it and a 16-bit or an 8-bit output
// (vLLM PR #6547 "Enable Dynamic Per Token fp8" prefers one scale per token
// because it fuses with the normalisation before it).  For every row of
// x [M,K], with residual r, weight w and t = 127 (int8) or 448 (E4M3):
//
//   h     = x + r                         (r optional)
//   rstd  = 1 / sqrt(sum(h^2) / K + eps)
//   16-bit: y = h * rstd * w
//   8-bit : y is held as codes times one scale per row, the scale taking the
//           row's largest |y| to t.  rstd divides out of y / scale:
//             A     = max |h * w|
//             code  = round(h * w * (t * (1 / A))),   scale = rstd * A / t
//           so the codes need no statistic but A, and a row is read for
//           both reductions at once.
//
// Every value is held in 32 bits: h is not rounded before the norm (only
// where it is stored), and y goes to its output in one rounding.  Each step
// of the 8-bit path is one explicitly rounded operation, so a code depends
// on its own row's values alone, whichever kernel computes it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "w4_epilogue.cuh"
#include "w4_internal.h"

namespace w4 {
namespace {

constexpr int kNormThreads = 256;

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int OUT>
__device__ __forceinline__ float norm_top() {
  return OUT == kNormE4M3 ? 448.f : 127.f;
}

// What a row's codes are made with.  A row that holds an infinity or a NaN,
// or whose sum of squares passes the fp32 range, gets scale NaN and codes 0;
// a row of zeros scale 0 and codes 0.
struct RowCode {
  float inv;    // t * (1 / (A * up)); 0 for a row without codes
  float up;     // 1, or a power of two that keeps t / A finite for tiny A
  float scale;  // the row's scale
};
template <int OUT>
__device__ __forceinline__ RowCode row_code(float sum, float A, float rstd) {
  constexpr float kInf = __builtin_huge_valf();
  RowCode c;
  c.up = A < 0x1p-100f ? 0x1p100f : 1.f;
  c.inv = A > 0.f && A < kInf && sum < kInf ? __fmul_rn(norm_top<OUT>(), __frcp_rn(A * c.up)) : 0.f;
  c.scale = A < kInf && sum < kInf ? __fdiv_rn(__fmul_rn(rstd, A), norm_top<OUT>())
                                   : __int_as_float(0x7fc00000);
  if (A == 0.f && sum < kInf) c.scale = 0.f;
  return c;
}

// the byte of one code (hw = h * w)
template <int OUT>
__device__ __forceinline__ uint32_t code_of(float hw, const RowCode& c) {
  if (c.inv == 0.f) return 0u;
  const float q = __fmul_rn(c.up == 1.f ? hw : __fmul_rn(hw, c.up), c.inv);
  if constexpr (OUT == kNormE4M3) {
    uint16_t e2;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e2) : "f"(0.f), "f"(q));
    return e2 & 0xFFu;
  } else {
    return static_cast<uint32_t>(__float2int_rn(q)) & 0xFFu;
  }
}

// One CTA per row, element by element: any K and alignment.  The row is read
// for the two reductions and again for the outputs; h and y are written only
// then, by the thread that has read the element, so they may take the place
// of x or r.
template <typename T, int OUT>
__global__ void __launch_bounds__(kNormThreads)
    norm_row_kernel(const T* x, const T* r, const T* w, int64_t K, float eps, T* h_out, void* y,
                    float* scales) {
  __shared__ float red[2][kNormThreads / 32];
  const int64_t m = blockIdx.x;
  const T* xr = x + m * K;
  const T* rr = r ? r + m * K : nullptr;
  auto h_at = [&](int64_t k) {
    const float v = ep_f32(xr[k]);
    return rr ? __fadd_rn(v, ep_f32(rr[k])) : v;
  };
  auto w_at = [&](int64_t k) { return w ? ep_f32(w[k]) : 1.f; };
  float sum = 0.f, A = 0.f;
  for (int64_t k = threadIdx.x; k < K; k += kNormThreads) {
    const float h = h_at(k);
    sum = fmaf(h, h, sum);
    if (OUT != kNorm16) A = max_nan(A, fabsf(__fmul_rn(h, w_at(k))));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (OUT != kNorm16) A = max_nan(A, __shfl_xor_sync(0xffffffffu, A, o));
  }
  if ((threadIdx.x & 31) == 0) {
    red[0][threadIdx.x >> 5] = sum;
    red[1][threadIdx.x >> 5] = A;
  }
  __syncthreads();
  sum = red[0][0];
  A = red[1][0];
#pragma unroll
  for (int i = 1; i < kNormThreads / 32; ++i) {
    sum += red[0][i];
    A = max_nan(A, red[1][i]);
  }
  const float rstd = rsqrtf(__fdiv_rn(sum, static_cast<float>(K)) + eps);
  RowCode c{};
  if (OUT != kNorm16) {
    c = row_code<OUT>(sum, A, rstd);
    if (threadIdx.x == 0) scales[m] = K == 0 ? 0.f : c.scale;
  }
  for (int64_t k = threadIdx.x; k < K; k += kNormThreads) {
    const float h = h_at(k);
    if (h_out) h_out[m * K + k] = ep_round<T>(h);
    if constexpr (OUT == kNorm16)
      static_cast<T*>(y)[m * K + k] = ep_round<T>(__fmul_rn(__fmul_rn(h, rstd), w_at(k)));
    else
      static_cast<uint8_t*>(y)[m * K + k] =
          static_cast<uint8_t>(code_of<OUT>(__fmul_rn(h, w_at(k)), c));
  }
}

template <typename T, int OUT>
cudaError_t launch_norm_t(const NormArgs& a, cudaStream_t s) {
  norm_row_kernel<T, OUT><<<static_cast<unsigned>(a.M), kNormThreads, 0, s>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.residual),
      static_cast<const T*>(a.weight), a.K, a.eps, static_cast<T*>(a.h_out), a.y, a.scales);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_norm_out(const NormArgs& a, cudaStream_t s) {
  switch (a.out) {
    case kNorm16: return launch_norm_t<T, kNorm16>(a, s);
    case kNormS8: return launch_norm_t<T, kNormS8>(a, s);
    default: return launch_norm_t<T, kNormE4M3>(a, s);
  }
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
  if (a.M == 0 || (a.K == 0 && a.out == kNorm16)) return cudaSuccess;
  return a.bf16 ? launch_norm_out<__nv_bfloat16>(a, s) : launch_norm_out<__half>(a, s);
}

}  // namespace w4
