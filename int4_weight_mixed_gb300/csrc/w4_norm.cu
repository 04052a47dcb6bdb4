// w4_norm.cu — root-mean-square norm of the rows that feed a product, with
// the residual stream's addition before it and a 16-bit or an 8-bit output
// (vLLM PR #6547 "Enable Dynamic Per Token fp8" prefers one scale per token
// because it fuses with the normalisation before it).  For every row of
// x [M,K], with residual r, weight w and t = 127 (int8) or 448 (E4M3):
//
//   h     = x + r                         (r optional)
//   rstd  = 1 / sqrt(sum(h^2) / K + eps)
//   16-bit: y = (h * w) * rstd
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
#include "w4_ptx.cuh"

namespace w4 {
namespace {

constexpr int kNormThreads = 256;      // a CTA of short rows
constexpr int kNormMaxThreads = 1024;  // a CTA of one long row
constexpr int kNormMaxCluster = 8;
constexpr size_t kNormMaxSmem = 224 * 1024;

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ void cp_async16(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// waits for all but the newest N groups
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
// hw = h * w as the codes take it: itself but for the rare rows above
__device__ __forceinline__ bool plain_codes(const RowCode& c) { return c.inv != 0.f && c.up == 1.f; }
__device__ __forceinline__ float fit_code(float hw, const RowCode& c) {
  return c.inv == 0.f ? 0.f : __fmul_rn(hw, c.up);
}

// The low byte is the code of a fitted hw.  int8: adding 1.5 * 2^23 rounds
// to the nearest integer, ties to even, and leaves it in the low mantissa
// bits (|q| <= 127 (1 + 2^-22)).
template <int OUT>
__device__ __forceinline__ uint32_t code_of(float hw, float inv) {
  const float q = __fmul_rn(hw, inv);
  if constexpr (OUT == kNormE4M3) {
    uint16_t e2;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e2) : "f"(0.f), "f"(q));
    return e2;
  } else {
    return __float_as_uint(__fadd_rn(q, 12582912.f));
  }
}
template <int OUT>
__device__ __forceinline__ uint32_t code4_of(const float* hw, float inv) {
  if constexpr (OUT == kNormE4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(lo) : "f"(__fmul_rn(hw[1], inv)), "f"(__fmul_rn(hw[0], inv)));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
        : "=h"(hi) : "f"(__fmul_rn(hw[3], inv)), "f"(__fmul_rn(hw[2], inv)));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  } else {
    const uint32_t lo = __byte_perm(code_of<OUT>(hw[0], inv), code_of<OUT>(hw[1], inv), 0x0040);
    const uint32_t hi = __byte_perm(code_of<OUT>(hw[2], inv), code_of<OUT>(hw[3], inv), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
  }
}

// Eight 16-bit values of a 16-byte load, or one value.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, __half>::value) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    } else {  // a bf16 is the upper half of its fp32
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (std::is_same<T, __half>::value) {
    const __half2 p = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
  } else {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
  }
}

// The rows' reductions: sum and A of each row's blockDim.x threads (a power
// of two up to 32, or a multiple of 32), in an order that depends on
// blockDim.x alone, which every launch takes from K: the bits of a row do not
// depend on how many rows there are.  red: [2][kNormMaxThreads / 32].
template <int OUT>
__device__ __forceinline__ void reduce_row(float& sum, float& A, float (*red)[kNormMaxThreads / 32]) {
  const int tpr = blockDim.x;
  for (int o = (tpr < 32 ? tpr : 32) / 2; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (OUT != kNorm16) A = max_nan(A, __shfl_xor_sync(0xffffffffu, A, o));
  }
  if (tpr <= 32) return;
  const int nw = tpr / 32, w0 = threadIdx.y * nw;
  if ((threadIdx.x & 31) == 0) {
    red[0][w0 + threadIdx.x / 32] = sum;
    red[1][w0 + threadIdx.x / 32] = A;
  }
  __syncthreads();
  sum = red[0][w0];
  A = red[1][w0];
  for (int i = 1; i < nw; ++i) {
    sum += red[0][w0 + i];
    if (OUT != kNorm16) A = max_nan(A, red[1][w0 + i]);
  }
}

// The same for the kernels that take any K, the warps' sums added by shuffles
// (at most P warps a row, a power of two; a longer butterfly over zeros adds
// the same numbers).
template <int OUT, int P>
__device__ __forceinline__ void reduce_any_row(float& sum, float& A,
                                               float (*red)[kNormMaxThreads / 32]) {
  const int tpr = blockDim.x;
  auto add = [&](int o) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (OUT != kNorm16) A = max_nan(A, __shfl_xor_sync(0xffffffffu, A, o));
  };
  if (tpr < 32) {
    for (int o = tpr / 2; o > 0; o >>= 1) add(o);
    return;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) add(o);
  if (tpr == 32) return;
  const int nw = tpr / 32, w0 = threadIdx.y * nw, lane = threadIdx.x & 31;
  if (lane == 0) {
    red[0][w0 + threadIdx.x / 32] = sum;
    if (OUT != kNorm16) red[1][w0 + threadIdx.x / 32] = A;
  }
  __syncthreads();
  const int i = lane & (P - 1);
  sum = i < nw ? red[0][w0 + i] : 0.f;
  if (OUT != kNorm16) A = i < nw ? red[1][w0 + i] : 0.f;
#pragma unroll
  for (int o = P / 2; o > 0; o >>= 1) add(o);
}

// The same over the CTAs of a row's cluster: every CTA writes its sums into
// each CTA's array, and adds them in the order of the ranks.
template <int OUT>
__device__ __forceinline__ void reduce_cluster(float& sum, float& A) {
  __shared__ float part[kNormMaxCluster][2];
  const uint32_t C = cluster_size(), me = cluster_rank();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA runs
  if (threadIdx.x < C) {
    const uint32_t to = peer_addr(smem_addr(&part[me][0]), threadIdx.x);
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(sum), "f"(A) : "memory");
  }
  cluster_sync_all();  // no CTA touches another's memory after this
  sum = part[0][0];
  A = part[0][1];
  for (uint32_t i = 1; i < C; ++i) {
    sum += part[i][0];
    if (OUT != kNorm16) A = max_nan(A, part[i][1]);
  }
}

// h of eight elements from 16 bytes of x and of r
template <typename T>
__device__ __forceinline__ void add8(const uint4& xv, const uint4& rv, bool has_r, float (&h)[8]) {
  unpack<T>(xv, h);
  if (has_r) {
    float g[8];
    unpack<T>(rv, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = __fadd_rn(h[e], g[e]);
  }
}
// the outputs of eight elements from hw = h * w
template <typename T, int OUT>
__device__ __forceinline__ void store8(const float* hw, float rstd, float inv, void* y,
                                       int64_t row, int i) {
  if constexpr (OUT == kNorm16) {
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = pack2<T>(__fmul_rn(hw[2 * e], rstd), __fmul_rn(hw[2 * e + 1], rstd));
    reinterpret_cast<uint4*>(static_cast<T*>(y) + row)[i] = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    reinterpret_cast<uint2*>(static_cast<uint8_t*>(y) + row)[i] =
        make_uint2(code4_of<OUT>(hw, inv), code4_of<OUT>(hw + 4, inv));
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&h)[8]) {
  return make_uint4(pack2<T>(h[0], h[1]), pack2<T>(h[2], h[3]), pack2<T>(h[4], h[5]),
                    pack2<T>(h[6], h[7]));
}

// Aligned rows, held in registers: each of a row's threads reads NV vectors
// of 16 bytes, all loads issued before the first is used, so x and r are read
// once.  h is stored as soon as it is formed, y once the row's statistics are
// known; every element is read and written by one thread, so an output may
// take the place of x or r.  64 registers a thread leave 1024 threads and up
// to 128 KB of loads in flight on an SM.  Bound by HBM, with a residual 4
// bytes read and 3 or 4 written per element: 16384 x 8192 fp16 to int8 133 us
// (104% of the copy bandwidth), 16384 x 4096 bf16 77 us (103%).
// CLUSTER: a row of more than 8192 values is split over the CTAs of a
// cluster, which exchange their sums through distributed shared memory: 4096 x
// 28672 to int8 139 us (87%), 1024 x 21760 to E4M3 30 us (77%, two and a half
// waves).  One CTA of the whole row took 147 and 35.5 us in registers (one CTA
// an SM at 64 registers x 704 threads), 147 and 36 staged in shared memory.
template <typename T, int OUT, int NV, bool CLUSTER>
__global__ void __launch_bounds__(kNormThreads, 4)
    norm_held_kernel(const T* x, const T* r, const T* __restrict__ w, int64_t M, int K, float eps,
                     T* h_out, void* y, float* scales) {
  __shared__ float red[2][kNormMaxThreads / 32];
  // launched while the kernel before may still run: wait for it, then let
  // the next one do the same
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int tpr = blockDim.x;
  const int64_t m = CLUSTER ? blockIdx.x / cluster_size()
                            : static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool live = CLUSTER || m < M;
  if constexpr (CLUSTER)  // this CTA runs: the others may write its shared memory
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  // this CTA's vectors of the row: i0 .. i0 + n - 1
  const int i0 = CLUSTER ? static_cast<int>(cluster_rank()) * NV * tpr : 0;
  const int n = CLUSTER ? min(K / 8 - i0, NV * tpr) : K / 8;
  const int64_t row = (live ? m : 0) * K + i0 * 8;
  if (CLUSTER && w) w += i0 * 8;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 xv[NV], rv[NV], wv[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = threadIdx.x + v * tpr;
    const bool in = live && i < n;
    xv[v] = in ? reinterpret_cast<const uint4*>(x + row)[i] : zero;
    rv[v] = in && r ? reinterpret_cast<const uint4*>(r + row)[i] : zero;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = threadIdx.x + v * tpr;
    wv[v] = w && i < n ? __ldg(reinterpret_cast<const uint4*>(w) + i) : zero;
  }
  float hw[NV * 8];
  float sum = 0.f, A = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = threadIdx.x + v * tpr;
    float h[8], u[8];
    add8<T>(xv[v], rv[v], r != nullptr, h);
    if (h_out && live && i < n) reinterpret_cast<uint4*>(h_out + row)[i] = pack8<T>(h);
    if (w) unpack<T>(wv[v], u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sum = fmaf(h[e], h[e], sum);
      hw[v * 8 + e] = w ? __fmul_rn(h[e], u[e]) : h[e];
      if (OUT != kNorm16) A = max_nan(A, fabsf(hw[v * 8 + e]));
    }
  }
  reduce_row<OUT>(sum, A, red);
  if constexpr (CLUSTER) reduce_cluster<OUT>(sum, A);
  if (!live) return;
  const float rstd = rsqrtf(__fdiv_rn(sum, static_cast<float>(K)) + eps);
  RowCode c{};
  if (OUT != kNorm16) {
    c = row_code<OUT>(sum, A, rstd);
    if (i0 == 0 && threadIdx.x == 0) scales[m] = c.scale;
    if (!plain_codes(c)) {
#pragma unroll
      for (int e = 0; e < NV * 8; ++e) hw[e] = fit_code(hw[e], c);
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = threadIdx.x + v * tpr;
    if (i < n) store8<T, OUT>(hw + v * 8, rstd, c.inv, y, row, i);
  }
}

// 16 bytes from byte n (0..15) of two neighbouring 16-byte pieces.
__device__ __forceinline__ uint4 bytes_from(const uint4& lo, const uint4& hi, uint32_t n) {
  const bool two = n & 8, one = n & 4;
  const uint32_t a0 = two ? lo.z : lo.x, a1 = two ? lo.w : lo.y, a2 = two ? hi.x : lo.z,
                 a3 = two ? hi.y : lo.w, a4 = two ? hi.z : hi.x, a5 = two ? hi.w : hi.y;
  const uint32_t b0 = one ? a1 : a0, b1 = one ? a2 : a1, b2 = one ? a3 : a2, b3 = one ? a4 : a3,
                 b4 = one ? a5 : a4;
  const uint32_t bits = (n & 3) * 8;
  return make_uint4(__funnelshift_r(b0, b1, bits), __funnelshift_r(b1, b2, bits),
                    __funnelshift_r(b2, b3, bits), __funnelshift_r(b3, b4, bits));
}

// `count` elements from shared memory (16-byte aligned) to any place of an
// array, by the `n` threads of a row: whole 16-byte pieces of the array, and
// what is left at the two ends by element.  Shared memory is read up to 16
// bytes past the elements.  At most NV * n pieces.
template <int NV, typename E>
__device__ __forceinline__ void copy_out(const uint4* from, E* to, int count, int t, int n) {
  constexpr int kPer = 16 / sizeof(E);
  const int head =
      min(static_cast<int>((0 - reinterpret_cast<uintptr_t>(to)) & 15) / static_cast<int>(sizeof(E)), count);
  const int pieces = (count - head) / kPer, tail = head + pieces * kPer;
  uint4* const to16 = reinterpret_cast<uint4*>(to + head);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int p = t + v * n;
    if (p < pieces) to16[p] = bytes_from(from[p], from[p + 1], head * sizeof(E));
  }
  const E* const src = reinterpret_cast<const E*>(from);
#pragma unroll 1
  for (int e = t; e < head; e += n) to[e] = src[e];
#pragma unroll 1
  for (int e = tail + t; e < count; e += n) to[e] = src[e];
}

// Any K from 9 to MAXT * NV * 8.  A block of blockDim.y rows is a contiguous
// range of x and of r, copied to shared memory in 16-byte pieces whatever the
// rows' own alignment (x and r start at 16-byte boundaries; what is left at
// the arrays' end by element).  A CTA takes every gridDim.x-th block and copies
// the next one while it works on this one.  A thread holds NV vectors of eight
// columns, each put together from the two pieces that it lies in; the outputs
// go back through the stage their inputs came from, so that they too leave in
// 16-byte pieces.  A piece that two blocks' rows share is read by both, each
// using its own values, and written by element.
// Bound by instruction issue and by the barriers between its steps: 10782 x
// 6165 bf16 with a residual to E4M3 101 us (68% of the copy bandwidth), 16384 x
// 8191 fp16 without one 98 (80%), 32768 x 2001 bf16 with one 94 (82%).  Four
// vectors a thread beyond 4096 columns: with two, whose rows take more threads,
// the first two were 117 and 123 us.  Two CTAs of four vectors an SM with a
// residual, three without: three spill with one (115 us), two were 105 without.  Element by element from the same stages
// they were 143 and 160.  Beyond 16384 columns the registers of a CTA of more
// than 512 threads do not hold four vectors without spilling: 4096 x 20001 fp16
// to int8 161 us (52%); with eight vectors a thread 165.
template <typename T, int OUT, bool RES, int NV, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT > kNormThreads ? 1 : NV == 2 ? 4 : RES ? 2 : 3)
    norm_ragged_kernel(const T* x, const T* r, const T* __restrict__ w, int64_t M, int K,
                       float eps, T* h_out, void* y, float* scales, uint32_t range) {
  extern __shared__ __align__(16) uint8_t raw[];  // [2][x range, r range]
  __shared__ float red[2][kNormMaxThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int R = blockDim.y, tpr = blockDim.x, n = (K + 7) / 8;
  const int t = threadIdx.y * tpr + threadIdx.x, nt = tpr * R;
  const int64_t blocks = (M + R - 1) / R;
  const uint32_t stage = RES ? 2 * range : range;
  auto copy = [&](int64_t b, uint32_t at) {  // block b to the stage at byte `at`
    const int64_t e0 = b * R * K;  // the block's first element; its last row may be the array's
    const bool last = (b + 1) * R >= M;
    const int len = static_cast<int>(last ? M * K - e0 : static_cast<int64_t>(R) * K);
    const int off = static_cast<int>(e0) & 7;
    const int pieces = last ? (off + len) / 8 : (off + len + 7) / 8;
    const uint32_t sx = smem_addr(raw) + at;
    const T* const px = x + (e0 - off);
    const T* const pr = RES ? r + (e0 - off) : nullptr;
#pragma unroll
    for (int v = 0; v <= NV; ++v) {  // up to R * n + 1 pieces
      const int g = v < NV ? t + v * nt : NV * nt;
      if (g < pieces && (v < NV || t == 0)) {
        cp_async16(sx + g * 16, px + g * 8);
        if (RES) cp_async16(sx + range + g * 16, pr + g * 8);
      }
    }
    if (last) {
      T* const tx = reinterpret_cast<T*>(raw + at);
      T* const tr = reinterpret_cast<T*>(raw + at + range);
#pragma unroll 1
      for (int e = pieces * 8 + t; e < off + len; e += nt) {
        tx[e] = px[e];
        if (RES) tr[e] = pr[e];
      }
    }
  };
  uint32_t at = 0;
  if (blockIdx.x < blocks) copy(blockIdx.x, 0);
  cp_async_commit();
  // This thread's vectors of a row: threadIdx.x + v * tpr.  Only its last one
  // can lie past the row's end (the host gives a row enough vectors for
  // that); it takes the row's last vector instead, with the columns masked.
  const int i_last = threadIdx.x + (NV - 1) * tpr;
  const int left = K - i_last * 8;  // columns from there on
  uint32_t mask[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    mask[j] = left >= 2 * j + 2 ? 0xffffffffu : left == 2 * j + 1 ? 0xffffu : 0u;
  auto vec = [&](int v) { return v < NV - 1 ? static_cast<int>(threadIdx.x) + v * tpr : min(i_last, n - 1); };
  uint4 wv[NV];  // a thread has the same columns in every row
  const bool w16 = (reinterpret_cast<uintptr_t>(w) & 15) == 0;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int k = vec(v) * 8;
    if (w && w16 && k + 8 <= K) {
      wv[v] = __ldg(reinterpret_cast<const uint4*>(w + k));
    } else {
      float u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = w && k + e < K ? ep_f32(w[k + e]) : 1.f;
      wv[v] = pack8<T>(u);
    }
  }
  const float inv_k = __frcp_rn(static_cast<float>(K));
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x, at ^= stage) {
    cp_async_wait<0>();
    __syncthreads();  // everyone's copies of this block; the other stage has been read
    if (b + gridDim.x < blocks) copy(b + gridDim.x, at ^ stage);
    cp_async_commit();
    const int64_t m = b * R + threadIdx.y;
    const bool live = m < M;  // other rows take the block's first one and store nothing
    const int64_t e0 = b * R * K;
    const int first = (static_cast<int>(e0) & 7) + (live ? static_cast<int>(threadIdx.y) * K : 0);
    uint4* const xs = reinterpret_cast<uint4*>(raw + at);
    uint4* const rs = reinterpret_cast<uint4*>(raw + at + range);
    const uint32_t off = (first & 7) * 2;
    float hw[NV * 8];
    uint4 hp[NV];
    float sum = 0.f, A = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int p = (first >> 3) + vec(v);
      auto piece = [&](const uint4* from) {
        uint4 q = bytes_from(from[p], from[p + 1], off);
        if (v == NV - 1) {
          q.x &= mask[0];
          q.y &= mask[1];
          q.z &= mask[2];
          q.w &= mask[3];
        }
        return q;
      };
      float h[8], u[8];
      const uint4 xv = piece(xs);
      add8<T>(xv, RES ? piece(rs) : xv, RES, h);
      unpack<T>(wv[v], u);
      if (RES) hp[v] = pack8<T>(h);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum = fmaf(h[e], h[e], sum);
        hw[v * 8 + e] = __fmul_rn(h[e], u[e]);
        if (OUT != kNorm16) A = max_nan(A, fabsf(hw[v * 8 + e]));
      }
    }
    reduce_any_row<OUT, MAXT / 32>(sum, A, red);
    if (tpr <= 32) __syncthreads();  // the stage has been read, as after a longer row's sums
    const float rstd = rsqrtf(fmaf(sum, inv_k, eps));
    RowCode c{};
    if (OUT != kNorm16) {
      c = row_code<OUT>(sum, A, rstd);
      if (live && threadIdx.x == 0) scales[m] = c.scale;
      if (!plain_codes(c)) {
#pragma unroll
        for (int e = 0; e < NV * 8; ++e) hw[e] = fit_code(hw[e], c);
      }
    }
    uint4* const ys = xs + threadIdx.y * n;
    uint4* const hs = rs + threadIdx.y * n;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (v == NV - 1 && left <= 0) continue;
      store8<T, OUT>(hw + v * 8, rstd, c.inv, ys, 0, vec(v));
      if (RES && h_out) hs[vec(v)] = hp[v];
    }
    __syncthreads();
    if (live) {
      const int64_t row = e0 + static_cast<int64_t>(threadIdx.y) * K;
      if constexpr (OUT == kNorm16)
        copy_out<NV>(ys, static_cast<T*>(y) + row, K, threadIdx.x, tpr);
      else
        copy_out<(NV + 1) / 2>(ys, static_cast<uint8_t*>(y) + row, K, threadIdx.x, tpr);
      if (RES && h_out) copy_out<NV>(hs, h_out + row, K, threadIdx.x, tpr);
    }
  }
}

// Whatever the others do not take (arrays that start off a 16-byte boundary,
// longer rows): both passes read x and r themselves, the second from L2; h
// and y are written in the second, by the thread that has read the element.
// A row is summed in the ragged kernel's order.
template <typename T, int OUT>
__global__ void __launch_bounds__(kNormMaxThreads)
    norm_any_kernel(const T* x, const T* r, const T* __restrict__ w, int64_t M, uint32_t K,
                    float eps, T* h_out, void* y, float* scales) {
  __shared__ float red[2][kNormMaxThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t m = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool live = m < M;
  const uint32_t tpr = blockDim.x;
  const T* const xr = x + m * K;
  const T* const rr = r + (r ? m * K : 0);
  auto h_at = [&](uint32_t k) {
    const float v = ep_f32(xr[k]);
    return r ? __fadd_rn(v, ep_f32(rr[k])) : v;
  };
  auto hw_at = [&](uint32_t k, float h) { return w ? __fmul_rn(h, ep_f32(w[k])) : h; };
  float sum = 0.f, A = 0.f;
  if (live) {
    for (uint32_t k = threadIdx.x * 8; k < K; k += tpr * 8) {
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) {
        const float h = k + e < K ? h_at(k + e) : 0.f;
        sum = fmaf(h, h, sum);
        if (OUT != kNorm16 && k + e < K) A = max_nan(A, fabsf(hw_at(k + e, h)));
      }
    }
  }
  reduce_any_row<OUT, kNormMaxThreads / 32>(sum, A, red);
  if (!live) return;
  const float rstd = rsqrtf(fmaf(sum, __frcp_rn(static_cast<float>(K)), eps));
  RowCode c{};
  if (OUT != kNorm16) {
    c = row_code<OUT>(sum, A, rstd);
    if (threadIdx.x == 0) scales[m] = c.scale;
  }
  auto put = [&](uint32_t k) {
    const float h = h_at(k), hw = hw_at(k, h);
    if (h_out) h_out[m * K + k] = ep_round<T>(h);
    if constexpr (OUT == kNorm16)
      static_cast<T*>(y)[m * K + k] = ep_round<T>(__fmul_rn(hw, rstd));
    else
      static_cast<uint8_t*>(y)[m * K + k] =
          static_cast<uint8_t>(code_of<OUT>(fit_code(hw, c), c.inv));
  };
#pragma unroll 2
  for (uint32_t k = threadIdx.x; k < K; k += tpr) put(k);
}

cudaLaunchConfig_t norm_config(dim3 grid, dim3 block, cudaLaunchAttribute* attr, cudaStream_t s) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// Threads for `per` of a row's n pieces of work each: a power of two within
// a warp, whole warps beyond.
int row_threads(int64_t n, int per) {
  const int64_t t = (n + per - 1) / per;
  int p = 1;
  while (p < 32 && p < t) p *= 2;
  if (t <= 32) return p;
  return static_cast<int>(t < kNormMaxThreads ? (t + 31) / 32 * 32 : kNormMaxThreads);
}
// rows of a CTA: one, or as many short ones as make kNormThreads threads
int cta_rows(int tpr) { return tpr < kNormThreads ? kNormThreads / tpr : 1; }

template <typename T, int OUT, int NV>
cudaError_t launch_held(const NormArgs& a, int tpr, cudaStream_t s) {
  const int rows = cta_rows(tpr);
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg =
      norm_config(dim3(static_cast<unsigned>((a.M + rows - 1) / rows)), dim3(tpr, rows), &attr, s);
  return cudaLaunchKernelEx(&cfg, &norm_held_kernel<T, OUT, NV, false>, static_cast<const T*>(a.x),
                            static_cast<const T*>(a.residual), static_cast<const T*>(a.weight),
                            a.M, static_cast<int>(a.K), a.eps, static_cast<T*>(a.h_out), a.y,
                            a.scales);
}

// A row over the CTAs of a cluster, NV vectors a thread.
template <typename T, int OUT, int NV>
cudaError_t launch_split(const NormArgs& a, int64_t n, cudaStream_t s) {
  const int C = static_cast<int>((n + NV * kNormThreads - 1) / (NV * kNormThreads));
  if (a.M > 0x7fffffff / C) return cudaErrorInvalidValue;  // more CTAs than a grid has
  const int tpr = static_cast<int>((n + NV * C * 32 - 1) / (NV * C * 32)) * 32;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg =
      norm_config(dim3(static_cast<unsigned>(a.M * C)), dim3(tpr), attr, s);
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, &norm_held_kernel<T, OUT, NV, true>, static_cast<const T*>(a.x),
                            static_cast<const T*>(a.residual), static_cast<const T*>(a.weight),
                            a.M, static_cast<int>(a.K), a.eps, static_cast<T*>(a.h_out), a.y,
                            a.scales);
}

// Lets a kernel use `bytes` of dynamic shared memory.
template <class Fn>
cudaError_t allow_smem(Fn* fn, size_t bytes) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kNormMaxSmem));
}

// Shared memory of a CTA of the ragged kernel: two stages of x and r, each
// from one 16-byte boundary to another or the rows' outputs, each row's from a
// boundary on, with a piece beyond.
size_t ragged_range(const NormArgs& a, int rows) {
  return (static_cast<size_t>(rows) * ((a.K + 7) / 8) + 2) * 16;
}
size_t ragged_bytes(const NormArgs& a, int rows) {
  return ragged_range(a, rows) * (a.residual ? 4 : 2);
}

template <typename T, int OUT, int NV, int MAXT>
cudaError_t launch_ragged(const NormArgs& a, int tpr, int rows, cudaStream_t s) {
  const size_t bytes = ragged_bytes(a, rows);
  auto* fn = a.residual ? &norm_ragged_kernel<T, OUT, true, NV, MAXT>
                        : &norm_ragged_kernel<T, OUT, false, NV, MAXT>;
  cudaError_t e = allow_smem(fn, bytes);
  if (e != cudaSuccess) return e;
  // the CTAs that are resident at once
  int dev = 0, sms = 0, per_sm = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, tpr * rows, bytes);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (a.M + rows - 1) / rows, most = static_cast<int64_t>(sms) * per_sm;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = norm_config(dim3(static_cast<unsigned>(blocks < most ? blocks : most)),
                                       dim3(tpr, rows), &attr, s);
  cfg.dynamicSmemBytes = bytes;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<const T*>(a.x),
                            static_cast<const T*>(a.residual), static_cast<const T*>(a.weight),
                            a.M, static_cast<int>(a.K), a.eps, static_cast<T*>(a.h_out), a.y,
                            a.scales, static_cast<uint32_t>(ragged_range(a, rows)));
}

template <typename T, int OUT>
cudaError_t launch_norm_t(const NormArgs& a, cudaStream_t s) {
  const auto at = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; };
  const bool in16 = at(a.x, 16) && at(a.residual, 16);
  const int64_t n = a.K / 8;
  if (a.K % 8 == 0 && in16 && at(a.weight, 16) && at(a.h_out, 16) &&
      at(a.y, OUT == kNorm16 ? 16 : 8)) {
    // two vectors a thread (65536 x 256 fp16 to int8 with a residual 25.5 us with
    // one, 19.4 with two, 18.7 with four; one row 1.26, 1.37 and 1.66)
    if (n <= 512) return launch_held<T, OUT, 2>(a, row_threads(n, 2), s);
    if (n <= 1024) return launch_held<T, OUT, 4>(a, row_threads(n, 4), s);
    if (n <= 4 * kNormThreads * kNormMaxCluster) return launch_split<T, OUT, 4>(a, n, s);
  }
  // vectors of a row a thread: by K alone, as the order of a row's sum
  const int64_t all = (a.K + 7) / 8;
  const int nv = all <= 2 * kNormThreads ? 2 : 4;
  const int tpr = row_threads(all, nv), rows = cta_rows(tpr);
  // (the second condition holds for every K from 9 on: a thread's vectors but
  // its last lie in the row)
  if (in16 && a.K > 8 && (nv - 1) * tpr < all && all <= nv * tpr &&
      ragged_bytes(a, rows) <= kNormMaxSmem) {
    if (nv == 2) return launch_ragged<T, OUT, 2, kNormThreads>(a, tpr, rows, s);
    if (tpr <= kNormThreads) return launch_ragged<T, OUT, 4, kNormThreads>(a, tpr, rows, s);
    if (tpr <= 512) return launch_ragged<T, OUT, 4, 512>(a, tpr, rows, s);
    return launch_ragged<T, OUT, 4, kNormMaxThreads>(a, tpr, rows, s);
  }
  cudaLaunchAttribute attr;
  const cudaLaunchConfig_t cfg =
      norm_config(dim3(static_cast<unsigned>((a.M + rows - 1) / rows)), dim3(tpr, rows), &attr, s);
  return cudaLaunchKernelEx(&cfg, &norm_any_kernel<T, OUT>, static_cast<const T*>(a.x),
                            static_cast<const T*>(a.residual), static_cast<const T*>(a.weight),
                            a.M, static_cast<uint32_t>(a.K), a.eps, static_cast<T*>(a.h_out), a.y,
                            a.scales);
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
