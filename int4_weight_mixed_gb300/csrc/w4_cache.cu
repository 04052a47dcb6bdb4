// w4_cache.cu — the paged key-value cache: rows of keys and values quantised as
// they are written (w4_cache_write), and read back as 16-bit rows
// (w4_cache_read).  One scale per position and head, from that row's own
// values, as the per-token activations have (vLLM PR #6547 "Enable Dynamic Per
// Token fp8"; pytorch/ao PR #1113: symmetric int8).  Their quantizer (w4_quant.cu)
// divides by 127 or 448, this one multiplies, so scales may differ in the last bits:
//
//   scale = max_d |x[d]| * (1 / 127) (int8) or (1 / 448) (E4M3), the reciprocal
//           and the product each rounded once to fp32;
//   code  = x[d] / scale rounded once to fp32, then to the nearest integer /
//           E4M3 value, ties to even;
//   read  = code * scale in fp32, rounded once to fp16 / bf16.
//
// Both are bound by HBM, 3 bytes a value and 8 bytes a row and head: 131072
// positions of 8 heads read in 139 us (5.9 TB/s), 21000 rows written as E4M3 in
// 45 us (2.9 TB/s; 35 us without the codes' instructions).  Eight
// values a lane: 16 bytes of them, 8 bytes of codes; a head's row is a group of
// dim / 8 lanes, and consecutive groups of a warp take consecutive heads of a
// row, which are contiguous on the 16-bit side.
#include <type_traits>

#include "w4_cache.cuh"
#include "w4_quant.cuh"

namespace w4 {
namespace {

constexpr int kCacheThreads = 256;
constexpr int kCacheWarps = kCacheThreads / 32;
constexpr int kMaxRows = 32;  // rows a CTA takes
// items (rows of a head) a thread has in flight: the reader 131072 positions in 139 us
// with four, 143 with two; the writer the same with two and four, one row sooner
constexpr int kReadDeep = 4, kWriteDeep = 2;

// A row that has no place: its position is before the first, or its page is
// none of the cache's; and a row of no sequence.
constexpr int64_t kNoPlace = -1, kNoSequence = -2;

// The place of each of the CTA's rows.
__device__ __forceinline__ void find_places(const CacheView& c, const BatchView& b, int row0,
                                            int rows, int64_t* at) {
  for (int r = threadIdx.x >> 5; r < rows; r += kCacheWarps) {
    const int row = row0 + r;
    const int i = find_sequence(b, row);
    int64_t p = kNoSequence;
    if (i < b.sequences) {
      const Sequence s = sequence(c, b, i);
      if (row >= s.row0 && row < s.row0 + s.n) {
        const int pos = s.prefix + (row - s.row0);
        p = pos >= 0 ? place(c, b, i, pos) : kNoPlace;
      }
    }
    if ((threadIdx.x & 31) == 0) at[r] = p;
  }
}

// Item `it` of a CTA: row r, head and kind kvh = kv * heads + h; steps without
// divisions.
struct Item {
  int r, kvh;
  __device__ __forceinline__ void step(int by, int per_row) {
    kvh += by;
    while (kvh >= per_row) {
      kvh -= per_row;
      ++r;
    }
  }
};

// Four values' E4M3 codes, nearest, ties to even.
__device__ __forceinline__ uint32_t pack4_e4m3(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
}
// The E4M3 codes of fl(f / s) without a division a value: with r = fl(1 / s), the
// products of f with r (1 - 2^-21) and r (1 + 2^-21) lie on either side of fl(f / s)
// (r, its multiple, the product and the quotient are each off by 2^-24 at most), so
// where both have the same code, so has what lies between.  The few vectors where
// they differ are divided.
__device__ __forceinline__ uint2 codes8_e4m3(const float (&f)[8], float s) {
  const float r = __frcp_rn(s);
  const float r0 = __fmul_rn(r, 1.f - 0x1p-21f), r1 = __fmul_rn(r, 1.f + 0x1p-21f);
  uint32_t lo[2], hi[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* const x = f + 4 * h;
    lo[h] = pack4_e4m3(x[0] * r0, x[1] * r0, x[2] * r0, x[3] * r0);
    hi[h] = pack4_e4m3(x[0] * r1, x[1] * r1, x[2] * r1, x[3] * r1);
  }
  if (lo[0] != hi[0] || lo[1] != hi[1]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float* const x = f + 4 * h;
      lo[h] = pack4_e4m3(__fdiv_rn(x[0], s), __fdiv_rn(x[1], s), __fdiv_rn(x[2], s), __fdiv_rn(x[3], s));
    }
  }
  return make_uint2(lo[0], lo[1]);
}

// Eight 16-bit values; 16 bytes at once where every row allows it.
template <typename T>
__device__ __forceinline__ uint4 load8(const T* p, bool vec) {
  if (vec) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[2 * i]) |
           static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[2 * i + 1]) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// max |x|, NaN where there is one
template <typename T>
__device__ __forceinline__ float amax_nan(const uint4& v);
template <>
__device__ __forceinline__ float amax_nan<__half>(const uint4& v) {
  const __half2* h = reinterpret_cast<const __half2*>(&v);
  const __half2 m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])),
                                __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
  return __half2float(__hmax_nan(__low2half(m), __high2half(m)));
}
template <>
__device__ __forceinline__ float amax_nan<__nv_bfloat16>(const uint4& v) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&v);
  const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(__habs2(h[0]), __habs2(h[1])),
                                       __hmax2_nan(__habs2(h[2]), __habs2(h[3])));
  return __bfloat162float(__hmax_nan(__low2bfloat16(m), __high2bfloat16(m)));
}

// lanes: lanes of a row (a power of two); dim / 8 of them have values
template <typename T, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads)
    cache_write_kernel(CacheWriteArgs a, int rows, int lanes, int vec) {
  __shared__ int64_t at[kMaxRows];
  const int row0 = blockIdx.x * rows;
  const int count = min(rows, a.b.rows - row0);
  find_places(a.c, a.b, row0, count, at);
  __syncthreads();
  const int H = a.c.heads, D = a.c.dim;
  const int groups = kCacheThreads / lanes;
  const int d = 8 * (threadIdx.x & (lanes - 1));
  const int items = count * 2 * H, first = threadIdx.x / lanes;
  Item next{first / (2 * H), first % (2 * H)};
  // (every thread of a warp makes every turn: the shuffles take whole warps)
  const int turns = (items + groups - 1) / groups;
  for (int turn = 0; turn < turns; turn += kWriteDeep) {
    uint4 x[kWriteDeep];
    int64_t to[kWriteDeep];
    int kv[kWriteDeep];
#pragma unroll
    for (int i = 0; i < kWriteDeep; ++i) {
      x[i] = make_uint4(0, 0, 0, 0);
      to[i] = kNoPlace;
      kv[i] = next.kvh >= H;
      if (next.r < count && d < D && at[next.r] >= 0) {
        const int h = kv[i] ? next.kvh - H : next.kvh;
        const T* const src = static_cast<const T*>(kv[i] ? a.v : a.k) +
                             static_cast<int64_t>(row0 + next.r) * (kv[i] ? a.v_stride : a.k_stride) + h * D + d;
        x[i] = load8(src, vec != 0);
        to[i] = at[next.r] + (static_cast<int64_t>(h) << a.c.page_shift);
      }
      next.step(groups, 2 * H);
    }
#pragma unroll
    for (int i = 0; i < kWriteDeep; ++i) {
      // a NaN or an infinity survives as one larger than any number
      float amax = amax_nan<T>(x[i]);
      if (!(amax < INFINITY)) amax = INFINITY;
      for (int o = lanes >> 1; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      if (to[i] < 0) continue;
      float s = __fmul_rn(amax, E4M3 ? 1.f / 448.f : 1.f / 127.f);
      const bool live = s >= 0x1p-100f && amax < INFINITY;
      if (!live) s = amax < INFINITY ? 0.f : NAN;
      float f[8];
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 v = pair_f32<T>(w[k]);
        f[2 * k] = v.x;
        f[2 * k + 1] = v.y;
      }
      uint2 o = make_uint2(0, 0);
      if (live) {
        if constexpr (E4M3) {
          o = codes8_e4m3(f, s);
        } else {
          float t[8];
          codes8_s8(f, s, __frcp_rn(s), true, t);
          o.x = pack4_s8(__float_as_int(t[0]), __float_as_int(t[1]), __float_as_int(t[2]),
                         __float_as_int(t[3]));
          o.y = pack4_s8(__float_as_int(t[4]), __float_as_int(t[5]), __float_as_int(t[6]),
                         __float_as_int(t[7]));
        }
      }
      *reinterpret_cast<uint2*>((kv[i] ? a.c.v : a.c.k) + to[i] * D + d) = o;
      if (d == 0) (kv[i] ? a.c.v_scales : a.c.k_scales)[to[i]] = s;
    }
  }
}

template <typename T, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads)
    cache_read_kernel(CacheReadArgs a, int rows, int lanes, int vec) {
  __shared__ int64_t at[kMaxRows];
  const int row0 = blockIdx.x * rows;
  const int count = min(rows, a.b.rows - row0);
  find_places(a.c, a.b, row0, count, at);
  __syncthreads();
  const int H = a.c.heads, D = a.c.dim;
  const int groups = kCacheThreads / lanes;
  const int d = 8 * (threadIdx.x & (lanes - 1));
  if (d >= D) return;
  const int first = threadIdx.x / lanes;
  Item next{first / (2 * H), first % (2 * H)};
  while (next.r < count) {
    uint2 c[kReadDeep];
    float s[kReadDeep];
    uint16_t* to[kReadDeep];
#pragma unroll
    for (int i = 0; i < kReadDeep; ++i) {
      c[i] = make_uint2(0, 0);
      s[i] = 0.f;
      to[i] = nullptr;
      if (next.r < count && at[next.r] != kNoSequence) {
        const int64_t p = at[next.r];
        const bool kv = next.kvh >= H;
        const int h = kv ? next.kvh - H : next.kvh;
        if (p >= 0) {
          const int64_t from = p + (static_cast<int64_t>(h) << a.c.page_shift);
          c[i] = __ldg(reinterpret_cast<const uint2*>((kv ? a.c.v : a.c.k) + from * D + d));
          s[i] = __ldg((kv ? a.c.v_scales : a.c.k_scales) + from);
        }
        to[i] = static_cast<uint16_t*>(kv ? a.v : a.k) + (static_cast<int64_t>(row0 + next.r) * H + h) * D + d;
      }
      next.step(groups, 2 * H);
    }
#pragma unroll
    for (int i = 0; i < kReadDeep; ++i) {
      if (!to[i]) continue;
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float2 v = codes2_f32<E4M3>((k < 2 ? c[i].x : c[i].y) >> (16 * (k & 1)));
        v.x *= s[i];
        v.y *= s[i];
        if constexpr (std::is_same<T, __half>::value) {
          const __half2 y = __floats2half2_rn(v.x, v.y);
          o[k] = *reinterpret_cast<const uint32_t*>(&y);
        } else {
          const __nv_bfloat162 y = __floats2bfloat162_rn(v.x, v.y);
          o[k] = *reinterpret_cast<const uint32_t*>(&y);
        }
      }
      if (vec) {
        *reinterpret_cast<uint4*>(to[i]) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) to[i][k] = static_cast<uint16_t>(o[k >> 1] >> (16 * (k & 1)));
      }
    }
  }
}

int lanes_of(int dim) {
  int l = 2;
  while (8 * l < dim) l *= 2;
  return l;
}
// Rows a CTA takes: one while that leaves CTAs for every SM, so that a decode
// batch is spread out; more for longer calls.
int rows_of(int64_t rows) {
  int r = 1;
  while (r < kMaxRows && rows / r > 152 * 16) r *= 2;
  return r;
}
bool aligned(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

cudaError_t launch_cache_write(const CacheWriteArgs& a, cudaStream_t s) {
  if (a.b.rows == 0 || a.b.sequences == 0) return cudaSuccess;
  const int rows = rows_of(a.b.rows), lanes = lanes_of(a.c.dim);
  const int vec = aligned(a.k) && aligned(a.v) && a.k_stride % 8 == 0 && a.v_stride % 8 == 0;
  const unsigned grid = static_cast<unsigned>((a.b.rows + rows - 1) / rows);
  if (a.bf16) {
    if (a.c.e4m3) cache_write_kernel<__nv_bfloat16, true><<<grid, kCacheThreads, 0, s>>>(a, rows, lanes, vec);
    else cache_write_kernel<__nv_bfloat16, false><<<grid, kCacheThreads, 0, s>>>(a, rows, lanes, vec);
  } else {
    if (a.c.e4m3) cache_write_kernel<__half, true><<<grid, kCacheThreads, 0, s>>>(a, rows, lanes, vec);
    else cache_write_kernel<__half, false><<<grid, kCacheThreads, 0, s>>>(a, rows, lanes, vec);
  }
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheReadArgs& a, cudaStream_t s) {
  if (a.b.rows == 0 || a.b.sequences == 0) return cudaSuccess;
  const int rows = rows_of(a.b.rows), lanes = lanes_of(a.c.dim);
  const int vec = aligned(a.k) && aligned(a.v);
  const unsigned grid = static_cast<unsigned>((a.b.rows + rows - 1) / rows);
  if (a.bf16) {
    if (a.c.e4m3) cache_read_kernel<__nv_bfloat16, true><<<grid, kCacheThreads, 0, s>>>(a, rows, lanes, vec);
    else cache_read_kernel<__nv_bfloat16, false><<<grid, kCacheThreads, 0, s>>>(a, rows, lanes, vec);
  } else {
    if (a.c.e4m3) cache_read_kernel<__half, true><<<grid, kCacheThreads, 0, s>>>(a, rows, lanes, vec);
    else cache_read_kernel<__half, false><<<grid, kCacheThreads, 0, s>>>(a, rows, lanes, vec);
  }
  return cudaGetLastError();
}

}  // namespace w4
