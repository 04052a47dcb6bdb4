// w4_attn.cu — attention over the paged key-value cache on the CUDA cores: any
// head dimension the cache takes, for those without a kernel on the tensor cores
// (a correctness path: 64 sequences of up to 8192 positions, 8 key heads of 128, take
// 5.5 ms here).
//
// For row i of a sequence and its visible keys j,
//   t_j = (q_i . k_j) * scale * log2 e,   out_i = sum_j 2^(t_j - m) v_j / sum_j 2^(t_j - m)
// in one pass with the running maximum m, all in fp32; a row that sees no key
// is zeros.  One warp a row and head: a lane a key for the products, a lane
// every 32nd dimension for the sums over values.
#include <cuda_bf16.h>

#include "w4_cache.cuh"

namespace w4 {
namespace {

constexpr int kSimtWarps = 4;
constexpr int kMaxDim = 256;

template <bool E4M3>
__global__ void __launch_bounds__(32 * kSimtWarps) attn_simt_kernel(AttnArgs a) {
  __shared__ float qs[kSimtWarps][kMaxDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kSimtWarps + warp;
  const int row = static_cast<int>(item / a.heads), head = static_cast<int>(item % a.heads);
  if (row >= a.b.rows) return;
  const int b = find_sequence(a.b, row);
  if (b >= a.b.sequences) return;
  const Sequence s = sequence(a.c, a.b, b);
  if (row < s.row0 || row >= s.row0 + s.n) return;
  const int D = a.c.dim, i = row - s.row0;
  const uint16_t* q = static_cast<const uint16_t*>(a.q) + row * a.q_stride + static_cast<int64_t>(head) * D;
  // queries times a power of two (the scores' scale takes it back): their largest is in
  // [1, 2), so that no product with the codes leaves fp32
  float top_q = 0.f;
  for (int d = lane; d < D; d += 32) {
    const uint16_t w = q[d];
    const float x = a.bf16 ? __bfloat162float(__ushort_as_bfloat16(w)) : __half2float(__ushort_as_half(w));
    qs[warp][d] = x;
    top_q = fmaxf(top_q, fabsf(x));
  }
  for (int o = 16; o > 0; o >>= 1) top_q = fmaxf(top_q, __shfl_xor_sync(0xffffffffu, top_q, o));
  const int E = __float_as_int(top_q) >> 23;
  const int up = E == 255 ? 127 : min(max(254 - E, 1), 253);
  for (int d = lane; d < D; d += 32) qs[warp][d] *= __int_as_float(up << 23);
  __syncwarp();
  const int hk = head / (a.heads / a.c.heads);
  const int pos = a.mask ? draft_position(a, s, i) : s.prefix + i;
  const Visible vis = visible(pos, a.mask ? s.len : min(s.len, pos + 1), a.window, a.sinks);
  const uint8_t* mask = a.mask ? a.mask + static_cast<int64_t>(row) * a.mask_width : nullptr;
  const float scale = a.scale * 1.44269504f * __int_as_float((254 - up) << 23);
  float m = -INFINITY, l = 0.f, acc[kMaxDim / 32];
#pragma unroll
  for (int e = 0; e < kMaxDim / 32; ++e) acc[e] = 0.f;
  // the first keys, then the rest: blocks of 32 below min(sinks, lo) first
  const int first = mask ? min(vis.lo, max(s.prefix, 0)) : vis.lo;
  const int sink_end = min(min(vis.sinks, first), vis.hi);
  for (int part = 0; part < 2; ++part) {
    const int end = part ? vis.hi : sink_end;
    for (int j0 = part ? max(first, sink_end) : 0; j0 < end; j0 += 32) {
      const int j = j0 + lane;
      bool see = j < end;
      if (see && mask) {
        if (j >= s.prefix) see = j - s.prefix < a.mask_width && mask[j - s.prefix] != 0;
        else see = j >= vis.lo || j < vis.sinks;
      }
      int64_t at = see ? place(a.c, a.b, b, j) : -1;
      float t = -INFINITY;
      if (at >= 0) {
        at += static_cast<int64_t>(hk) << a.c.page_shift;
        const uint8_t* k = a.c.k + at * D;
        float dot = 0.f;
        for (int d = 0; d < D; d += 8) {
          const uint2 c = __ldg(reinterpret_cast<const uint2*>(k + d));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 v = codes2_f32<E4M3>((e < 2 ? c.x : c.y) >> (16 * (e & 1)));
            dot = fmaf(v.x, qs[warp][d + 2 * e], dot);
            dot = fmaf(v.y, qs[warp][d + 2 * e + 1], dot);
          }
        }
        t = dot * (scale * __ldg(a.c.k_scales + at));
      }
      float top = t;
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float m_new = fmaxf(m, top);
      const float from = m_new == -INFINITY ? 0.f : m_new;
      const float shrink = exp2f(m - from);
      m = m_new;
      const float p = at >= 0 ? exp2f(t - from) : 0.f;
      l = l * shrink + p;
      const float pv = at >= 0 ? p * __ldg(a.c.v_scales + at) : 0.f;
      // 32 keys' part by itself: added one by one, many small ones would vanish beside a
      // large one (131072 at 2^-25 of it)
      float sum[kMaxDim / 32];
#pragma unroll
      for (int e = 0; e < kMaxDim / 32; ++e) sum[e] = 0.f;
      for (int n = 0; n < 32; ++n) {
        const int64_t from_n = __shfl_sync(0xffffffffu, at, n);
        const float w = __shfl_sync(0xffffffffu, pv, n);
        if (from_n < 0) continue;
        const uint8_t* v = a.c.v + from_n * D;
#pragma unroll
        for (int e = 0; e < kMaxDim / 32; ++e)
          if (lane + 32 * e < D) sum[e] = fmaf(w, codes2_f32<E4M3>(v[lane + 32 * e]).x, sum[e]);
      }
#pragma unroll
      for (int e = 0; e < kMaxDim / 32; ++e) acc[e] = fmaf(acc[e], shrink, sum[e]);
    }
  }
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  // l is 0 where the row sees no key, NaN where it sees a row that holds one
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t* out = static_cast<uint16_t*>(a.out) + (static_cast<int64_t>(row) * a.heads + head) * D;
#pragma unroll
  for (int e = 0; e < kMaxDim / 32; ++e)
    if (lane + 32 * e < D) {
      const float y = acc[e] * inv;
      out[lane + 32 * e] = a.bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(y))
                                  : __half_as_ushort(__float2half_rn(y));
    }
}

}  // namespace

cudaError_t launch_attn_simt(const AttnArgs& a, cudaStream_t s) {
  if (a.b.rows == 0 || a.b.sequences == 0) return cudaSuccess;
  const int64_t items = static_cast<int64_t>(a.b.rows) * a.heads;
  const unsigned grid = static_cast<unsigned>((items + kSimtWarps - 1) / kSimtWarps);
  if (a.c.e4m3) attn_simt_kernel<true><<<grid, 32 * kSimtWarps, 0, s>>>(a);
  else attn_simt_kernel<false><<<grid, 32 * kSimtWarps, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace w4
