// w4_attn_dec.cu — attention over the paged key-value cache for few rows a key
// head (decode steps): bound by the bytes of the visible codes and, short of that,
// by the instructions that make operands of them (646 a warp for 32 keys of 128
// dimensions).  64 sequences of up to 8192 positions, 8 key heads of 128: 131 us,
// 5.0 TB/s; two of 131072: 74 us, 4.9 TB/s; one of 1500: 10 us, latency.  With the
// unit's rows as the MMA's 16 and the keys as its 8 (half of it empty with up to
// eight rows): 144 and 77 us.
//
// A unit is 8 or 16 rows (query heads of a key head, of one token or a few) by the
// key tiles they see; four warps of a CTA take 32 keys each of a 128-key tile.
// mma.sync m16n8k16 in fp16, both kinds of codes being exact there, with keys (for
// the sums, dimensions) as its 16 rows and the unit's rows as its 8 columns: a decode
// step's few rows leave none of it empty.
//
//   t_j = (q . code_j) * (scale * log2 e * ks_j) + log2 vs_j
//   p_j = 2^(t_j - m + 7) <= 2^15,  m a running maximum of t
//   O  += p_j * code_j (fp16 p, fp32 sums),  l += p_j 2^-7 / vs_j,  out = 2^-7 O / l
//
// with ks, vs the key's and value's scales: both enter the exponent, so the
// codes go to the tensor cores as they are, and p is rounded to fp16 relative to
// what it weighs, however far apart the values' scales are.  m moves only when a
// row's maximum grows by more than 2^8 (sums are rescaled then).  Queries are
// fp16 times a power of two of each row (bf16 ones fit: what falls below fp16's
// subnormals is 2^-25 of the row's largest).
//
// Every warp streams its own keys through its own ring of shared memory
// (cp.async, 16 bytes a lane) and meets the others only at the unit's end.
// Positions are read in any order within an MMA, so that a lane loads 16
// neighbouring codes at once: for scores they are consecutive k of its key's
// row, for sums consecutive dimensions of its four keys, whose bytes PRMT pairs.
// Probabilities come out a key a lane and are transposed by movmatrix.
// Slots behind the sequence's end and pages that are none are not read: zeros
// stand for their codes, and log2 vs = kNoKey for their scales.
#include <cuda_bf16.h>

#include "w4_attn_math.cuh"
#include "w4_attn_plan.cuh"

namespace w4 {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 32;          // keys of a warp's stage
constexpr int kTile = kKeys * kWarps;
constexpr int kThreads = 32 * kWarps;
constexpr float kUnlift = 1.f / (1 << kDecLift);

// CTAs an SM: two for 16 rows of 128 dimensions (three spill registers), else three
// (64 sequences 131 us, with two 139; 64 dimensions: 48 windows 50 us, with four 51).
__host__ __device__ constexpr int ctas_per_sm(int dim, int nt) { return dim == 128 && nt == 2 ? 2 : 3; }

template <int D, int NT>
struct Ring {
  static constexpr int kCodes = kKeys * D;                // bytes of one array
  static constexpr int kStage = 2 * kCodes + 2 * kKeys * 4;
  static constexpr int kStages = D == 64 ? 4 : NT == 2 ? 3 : 2;
  // then the factors of the stage in use: of a key ks, log2 vs, 2^-7 / vs
  static constexpr int kFactors = kStage * kStages;
  static constexpr int kWarp = kFactors + kKeys * 16;
};
template <int D, int NT>
constexpr size_t smem_bytes() {
  constexpr size_t ring = static_cast<size_t>(Ring<D, NT>::kWarp) * kWarps;
  constexpr size_t sums = static_cast<size_t>(kWarps) * 8 * NT * D * 4;
  return ring > sums ? ring : sums;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Transposes an 8 x 8 matrix of 16-bit values, a row's pair a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Where 16-byte chunk c of key `key` (of the stage's 16) lies within an array's
// bytes, so that the lanes of a 16-byte (8-byte: values of 64) access hit
// different banks: for keys, lanes 0-7 read four chunks of two neighbouring keys;
// for values, two neighbouring chunks of every other key.
template <int D>
__device__ __forceinline__ uint32_t k_chunk(int key, int c) {
  if constexpr (D == 128) return key * 128 + ((c ^ (key & 1) << 2) << 4);
  else return key * 64 + (c << 4);
}
template <int D>
__device__ __forceinline__ uint32_t v_chunk(int key, int c) {
  if constexpr (D == 128) return key * 128 + ((c ^ (key & 7)) << 4);
  else
    return (key >> 1) * 128 + ((key ^ key >> 1) & 1) * 64 + ((c ^ (key >> 2 & 1) << 1) << 4);
}
// The place of 16-byte chunk c of a row of sums, by the same token: lanes write D / 8
// neighbouring dimensions of every other row.
template <int D>
__device__ __forceinline__ int sum_chunk(int row, int c) {
  const int t = row >> 1 & 3;
  const int x = D == 128 ? t : (t & 1) | (t & 2) << 1;
  return row * (D / 4) + (c ^ x);
}

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(D, NT)) attn_dec_kernel(AttnArgs a, int least) {
  using R = Ring<D, NT>;
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Piece piece;
  __shared__ float part_m[kWarps][kRows], part_l[kWarps][kRows];
  __shared__ int position[kRows];
  __shared__ int last_one;
  plan_piece<kRows, kTile, kThreads>(a, least, &piece);
  if (piece.begin == piece.end) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int group = a.heads / a.c.heads;
  const uint32_t ring = smem_addr(smem) + warp * R::kWarp;
  const uint8_t* const ring_p = smem + warp * R::kWarp;
  float4* const factors = reinterpret_cast<float4*>(smem + warp * R::kWarp + R::kFactors);
  float4* const sums = reinterpret_cast<float4*>(smem);

  Walk<kRows, kTile> w;
  w.start(a, piece);
  for (;;) {
    const Sequence s = w.s;
    const int r0 = w.rt * kRows, nr = min(kRows, s.n * group - r0);
    // positions of the rows of a tree
    if (a.mask) {
      __syncthreads();
      const int first = r0 / group, count = (r0 + nr - 1) / group - first + 1;
      for (int i = warp; i < count; i += kWarps) {
        const int p = draft_position(a, s, first + i);
        if (lane == 0) position[i] = p;
      }
      __syncthreads();
    }

    // queries of row 8 e + g, as fp16 times a power of two; the scale of its scores
    float row_rf[NT];
    uint32_t qf[NT][D / 16][2];
#pragma unroll
    for (int e = 0; e < NT; ++e) {
      const int r = g + 8 * e;
      float x[D / 4];
#pragma unroll
      for (int i = 0; i < D / 4; ++i) x[i] = 0.f;
      if (r < nr) {
        const int token = (r0 + r) / group, head = w.h * group + (r0 + r) % group;
        const uint16_t* q = static_cast<const uint16_t*>(a.q) +
                            (static_cast<int64_t>(s.row0) + token) * a.q_stride + head * D;
        const bool vec = (reinterpret_cast<uintptr_t>(q) & 15) == 0;
#pragma unroll
        for (int j = 0; j < D / 64; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint16_t* from = q + 64 * j + 16 * t4 + 8 * i;
            uint32_t u[4];
            if (vec) {
              const uint4 v4 = __ldg(reinterpret_cast<const uint4*>(from));
              u[0] = v4.x, u[1] = v4.y, u[2] = v4.z, u[3] = v4.w;
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                u[k] = static_cast<uint32_t>(from[2 * k]) | static_cast<uint32_t>(from[2 * k + 1]) << 16;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float2 f;
              if (a.bf16) f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[k]));
              else f = __half22float2(*reinterpret_cast<const __half2*>(&u[k]));
              x[16 * j + 8 * i + 2 * k] = f.x;
              x[16 * j + 8 * i + 2 * k + 1] = f.y;
            }
          }
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(x[i]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^up, with top * 2^up in [1, 2) (an infinity stays one)
      const int E = __float_as_int(top) >> 23;
      const int up = E == 255 ? 127 : min(max(254 - E, 1), 253);
      const float grow = __int_as_float(up << 23);
      row_rf[e] = a.scale * 1.44269504f * __int_as_float((254 - up) << 23);
#pragma unroll
      for (int j = 0; j < D / 64; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int o = 16 * j + 4 * i;
          const __half2 p0 = __floats2half2_rn(x[o] * grow, x[o + 1] * grow);
          const __half2 p1 = __floats2half2_rn(x[o + 2] * grow, x[o + 3] * grow);
          qf[e][4 * j + i][0] = *reinterpret_cast<const uint32_t*>(&p0);
          qf[e][4 * j + i][1] = *reinterpret_cast<const uint32_t*>(&p1);
        }
    }
    // this lane's rows of the scores, 8 e + 2 t4 + i: what they see
    int hi[NT][2], lo[NT][2];
    const uint8_t* mask[NT][2];
    float2 rf[NT];
#pragma unroll
    for (int e = 0; e < NT; ++e) {
      rf[e].x = __shfl_sync(0xffffffffu, row_rf[e], 8 * t4);
      rf[e].y = __shfl_sync(0xffffffffu, row_rf[e], 8 * t4 + 4);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 8 * e + 2 * t4 + i;
        hi[e][i] = lo[e][i] = 0;
        mask[e][i] = nullptr;
        if (r < nr) {
          const int token = (r0 + r) / group;
          const int pos = a.mask ? position[token - r0 / group] : s.prefix + token;
          const Visible v = visible(pos, a.mask ? s.len : min(s.len, pos + 1), a.window, a.sinks);
          hi[e][i] = v.hi;
          lo[e][i] = v.lo;
          if (a.mask) mask[e][i] = a.mask + (static_cast<int64_t>(s.row0) + token) * a.mask_width;
        }
      }
    }
    // keys that every row sees: [lo_all, hi_all) and below `sinks`
    int hi_all, lo_all;
    if (a.mask) {
      hi_all = s.prefix;
      lo_all = a.window > 0 ? s.prefix + s.n - a.window : 0;
    } else {
      hi_all = min(s.len, s.prefix + r0 / group + 1);
      lo_all = a.window > 0 ? s.prefix + (r0 + nr - 1) / group - a.window + 1 : 0;
    }

    float m[NT][2];
    float2 l[NT];  // of rows 2 t4 and 2 t4 + 1, this lane's keys
    float o[NT][D / 16][4];
#pragma unroll
    for (int e = 0; e < NT; ++e) {
      m[e][0] = m[e][1] = -INFINITY;
      l[e] = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[e][i][k] = 0.f;
    }

    // the pages of this warp's two groups of 16 keys in a tile, looked up 16 tiles at
    // a time: lane 2 i + n has that of group n of tile base + i
    const int32_t* const line = a.b.table + w.b * a.b.width;
    const auto look_up = [&](int i) -> int {
      i += lane >> 1;
      if (i >= w.to) return -1;
      const int key = tile_at(w.t, i) * kTile + warp * kKeys + 16 * (lane & 1);
      if (key >= s.len) return -1;
      const int page = __ldg(line + (key >> a.c.page_shift));
      return page >= 0 && page < a.c.pages ? page : -1;
    };
    int base = w.from;
    int pages = look_up(base), pages_next = look_up(base + 16);
    const auto page_of = [&](int i, int n) -> int {
      const int d = 2 * (i - base) + n;
      return d < 32 ? __shfl_sync(0xffffffffu, pages, d) : __shfl_sync(0xffffffffu, pages_next, d - 32);
    };
    const auto load = [&](int i, int slot) {
      const uint32_t dst = ring + slot * R::kStage;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int page = page_of(i, n);
        const int key = tile_at(w.t, i) * kTile + warp * kKeys + 16 * n;
        const int valid = page >= 0 ? min(s.len - key, 16) : 0;
        const int64_t at = page < 0 ? 0
                                    : ((static_cast<int64_t>(page) * a.c.heads + w.h) << a.c.page_shift) +
                                          (key & ((1 << a.c.page_shift) - 1));
        const uint8_t *k = a.c.k + at * D, *v = a.c.v + at * D;
#pragma unroll
        for (int u = 0; u < D / 32; ++u) {
          const int e = lane + 32 * u, row = e / (D / 16), c = e % (D / 16);
          const uint32_t bytes = row < valid ? 16 : 0;
          cp_async16(dst + n * 16 * D + k_chunk<D>(row, c), k + e * 16, bytes);
          cp_async16(dst + R::kCodes + n * 16 * D + v_chunk<D>(row, c), v + e * 16, bytes);
        }
        if (lane >> 3 == n) {  // four lanes for ks, four for vs
          const int q = lane & 3;
          const float* sc = (lane & 4 ? a.c.v_scales : a.c.k_scales) + at + 4 * q;
          cp_async16(dst + 2 * R::kCodes + (lane & 4 ? kKeys * 4 : 0) + n * 64 + q * 16, sc,
                     4 * min(max(valid - 4 * q, 0), 4));
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < R::kStages - 1; ++i) load(w.from + i, i);

    int slot = 0;
    for (int i = w.from; i < w.to; ++i) {
      if (i - base >= 16) {
        base += 16;
        pages = pages_next;
        pages_next = look_up(base + 16);
      }
      cp_async_wait<R::kStages - 2>();
      __syncwarp();
      // (asked for before this stage is used: its slot is the one left last)
      load(i + R::kStages - 1, slot == 0 ? R::kStages - 1 : slot - 1);
      const int page0 = page_of(i, 0), page1 = page_of(i, 1);
      if (page0 >= 0 || page1 >= 0) {
        const uint8_t* const st = ring_p + slot * R::kStage;
        const int key0 = tile_at(w.t, i) * kTile + warp * kKeys;
        // the factors of the warp's keys, a key a lane
        {
          const float* const sc = reinterpret_cast<const float*>(st + 2 * R::kCodes);
          const bool in = (lane < 16 ? page0 : page1) >= 0 && key0 + lane < s.len;
          const float ks = sc[lane], vs = sc[kKeys + lane];
          const float safe = counted(vs);
          factors[lane] = make_float4(in ? ks + (vs - vs) : 0.f,  // NaN where vs is
                                      in ? lg2(safe) : kNoKey,
                                      in ? rcp(safe) * kUnlift : 0.f, 0.f);
          __syncwarp();
        }
        // scores: two blocks of sixteen keys by the rows
        float c[2][NT][4];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int e = 0; e < NT; ++e)
#pragma unroll
            for (int k = 0; k < 4; ++k) c[b][e][k] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          uint32_t ww[4][4];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const uint4 w4 = *reinterpret_cast<const uint4*>(st + (n >> 1) * 16 * D +
                                                             k_chunk<D>(8 * (n & 1) + g, 4 * j + t4));
            ww[n][0] = w4.x, ww[n][1] = w4.y, ww[n][2] = w4.z, ww[n][3] = w4.w;
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              uint32_t a0, a1, a2, a3;
              codes4_f16<E4M3>(ww[2 * b][q], a0, a2);
              codes4_f16<E4M3>(ww[2 * b + 1][q], a1, a3);
#pragma unroll
              for (int e = 0; e < NT; ++e)
                mma16816(c[b][e], a0, a1, a2, a3, qf[e][4 * j + q][0], qf[e][4 * j + q][1]);
            }
        }
        // this lane's keys: g, g + 8, g + 16, g + 24
        float rvs[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const float4 f = factors[8 * n + g];
          rvs[n] = f.z;
#pragma unroll
          for (int e = 0; e < NT; ++e) {
            float* const y = &c[n >> 1][e][2 * (n & 1)];
            // (the factors first: products of large queries would leave fp32 before a small
            // key's scale brings them back)
            const float2 x = fma2(make_float2(y[0], y[1]), mul2(rf[e], make_float2(f.x, f.x)),
                                  make_float2(f.y, f.y));
            y[0] = x.x, y[1] = x.y;
          }
        }
        if (!(key0 + kKeys <= hi_all && (key0 >= lo_all || key0 + kKeys <= a.sinks))) {
#pragma unroll
          for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < NT; ++e)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int j = key0 + 8 * n + g;
                bool see = j < hi[e][i];
                if (mask[e][i] && j >= s.prefix)
                  see = see && j - s.prefix < a.mask_width && mask[e][i][j - s.prefix] != 0;
                else
                  see = see && (j >= lo[e][i] || j < a.sinks);
                if (!see) c[n >> 1][e][2 * (n & 1) + i] = -INFINITY;
              }
        }
        // the running maximum, of a row over the eight lanes that have its keys
        float top[NT][2];
        bool grows = false;
#pragma unroll
        for (int e = 0; e < NT; ++e)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x = fmaxf(max3(c[0][e][i], c[0][e][2 + i], c[1][e][i]), c[1][e][2 + i]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            if (x < 0.5f * kNoKey) x = -INFINITY;  // no key but such that are none
            top[e][i] = x;
            grows |= x > m[e][i] + kSlack;
          }
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
          for (int e = 0; e < NT; ++e) {
            float shrink[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float to = fmaxf(m[e][i], top[e][i]);
              shrink[i] = to == -INFINITY ? 1.f : ex2(m[e][i] - to);
              m[e][i] = to;
            }
            l[e].x *= shrink[0];
            l[e].y *= shrink[1];
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              o[e][d][0] *= shrink[0];
              o[e][d][1] *= shrink[1];
              o[e][d][2] *= shrink[0];
              o[e][d][3] *= shrink[1];
            }
          }
        }
        uint32_t p[NT][4];  // of eight keys each: row g's pair of keys 2 t4
#pragma unroll
        for (int e = 0; e < NT; ++e) {
          const float2 from = make_float2(m[e][0] == -INFINITY ? 0.f : kDecLift - m[e][0],
                                          m[e][1] == -INFINITY ? 0.f : kDecLift - m[e][1]);
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const float* const y = &c[n >> 1][e][2 * (n & 1)];
            float2 x = add2(make_float2(y[0], y[1]), from);
            x.x = ex2(x.x);
            x.y = ex2(x.y);
            l[e] = fma2(x, make_float2(rvs[n], rvs[n]), l[e]);
            const __half2 h = __floats2half2_rn(x.x, x.y);
            p[e][n] = transpose8(*reinterpret_cast<const uint32_t*>(&h));
          }
        }
        // sums: this lane's dimensions D / 8 * g .. of four keys at a time
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          const uint8_t* const vp = st + R::kCodes + kk * 16 * D;
          uint32_t v[4][D / 32];
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const int key = 8 * (n >> 1) + 2 * t4 + (n & 1);
            if constexpr (D == 128) {
              const uint4 w4 = *reinterpret_cast<const uint4*>(vp + v_chunk<D>(key, g));
              v[n][0] = w4.x, v[n][1] = w4.y, v[n][2] = w4.z, v[n][3] = w4.w;
            } else {
              const uint2 w2 = *reinterpret_cast<const uint2*>(vp + v_chunk<D>(key, g >> 1) + 8 * (g & 1));
              v[n][0] = w2.x, v[n][1] = w2.y;
            }
          }
#pragma unroll
          for (int q = 0; q < D / 32; ++q)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              // dimensions 4 q + 2 hf and the next of the lane's: rows g and g + 8
              const uint32_t sel = hf ? 0x7362 : 0x5140;
              uint32_t a0, a1, a2, a3;
              codes4_f16<E4M3>(prmt(v[0][q], v[1][q], sel), a0, a1);
              codes4_f16<E4M3>(prmt(v[2][q], v[3][q], sel), a2, a3);
#pragma unroll
              for (int e = 0; e < NT; ++e)
                mma16816(o[e][2 * q + hf], a0, a1, a2, a3, p[e][2 * kk], p[e][2 * kk + 1]);
            }
        }
      }
      slot = slot + 1 == R::kStages ? 0 : slot + 1;
    }
    cp_async_wait<0>();

    // the four warps' sums, relative to the largest maximum
#pragma unroll
    for (int e = 0; e < NT; ++e) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        l[e].x += __shfl_xor_sync(0xffffffffu, l[e].x, x);
        l[e].y += __shfl_xor_sync(0xffffffffu, l[e].y, x);
      }
      if (g == 0) {
        part_m[warp][8 * e + 2 * t4] = m[e][0];
        part_m[warp][8 * e + 2 * t4 + 1] = m[e][1];
        part_l[warp][8 * e + 2 * t4] = l[e].x;
        part_l[warp][8 * e + 2 * t4 + 1] = l[e].y;
      }
    }
    __syncthreads();  // the rings are free
#pragma unroll
    for (int e = 0; e < NT; ++e)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * e + 2 * t4 + i;
        if (row < nr) {
#pragma unroll
          for (int q = 0; q < D / 32; ++q)
            sums[warp * kRows * (D / 4) + sum_chunk<D>(row, (D / 32) * g + q)] =
                make_float4(o[e][2 * q][i], o[e][2 * q][2 + i], o[e][2 * q + 1][i], o[e][2 * q + 1][2 + i]);
        }
      }
    __syncthreads();
    const int64_t u0 = w.unit_begin();
    const int c0 = piece_of(piece.total, piece.pieces, u0);
    const int c1 = piece_of(piece.total, piece.pieces, u0 + w.t.count - 1);
    const bool whole = c0 == c1;
    // partial sums of CTA c: slot 2 c where the unit began before its piece, 2 c + 1
    // where it begins in it
    constexpr int kSlot = kRows * D + 2 * kRows;  // floats
    const auto slot_of = [&](int c) {
      return a.partials + (2 * static_cast<int64_t>(c) + (c == c0)) * kSlot;
    };
    const auto store = [&](int r, int c, float4 y) {
      const int token = (r0 + r) / group, head = w.h * group + (r0 + r) % group;
      uint16_t* const to = static_cast<uint16_t*>(a.out) +
                           ((static_cast<int64_t>(s.row0) + token) * a.heads + head) * D + 4 * c;
      uint32_t u[2];
      if (a.bf16) {
        const __nv_bfloat162 p0 = __floats2bfloat162_rn(y.x, y.y), p1 = __floats2bfloat162_rn(y.z, y.w);
        u[0] = *reinterpret_cast<const uint32_t*>(&p0);
        u[1] = *reinterpret_cast<const uint32_t*>(&p1);
      } else {
        const __half2 p0 = __floats2half2_rn(y.x, y.y), p1 = __floats2half2_rn(y.z, y.w);
        u[0] = *reinterpret_cast<const uint32_t*>(&p0);
        u[1] = *reinterpret_cast<const uint32_t*>(&p1);
      }
      if ((reinterpret_cast<uintptr_t>(to) & 7) == 0) {
        *reinterpret_cast<uint2*>(to) = make_uint2(u[0], u[1]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = static_cast<uint16_t>(u[i >> 1] >> (16 * (i & 1)));
      }
    };
    for (int i = tid; i < nr * (D / 4); i += kThreads) {
      const int r = i / (D / 4), c = i % (D / 4);
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) top = fmaxf(top, part_m[k][r]);
      const float from = top == -INFINITY ? 0.f : top;
      float sum_l = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float f = ex2(part_m[k][r] - from);
        const float4 x = sums[k * kRows * (D / 4) + sum_chunk<D>(r, c)];
        sum_l = fmaf(f, part_l[k][r], sum_l);
        y.x = fmaf(f, x.x, y.x);
        y.y = fmaf(f, x.y, y.y);
        y.z = fmaf(f, x.z, y.z);
        y.w = fmaf(f, x.w, y.w);
      }
      if (whole) {
        const float inv = sum_l == 0.f ? 0.f : kUnlift / sum_l;
        store(r, c, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
      } else {
        float* const to = slot_of(blockIdx.x);
        __stcg(reinterpret_cast<float4*>(to) + r * (D / 4) + c, y);
        if (c == 0) __stcg(reinterpret_cast<float2*>(to + kRows * D) + r, make_float2(top, sum_l));
      }
    }
    if (!whole) {
      // the last of the unit's CTAs adds the partial sums, in their order
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const int n = atomicAdd(a.counters + c0, 1);
        last_one = n == c1 - c0;
        if (last_one) a.counters[c0] = 0;
        __threadfence();
      }
      __syncthreads();
      if (last_one) {
        for (int i = tid; i < nr * (D / 4); i += kThreads) {
          const int r = i / (D / 4), c = i % (D / 4);
          float top = -INFINITY, sum_l = 0.f;
          float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
          constexpr int kAhead = 4;
          for (int k0 = c0; k0 <= c1; k0 += kAhead) {
            float4 x[kAhead];
            float2 ml[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
              ml[k] = make_float2(-INFINITY, 0.f);
              x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (k0 + k <= c1) {
                const float* const at = slot_of(k0 + k);
                ml[k] = __ldcg(reinterpret_cast<const float2*>(at + kRows * D) + r);
                x[k] = __ldcg(reinterpret_cast<const float4*>(at) + r * (D / 4) + c);
              }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
              const float to = fmaxf(top, ml[k].x);
              const float from = to == -INFINITY ? 0.f : to;
              const float f = ex2(top - from), fk = ex2(ml[k].x - from);
              top = to;
              sum_l = sum_l * f + fk * ml[k].y;
              y.x = y.x * f + fk * x[k].x;
              y.y = y.y * f + fk * x[k].y;
              y.z = y.z * f + fk * x[k].z;
              y.w = y.w * f + fk * x[k].w;
            }
          }
          const float inv = sum_l == 0.f ? 0.f : kUnlift / sum_l;
          store(r, c, make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv));
        }
      }
    }
    if (!w.next(a)) break;
    __syncthreads();  // the sums are read
  }
}

template <int D, bool E4M3, int NT>
cudaError_t launch(const AttnArgs& a, int sms, cudaStream_t s) {
  constexpr size_t smem = smem_bytes<D, NT>();
  const cudaError_t e = cudaFuncSetAttribute(attn_dec_kernel<D, E4M3, NT>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  // no more CTAs than there can be tiles
  const int64_t units = static_cast<int64_t>(a.c.heads) *
                        (static_cast<int64_t>(a.b.rows) * (a.heads / a.c.heads) / (8 * NT) + a.b.sequences);
  const int64_t tiles = units * (((a.b.width << a.c.page_shift) + kTile - 1) / kTile + 1);
  const int ctas = ctas_per_sm(D, NT) * sms;
  attn_dec_kernel<D, E4M3, NT>
      <<<tiles < ctas ? static_cast<int>(tiles) : ctas, kThreads, smem, s>>>(a, 1);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_dim(const AttnArgs& a, int sms, cudaStream_t s) {
  // eight rows a unit where a key head has no more on average
  const bool eight = static_cast<int64_t>(a.b.rows) * a.heads <=
                     8 * static_cast<int64_t>(a.b.sequences) * a.c.heads;
  if (eight) return a.c.e4m3 ? launch<D, true, 1>(a, sms, s) : launch<D, false, 1>(a, sms, s);
  return a.c.e4m3 ? launch<D, true, 2>(a, sms, s) : launch<D, false, 2>(a, sms, s);
}

}  // namespace

size_t attn_dec_partials(int sms, int dim) {
  const auto bytes = [&](int nt) {
    return 2 * static_cast<size_t>(ctas_per_sm(dim, nt) * sms) * (8 * nt * dim + 2 * 8 * nt) * sizeof(float);
  };
  return bytes(1) > bytes(2) ? bytes(1) : bytes(2);
}

cudaError_t launch_attn_dec(const AttnArgs& a, int sms, cudaStream_t s) {
  return a.c.dim == 128 ? launch_dim<128>(a, sms, s) : launch_dim<64>(a, sms, s);
}

}  // namespace w4
