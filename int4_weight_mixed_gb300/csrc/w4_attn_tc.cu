// w4_attn_tc.cu — attention over the paged key-value cache for many rows a key
// head (prompts, chunks, trees of drafts): on the tensor cores (tcgen05), bound
// by them and, short of that, by the instructions of the softmax.
//
// A unit is up to 256 rows (query heads of a key head times tokens) by the tiles
// of 128 keys they see.  Per tile and 128 rows X:
//
//   S_X = Q_X K^T         K: codes as 16-bit values, exact; S in tensor memory
//   t_j = S_j * (scale * log2 e * ks_j) + log2 vs_j       (ks, vs: the scales)
//   P_j = 2^(t_j - m) <= 2^8, fp16, written over S in tensor memory
//   O_X += P V            V: codes as fp16, exact;  l += P_j / vs_j;  out = O / l
//
// as in w4_attn_dec.cu: both scales enter the exponent, so that no code is
// rounded and P is rounded relative to what it weighs.  Keys that are none
// (behind the end, of no page) have log2 vs = -infinity and codes of zero.
//
// Sixteen warps, one CTA an SM:
//   warps 0-3, 4-7   the softmax of rows 0-127 and 128-255, a thread a row; they
//                    also load Q, rescale O when m moves, and write the result
//   warps 8-11       load codes (a tile ahead, in registers) and write them as
//                    16-bit values in the MMA's layout: K rows by key, V
//                    transposed (rows by dimension, bytes of key pairs put
//                    together by PRMT); they also make the scales' factors
//   warp 12          issues the MMAs.  While the softmax works on one half, the
//                    tensor cores work on the other.
// Units of up to 128 rows put their even key tiles through the first half and
// the odd ones through the second, with the same Q, and join the two at the end.
// Units cut between CTAs leave partial sums that attn_tc_reduce_kernel adds.
#include "w4_attn_math.cuh"
#include "w4_attn_plan.cuh"

namespace w4 {
namespace {

constexpr int kTcRows = 256;   // rows of a unit
constexpr int kHalf = 128;
constexpr int kTcKeys = 128;   // keys of a tile
constexpr int kTcCta = 512;
constexpr int kConvWarp = 8, kIssueWarp = 12;
// registers a thread after the split: 2 * 176 + 104 + 56 = 512 = 4 * 128 launched
constexpr int kSoftRegs = 176, kConvRegs = 104, kIssueRegs = 56;
static_assert(2 * kSoftRegs + kConvRegs + kIssueRegs <= 4 * 128, "register split");

template <int D>
struct Tc {
  static constexpr int kStages = D == 128 ? 2 : 4;    // of K and of V
  // of the scales' factors: a slot is written again two tiles after the stage's
  // last use, when the softmax has read it
  static constexpr int kSlots = kStages + 2;
  static constexpr int kQ = kHalf * D * 2;            // bytes of a half's queries
  static constexpr int kTileBytes = kTcKeys * D * 2;  // of a stage of K or V
  static constexpr int kFactors = 3 * kTcKeys * 4;    // ks', log2 vs, 1 / vs
  static constexpr int kBytes = 2 * kQ + 2 * kStages * kTileBytes + kSlots * kFactors;
  static constexpr int kSmem = kBytes + 1024;         // (for the alignment of the first)
  // tensor memory columns: S (P in its first half) of both halves, then O
  static constexpr int kS = 0, kO = 2 * kTcKeys;
  // partial sums of a piece, in floats: [D / 4][rows] of 16 bytes, [rows] of (m, l)
  static constexpr int64_t kSlot = static_cast<int64_t>(kTcRows) * (D + 2);
};

struct TcBarriers {
  uint64_t q_full, join, k_full[4], k_empty[4], v_full[4], v_empty[4], f_full[6], s_full[2], p_full[2],
      pv_done[2];
};

__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// D[128 x N] (+)= A[128 x 16] B[16 x N], both operands in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// A unit cut between CTAs, for the kernel that adds it up: written by the CTA
// that it begins in (last_cta < 0: none).
struct Cut {
  int b, h, rt, last_cta;
};
constexpr int kCutInts = sizeof(Cut) / 4;

// Bits i < n of a word.
__device__ __forceinline__ uint32_t below(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1;
}

// ---------------------------------------------------------------- the roles
template <int D, bool E4M3, bool BF16>
struct AttnTc {
  using T = Tc<D>;
  const AttnArgs& a;
  const Piece& piece;
  TcBarriers& bar;
  uint8_t* smem;
  uint32_t base;  // shared address of smem
  uint32_t tmem;
  volatile int* abort;
  Cut* cuts;
  float* partials;
  float *join_m, *join_l;

  using Way = Walk<kTcRows, kTcKeys>;

  __device__ __forceinline__ uint32_t q_at(int half) const { return base + half * T::kQ; }
  __device__ __forceinline__ uint32_t k_at(int st) const { return base + 2 * T::kQ + st * T::kTileBytes; }
  __device__ __forceinline__ uint32_t v_at(int st) const {
    return base + 2 * T::kQ + (T::kStages + st) * T::kTileBytes;
  }
  __device__ __forceinline__ float* factors(int slot) const {
    return reinterpret_cast<float*>(smem + 2 * T::kQ + 2 * T::kStages * T::kTileBytes +
                                    slot * T::kFactors);
  }
  // A whole warp: it goes on or gives up as one.
  __device__ __forceinline__ bool wait(uint64_t& b, uint32_t parity) const {
    return __all_sync(0xffffffffu, mbar_wait(&b, parity & 1, abort, a.status));
  }
  // The one thread that issues.
  __device__ __forceinline__ bool wait1(uint64_t& b, uint32_t parity) const {
    return mbar_wait(&b, parity & 1, abort, a.status);
  }
  // Both halves of the softmax meet (bounded, like every wait here).
  __device__ __forceinline__ bool meet(uint32_t& meets) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bar.join);
    return wait(bar.join, meets++);
  }
  __device__ __forceinline__ int rows_of(const Way& w) const {
    return min(kTcRows, w.s.n * (a.heads / a.c.heads) - w.rt * kTcRows);
  }

  // ---- warp 12, one thread
  __device__ void issue() {
    const uint32_t id_qk = idesc_f16(BF16 ? 1u : 0u, kTcKeys), id_pv = idesc_f16(0u, D);
    uint32_t units = 0, kc = 0, vc = 0, pc[2] = {0, 0};
    Way w;
    w.start(a, piece);
    const auto qk = [&](int half, int q, uint32_t st) {
      const uint64_t qd = sw128_kmajor_desc(q_at(q)), kd = sw128_kmajor_desc(k_at(st));
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint64_t off = static_cast<uint64_t>(i >> 2) * (kHalf * 128 >> 4) + 2 * (i & 3);
        mma_ss(tmem + T::kS + half * kTcKeys, qd + off, kd + off, id_qk, i != 0);
      }
      mma_commit(&bar.s_full[half]);
    };
    const auto pv = [&](int half, uint32_t st, bool add) {
      const uint64_t vd = sw128_kmajor_desc(v_at(st));
#pragma unroll
      for (int i = 0; i < kTcKeys / 16; ++i)
        mma_ts(tmem + T::kO + half * D, tmem + T::kS + half * kTcKeys + 8 * i,
               vd + static_cast<uint64_t>(i >> 2) * (D * 128 >> 4) + 2 * (i & 3), id_pv,
               add || i != 0);
      mma_commit(&bar.pv_done[half]);
    };
    for (;;) {
      const int n = w.to - w.from;
      const bool full = rows_of(w) > kHalf;
      if (!wait1(bar.q_full, units++)) return;
      if (full) {
        uint32_t st = kc % T::kStages;
        if (!wait1(bar.k_full[st], kc / T::kStages)) return;
        tc_fence_after();
        qk(0, 0, st);
        qk(1, 1, st);
        mma_commit(&bar.k_empty[st]);
        ++kc;
        for (int i = 0; i < n; ++i) {
          const uint32_t vs = vc % T::kStages;
          st = kc % T::kStages;
          if (!wait1(bar.v_full[vs], vc / T::kStages)) return;
          if (!wait1(bar.p_full[0], pc[0]++)) return;
          tc_fence_after();
          pv(0, vs, i > 0);
          if (i + 1 < n) {
            if (!wait1(bar.k_full[st], kc / T::kStages)) return;
            tc_fence_after();
            qk(0, 0, st);
          }
          if (!wait1(bar.p_full[1], pc[1]++)) return;
          tc_fence_after();
          pv(1, vs, i > 0);
          mma_commit(&bar.v_empty[vs]);
          ++vc;
          if (i + 1 < n) {
            qk(1, 1, st);
            mma_commit(&bar.k_empty[st]);
            ++kc;
          }
        }
      } else {
        const auto next_qk = [&](int half) {
          const uint32_t st = kc % T::kStages;
          if (!wait1(bar.k_full[st], kc / T::kStages)) return false;
          tc_fence_after();
          qk(half, 0, st);
          mma_commit(&bar.k_empty[st]);
          ++kc;
          return true;
        };
        if (!next_qk(0)) return;
        if (n > 1 && !next_qk(1)) return;
        for (int i = 0; i < n; ++i) {
          const int half = i & 1;
          const uint32_t vs = vc % T::kStages;
          if (!wait1(bar.v_full[vs], vc / T::kStages)) return;
          if (!wait1(bar.p_full[half], pc[half]++)) return;
          tc_fence_after();
          pv(half, vs, i > 1);
          mma_commit(&bar.v_empty[vs]);
          ++vc;
          if (i + 2 < n && !next_qk(half)) return;
        }
      }
      if (!w.next(a)) return;
    }
  }

  // ---- warps 8-11
  // Codes of a tile as this thread loads them, and where.  K: a lane has 16
  // dimensions of a key, its warp 64 of them and 8 keys a turn.  V: a lane has
  // eight neighbouring keys by 16 dimensions (8 where D is 64).
  static constexpr int kTurns = D == 128 ? 8 : 4;
  static constexpr int kVWords = D == 128 ? 4 : 2;

  // A tile of the piece: its keys' pages (lane i: of the 16-key group i % 8).
  struct At {
    int tile, len, h, pages;
  };
  __device__ __forceinline__ At at_tile(const Way& w, int i) const {
    At t;
    t.tile = tile_at(w.t, i);
    t.len = w.s.len;
    t.h = w.h;
    t.pages = -1;
    const int key = t.tile * kTcKeys + 16 * (threadIdx.x & 7);
    if (key < t.len) {
      const int page = __ldg(a.b.table + w.b * a.b.width + (key >> a.c.page_shift));
      if (page < a.c.pages) t.pages = page;
    }
    return t;
  }
  // Row of codes (and scales) of a tile's key, -1 if it is none.
  __device__ __forceinline__ int64_t row_of(const At& t, int key) const {
    const int page = __shfl_sync(0xffffffffu, t.pages, key >> 4);
    const int pos = t.tile * kTcKeys + key;
    if (page < 0 || pos >= t.len) return -1;
    return ((static_cast<int64_t>(page) * a.c.heads + t.h) << a.c.page_shift) +
           (pos & ((1 << a.c.page_shift) - 1));
  }
  __device__ __forceinline__ void load_k(const At& t, uint4 (&c)[kTurns], float& ks, float& vs) const {
    const int cw = (threadIdx.x >> 5) - kConvWarp, lane = threadIdx.x & 31;
    const int d = (D == 128 ? 64 * (cw & 1) : 0) + 16 * (lane >> 3);
    const int key0 = (D == 128 ? 64 * (cw >> 1) : 32 * cw) + (lane & 7);
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
      const int64_t r = row_of(t, key0 + 8 * u);
      c[u] = r < 0 ? make_uint4(0, 0, 0, 0) : __ldg(reinterpret_cast<const uint4*>(a.c.k + r * D + d));
    }
    const int64_t r = row_of(t, 32 * cw + lane);
    ks = r < 0 ? 0.f : __ldg(a.c.k_scales + r);
    vs = r < 0 ? -1.f : __ldg(a.c.v_scales + r);
  }
  __device__ __forceinline__ void store_k(uint32_t st, const uint4 (&c)[kTurns]) const {
    const int cw = (threadIdx.x >> 5) - kConvWarp, lane = threadIdx.x & 31;
    const int key0 = (D == 128 ? 64 * (cw >> 1) : 32 * cw) + (lane & 7);
    const uint32_t to = k_at(st) + (D == 128 ? (cw & 1) * (kTcKeys * 128) : 0);
    const int ch = 2 * (lane >> 3);
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
      const int key = key0 + 8 * u;
      const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t o[4];
        if constexpr (BF16) {
          codes4_bf16<E4M3>(w[2 * e], o[0], o[1]);
          codes4_bf16<E4M3>(w[2 * e + 1], o[2], o[3]);
        } else {
          codes4_f16<E4M3>(w[2 * e], o[0], o[1]);
          codes4_f16<E4M3>(w[2 * e + 1], o[2], o[3]);
        }
        const uint32_t at = to + key * 128 + (((ch + e) ^ (key & 7)) << 4);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(o[0]), "r"(o[1]),
                     "r"(o[2]), "r"(o[3])
                     : "memory");
      }
    }
  }
  __device__ __forceinline__ void load_v(const At& t, uint32_t (&c)[8][kVWords]) const {
    const int cw = (threadIdx.x >> 5) - kConvWarp, lane = threadIdx.x & 31;
    const int key0 = 64 * (cw & 1) + 8 * (lane & 7);
    const int d = D / 2 * (cw >> 1) + 4 * kVWords * (lane >> 3);
    const int64_t r0 = row_of(t, key0);  // (eight keys lie in one page)
    const int valid = r0 < 0 ? 0 : t.len - (t.tile * kTcKeys + key0);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint8_t* const p = a.c.v + (r0 + u) * D + d;
      if constexpr (D == 128) {
        const uint4 x = u < valid ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
        c[u][0] = x.x, c[u][1] = x.y, c[u][2] = x.z, c[u][3] = x.w;
      } else {
        const uint2 x = u < valid ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0);
        c[u][0] = x.x, c[u][1] = x.y;
      }
    }
  }
  __device__ __forceinline__ void store_v(uint32_t st, const uint32_t (&c)[8][kVWords]) const {
    const int cw = (threadIdx.x >> 5) - kConvWarp, lane = threadIdx.x & 31;
    const int kg = lane & 7;
    const int d0 = D / 2 * (cw >> 1) + 4 * kVWords * (lane >> 3);
    const uint32_t to = v_at(st) + (cw & 1) * (D * 128);
#pragma unroll
    for (int q = 0; q < kVWords; ++q)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t o[2][4];
#pragma unroll
        for (int p = 0; p < 4; ++p)
          codes4_f16<E4M3>(prmt(c[2 * p][q], c[2 * p + 1][q], hf ? 0x7362 : 0x5140), o[0][p], o[1][p]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = d0 + 4 * q + 2 * hf + e;
          const uint32_t at = to + d * 128 + ((kg ^ (d & 7)) << 4);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(o[e][0]),
                       "r"(o[e][1]), "r"(o[e][2]), "r"(o[e][3])
                       : "memory");
        }
      }
  }
  __device__ __forceinline__ void done(uint64_t& b) const {
    fence_async_shared();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&b);
  }

  __device__ void convert() {
    const int tid = threadIdx.x - 32 * kConvWarp;
    // K runs a tile ahead of V
    Way w;
    w.start(a, piece);
    int i = w.from;
    uint32_t vc = 0;
    const float to_log2 = a.scale * 1.44269504f;
    uint4 ck[kTurns];
    uint32_t cv[8][kVWords];
    float ks, vs;
    At now = at_tile(w, i), before = now;
    load_k(now, ck, ks, vs);
    const uint32_t tiles = static_cast<uint32_t>(piece.end - piece.begin);
    for (uint32_t kc = 0; kc <= tiles; ++kc) {
      before = now;
      if (kc < tiles) {
        const uint32_t st = kc % T::kStages, slot = kc % T::kSlots;
        if (!wait(bar.k_empty[st], kc / T::kStages + 1)) return;
        store_k(st, ck);
        // (vs is -1 for a key that is none, NaN or not negative otherwise)
        const float safe = fmaxf(vs, kLeastScale);
        float* const f = factors(slot);
        const bool none = vs < 0.f;
        f[tid] = none ? 0.f : (ks + (vs - vs)) * to_log2;
        f[kTcKeys + tid] = none ? -INFINITY : lg2(safe);
        f[2 * kTcKeys + tid] = none ? 0.f : rcp(safe);
        done(bar.k_full[st]);
        if ((threadIdx.x & 31) == 0) mbar_arrive(&bar.f_full[slot]);
        if (kc + 1 < tiles) {
          if (++i >= w.to) {
            w.next(a);
            i = w.from;
          }
          now = at_tile(w, i);
          load_k(now, ck, ks, vs);
        }
      }
      if (kc > 0) {
        const uint32_t st = vc % T::kStages;
        if (!wait(bar.v_empty[st], vc / T::kStages + 1)) return;
        store_v(st, cv);
        done(bar.v_full[st]);
        ++vc;
      }
      if (kc < tiles) load_v(before, cv);
    }
  }

  // ---- warps 0-3 (half 0) and 4-7 (half 1)
  __device__ __forceinline__ void load_q(const Way& w, int half, int nr) const {
    const int group = a.heads / a.c.heads, r0 = w.rt * kTcRows + half * kHalf;
    constexpr int kChunks = D / 8;
    const int tid = threadIdx.x & 127;
#pragma unroll 4
    for (int u = 0; u < kChunks; ++u) {
      const int i = tid + 128 * u, r = i / kChunks, c = i % kChunks;
      uint32_t x[4] = {0, 0, 0, 0};
      if (half * kHalf + r < nr) {
        const int token = (r0 + r) / group, head = w.h * group + (r0 + r) % group;
        const uint16_t* q = static_cast<const uint16_t*>(a.q) +
                            (static_cast<int64_t>(w.s.row0) + token) * a.q_stride + head * D + 8 * c;
        if ((reinterpret_cast<uintptr_t>(q) & 15) == 0) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(q));
          x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x[k] = static_cast<uint32_t>(q[2 * k]) | static_cast<uint32_t>(q[2 * k + 1]) << 16;
        }
      }
      const uint32_t at = q_at(half) + (c >> 3) * (kHalf * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x[0]), "r"(x[1]),
                   "r"(x[2]), "r"(x[3])
                   : "memory");
    }
  }

  __device__ __forceinline__ void store_row(uint16_t* to, int d, const float* y) const {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (BF16) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(y[2 * k], y[2 * k + 1]);
        u[k] = *reinterpret_cast<const uint32_t*>(&p);
      } else {
        const __half2 p = __floats2half2_rn(y[2 * k], y[2 * k + 1]);
        u[k] = *reinterpret_cast<const uint32_t*>(&p);
      }
    }
    if ((reinterpret_cast<uintptr_t>(to) & 15) == 0) {
      *reinterpret_cast<uint4*>(to + d) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) to[d + k] = static_cast<uint16_t>(u[k >> 1] >> (16 * (k & 1)));
    }
  }

  __device__ void softmax() {
    const int half = threadIdx.x >> 7, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tid = threadIdx.x & 127;
    const int group = a.heads / a.c.heads;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes a warp, at bit 16
    const uint32_t s_at = tmem + lanes + T::kS + half * kTcKeys;
    const uint32_t o_at = tmem + lanes + T::kO + half * D;
    uint32_t sc = 0, first_tile = 0, meets = 0;  // S tiles of this half so far; tiles of the piece so far
    Way w;
    w.start(a, piece);
    for (;;) {
      const int nr = rows_of(w), n = w.to - w.from;
      const bool full = nr > kHalf;
      const Sequence s = w.s;
      if (full || half == 0) load_q(w, half, nr);
      done(bar.q_full);

      // this thread's row
      const int r = (full ? half * kHalf : 0) + tid;
      const int flat = w.rt * kTcRows + r;
      const bool mine = r < nr;
      const int token = mine ? flat / group : 0;
      int pos = s.prefix + token, hi = 0x7fffffff, lo = 0;
      const uint8_t* mask = nullptr;
      if (a.mask) {
        mask = a.mask + (static_cast<int64_t>(s.row0) + token) * a.mask_width;
        if (a.window > 0) {  // (else its place does not matter)
          const int t0 = __shfl_sync(0xffffffffu, token, 0);
          const int t1 = __reduce_max_sync(0xffffffffu, token);
          for (int t = t0; t <= t1; ++t) {
            const int p = draft_position(a, s, t);
            if (t == token) pos = p;
          }
        }
      }
      if (mine) {
        const Visible v = visible(pos, a.mask ? max(s.prefix, 0) : min(s.len, pos + 1), a.window, a.sinks);
        hi = v.hi;
        lo = v.lo;
      }
      const int hi_all = __reduce_min_sync(0xffffffffu, hi);
      const int lo_all = __reduce_max_sync(0xffffffffu, lo);

      float m = -INFINITY, l = 0.f;
      bool begun = false;
      for (int i = full ? 0 : half; i < n; i += full ? 1 : 2) {
        const int key0 = tile_at(w.t, w.from + i) * kTcKeys;
        const uint32_t fc = first_tile + i, slot = fc % T::kSlots;
        if (!wait(bar.s_full[half], sc)) return;
        if (!wait(bar.f_full[slot], fc / T::kSlots)) return;
        tc_fence_after();
        float x[kTcKeys];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_at + 32 * c, x + 32 * c);
        tmem_wait_ld();
        const float4* const f = reinterpret_cast<const float4*>(factors(slot));
#pragma unroll
        for (int c = 0; c < kTcKeys / 4; ++c) {
          const float4 k4 = f[c], v4 = f[kTcKeys / 4 + c];
          const float2 p = fma2(make_float2(x[4 * c], x[4 * c + 1]), make_float2(k4.x, k4.y),
                                make_float2(v4.x, v4.y));
          const float2 q = fma2(make_float2(x[4 * c + 2], x[4 * c + 3]), make_float2(k4.z, k4.w),
                                make_float2(v4.z, v4.w));
          x[4 * c] = p.x, x[4 * c + 1] = p.y, x[4 * c + 2] = q.x, x[4 * c + 3] = q.y;
        }
        const bool all = key0 + kTcKeys <= hi_all && (key0 >= lo_all || key0 + kTcKeys <= a.sinks);
        if (!all) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int at = key0 + 32 * c;
            uint32_t see = below(hi - at) & (~below(lo - at) | below(a.sinks - at));
            if (a.mask && at + 32 > s.prefix) {
              // the drafts among these keys, a token of the warp's rows at a time
              const int t0 = __shfl_sync(0xffffffffu, token, 0);
              const int t1 = __reduce_max_sync(0xffffffffu, token);
              const int j = at + lane - s.prefix;
              const bool in = j >= 0 && j < s.n && j < a.mask_width;
#pragma unroll 4
              for (int t = t0; t <= t1; ++t) {
                const bool bit = in && __ldg(a.mask + (static_cast<int64_t>(s.row0) + t) * a.mask_width + j) != 0;
                const uint32_t bits = __ballot_sync(0xffffffffu, bit);
                if (t == token) see |= bits;
              }
            }
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!(see >> k & 1)) x[32 * c + k] = -INFINITY;
          }
        }
        float top = -INFINITY, top2 = -INFINITY;
#pragma unroll
        for (int k = 0; k < kTcKeys; k += 4) {
          top = max3(top, x[k], x[k + 1]);
          top2 = max3(top2, x[k + 2], x[k + 3]);
        }
        top = fmaxf(top, top2);
        const bool grows = top > m + kSlack;
        if (__any_sync(0xffffffffu, grows)) {
          const float to = grows ? top : m;
          const float shrink = grows ? ex2(m - to) : 1.f;
          m = to;
          l *= shrink;
          if (begun) {
            // O holds the sums of the tiles before: the last of them is done
            if (!wait(bar.pv_done[half], sc - 1)) return;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t y[8], z[8];
              tmem_ld8(o_at + c, y);
              tmem_ld8(o_at + c + 8, z);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                y[k] = __float_as_uint(__uint_as_float(y[k]) * shrink);
                z[k] = __float_as_uint(__uint_as_float(z[k]) * shrink);
              }
              tmem_st8(o_at + c, y);
              tmem_st8(o_at + c + 8, z);
            }
            tmem_wait_st();
          }
        }
        begun = true;
        const float from = m == -INFINITY ? 0.f : -m;
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t p[32];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int e = 64 * c + 4 * k;
            const float4 v4 = f[2 * (kTcKeys / 4) + (e >> 2)];
            float2 u = add2(make_float2(x[e], x[e + 1]), make_float2(from, from));
            float2 v = add2(make_float2(x[e + 2], x[e + 3]), make_float2(from, from));
            u.x = ex2(u.x), u.y = ex2(u.y), v.x = ex2(v.x), v.y = ex2(v.y);
            sum = fma2(u, make_float2(v4.x, v4.y), sum);
            sum = fma2(v, make_float2(v4.z, v4.w), sum);
            const __half2 h0 = __floats2half2_rn(u.x, u.y), h1 = __floats2half2_rn(v.x, v.y);
            p[2 * k] = *reinterpret_cast<const uint32_t*>(&h0);
            p[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&h1);
          }
          tmem_st32(s_at + 32 * c, p);
        }
        l += sum.x + sum.y;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[half]);
        ++sc;
      }
      first_tile += n;
      if (begun) {
        if (!wait(bar.pv_done[half], sc - 1)) return;
        tc_fence_after();
      }
      if (!finish(w, full, half, r, mine, token, flat, begun, m, l, o_at, meets)) return;
      if (!w.next(a)) return;
    }
  }

  // The unit's sums: written out, or left for the kernel that adds them up.
  __device__ __forceinline__ bool finish(const Way& w, bool full, int half, int r, bool mine,
                                         int token, int flat, bool begun, float m, float l,
                                         uint32_t o_at, uint32_t& meets) const {
    const int tid = threadIdx.x & 127;
    const int group = a.heads / a.c.heads;
    const int64_t u0 = w.unit_begin();
    const int c0 = piece_of(piece.total, piece.pieces, u0);
    const int c1 = piece_of(piece.total, piece.pieces, u0 + w.t.count - 1);
    const bool whole = c0 == c1;
    float other_f = 0.f, mine_f = 1.f;
    float4* const scratch = reinterpret_cast<float4*>(smem);  // of the queries: [row][D / 4]
    if (!full) {
      // the second half's sums through the queries' shared memory: both halves'
      // products are done
      if (!meet(meets)) return false;
      if (half == 1) {
        if (begun) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float y[32];
            tmem_ld32(o_at + c, y);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 8; ++k)
              scratch[tid * (D / 4) + ((c / 4 + k) ^ (tid & 7))] =
                  make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
          }
        }
        join_m[tid] = begun ? m : -INFINITY;
        join_l[tid] = begun ? l : 0.f;
        tc_fence_before();
      }
      if (!meet(meets)) return false;
      if (half == 1) return meet(meets);  // (the first half has read it)
    }
    float om = -INFINITY, ol = 0.f;
    if (!full) {
      om = join_m[tid];
      ol = join_l[tid];
    }
    const bool two = !full && w.to - w.from > 1;
    const float top = fmaxf(m, om), from = top == -INFINITY ? 0.f : top;
    mine_f = ex2(m - from);
    other_f = ex2(om - from);
    const float sum_l = full ? l : l * mine_f + ol * other_f;
    const float inv = sum_l == 0.f ? 0.f : 1.f / sum_l;
    uint16_t* const to = static_cast<uint16_t*>(a.out) +
                         ((static_cast<int64_t>(w.s.row0) + token) * a.heads + w.h * group +
                          (mine ? flat % group : 0)) * D;
    float4* const part = reinterpret_cast<float4*>(
        partials + (2 * static_cast<int64_t>(blockIdx.x) + (static_cast<int>(blockIdx.x) == c0)) *
                       T::kSlot);
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float y[32];
      tmem_ld32(o_at + c, y);
      tmem_wait_ld();
      if (!full) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
          if (two) z = scratch[tid * (D / 4) + ((c / 4 + k) ^ (tid & 7))];
          y[4 * k] = fmaf(other_f, z.x, y[4 * k] * mine_f);
          y[4 * k + 1] = fmaf(other_f, z.y, y[4 * k + 1] * mine_f);
          y[4 * k + 2] = fmaf(other_f, z.z, y[4 * k + 2] * mine_f);
          y[4 * k + 3] = fmaf(other_f, z.w, y[4 * k + 3] * mine_f);
        }
      }
      if (mine) {
        if (whole) {
#pragma unroll
          for (int k = 0; k < 32; ++k) y[k] *= inv;
#pragma unroll
          for (int k = 0; k < 4; ++k) store_row(to, c + 8 * k, y + 8 * k);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            __stcg(part + (c / 4 + k) * kTcRows + r,
                   make_float4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]));
        }
      }
    }
    if (!whole && mine)
      __stcg(reinterpret_cast<float2*>(part + (D / 4) * kTcRows) + r,
             make_float2(full ? m : top, sum_l));
    if (!whole && static_cast<int>(blockIdx.x) == c0 && threadIdx.x == 0) {
      Cut cut;
      cut.b = w.b, cut.h = w.h, cut.rt = w.rt, cut.last_cta = c1;
      cuts[blockIdx.x] = cut;
    }
    tc_fence_before();
    return full || meet(meets);
  }
};

template <int D, bool E4M3, bool BF16>
__global__ void __launch_bounds__(kTcCta, 1) attn_tc_kernel(AttnArgs a, int least) {
  using T = Tc<D>;
  extern __shared__ uint8_t raw[];
  __shared__ Piece piece;
  __shared__ TcBarriers bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort;
  __shared__ float join_m[kHalf], join_l[kHalf];
  const int tid = threadIdx.x, warp = tid >> 5;
  Cut* const cuts = reinterpret_cast<Cut*>(a.partials);
  if (tid == 0) {
    Cut none;
    none.b = none.h = none.rt = 0;
    none.last_cta = -1;
    cuts[blockIdx.x] = none;
  }
  plan_piece<kTcRows, kTcKeys, kTcCta>(a, least, &piece);
  if (piece.begin == piece.end) return;
  uint8_t* const smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  if (tid == 0) {
    abort = 0;
    mbar_init(&bar.q_full, 8);
    mbar_init(&bar.join, 8);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.k_full[i], 4);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.v_full[i], 4);
      mbar_init(&bar.v_empty[i], 1);
    }
    for (int i = 0; i < 6; ++i) mbar_init(&bar.f_full[i], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_full[i], 4);
      mbar_init(&bar.pv_done[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == kIssueWarp) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  AttnTc<D, E4M3, BF16> r{a, piece, bar, smem, smem_addr(smem), tmem_slot, &abort, cuts,
                           a.partials + static_cast<int64_t>(gridDim.x) * kCutInts, join_m, join_l};
  if (warp < kConvWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    r.softmax();
  } else if (warp < kIssueWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    r.convert();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (tid == 32 * kIssueWarp) r.issue();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssueWarp) {
    tc_fence_after();
    tmem_dealloc(tmem_slot, 512);
  }
}

// Adds up the units that were cut between CTAs, in the order of the CTAs: a
// block takes a share of the rows of the unit that began in CTA blockIdx.x.
constexpr int kReduceThreads = 256, kReduceShare = 16;
template <int D>
__global__ void __launch_bounds__(kReduceThreads) attn_tc_reduce_kernel(AttnArgs a, int ctas) {
  const int c0 = blockIdx.x;
  const Cut cut = reinterpret_cast<const Cut*>(a.partials)[c0];
  if (cut.last_cta < 0) return;
  const float* const partials = a.partials + static_cast<int64_t>(ctas) * kCutInts;
  const Sequence s = sequence(a.c, a.b, cut.b);
  const int group = a.heads / a.c.heads;
  const int r0 = cut.rt * kTcRows, nr = min(kTcRows, s.n * group - r0);
  // a warp takes 32 rows of one chunk of four columns
  const int lane = threadIdx.x & 31;
  const int tasks = (nr + 31) / 32 * (D / 4);
  for (int i = blockIdx.y * (kReduceThreads / 32) + (threadIdx.x >> 5); i < tasks;
       i += kReduceShare * (kReduceThreads / 32)) {
    const int c = i % (D / 4), r = i / (D / 4) * 32 + lane;
    if (r >= nr) continue;
    float top = -INFINITY, sum_l = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAhead = 4;
    for (int k0 = c0; k0 <= cut.last_cta; k0 += kAhead) {
      float4 x[kAhead];
      float2 ml[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + k <= cut.last_cta) {
          const float4* const at = reinterpret_cast<const float4*>(
              partials + (2 * static_cast<int64_t>(k0 + k) + (k0 + k == c0)) * Tc<D>::kSlot);
          ml[k] = __ldcg(reinterpret_cast<const float2*>(at + (D / 4) * kTcRows) + r);
          x[k] = __ldcg(at + c * kTcRows + r);
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
    const float inv = sum_l == 0.f ? 0.f : 1.f / sum_l;
    const int token = (r0 + r) / group, head = cut.h * group + (r0 + r) % group;
    uint16_t* const to = static_cast<uint16_t*>(a.out) +
                         ((static_cast<int64_t>(s.row0) + token) * a.heads + head) * D + 4 * c;
    const float z[4] = {y.x * inv, y.y * inv, y.z * inv, y.w * inv};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      to[k] = a.bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(z[k]))
                     : __half_as_ushort(__float2half_rn(z[k]));
  }
}

template <int D, bool E4M3, bool BF16>
cudaError_t launch_tc_kernel(const AttnArgs& a, int sms, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<D, E4M3, BF16>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<D>::kSmem);
  if (e != cudaSuccess) return e;
  attn_tc_kernel<D, E4M3, BF16><<<sms, kTcCta, Tc<D>::kSmem, s>>>(a, 2);
  const cudaError_t l = cudaGetLastError();
  if (l != cudaSuccess) return l;
  attn_tc_reduce_kernel<D><<<dim3(sms, kReduceShare), kReduceThreads, 0, s>>>(a, sms);
  return cudaGetLastError();
}
template <int D>
cudaError_t launch_tc_dim(const AttnArgs& a, int sms, cudaStream_t s) {
  if (a.bf16)
    return a.c.e4m3 ? launch_tc_kernel<D, true, true>(a, sms, s)
                    : launch_tc_kernel<D, false, true>(a, sms, s);
  return a.c.e4m3 ? launch_tc_kernel<D, true, false>(a, sms, s)
                  : launch_tc_kernel<D, false, false>(a, sms, s);
}

}  // namespace

size_t attn_tc_partials(int sms, int dim) {
  return static_cast<size_t>(sms) * sizeof(Cut) +
         2 * static_cast<size_t>(sms) * kTcRows * (dim + 2) * sizeof(float);
}

cudaError_t launch_attn_tc(const AttnArgs& a, int sms, cudaStream_t s) {
  return a.c.dim == 128 ? launch_tc_dim<128>(a, sms, s) : launch_tc_dim<64>(a, sms, s);
}

}  // namespace w4
