// w4_attn_tc.cu — attention over the paged key-value cache for many rows a key
// head (prompts, chunks, trees of drafts): on the tensor cores (tcgen05), bound
// by them and, short of that, by the instructions of the softmax.  A causal prompt
// of 8192, 32 heads over 8 of 128 dimensions: 744 us, 739 TFLOP/s.
//
// A unit is up to 256 rows (query heads of a key head times tokens) by the tiles
// of 128 keys they see.  Per tile and 128 rows X:
//
//   S_X = Q_X K^T         K: codes as 16-bit values, exact (bf16: times 2^-8, which ks
//                         takes back); S in tensor memory
//   t_j = S_j * (scale * log2 e * ks_j) + log2 vs_j       (ks, vs: the scales)
//   P_j = 2^(t_j - m + 6) <= 2^15, fp16, written over S in tensor memory
//   O_X += P V            V: codes as fp16, exact;  l += P_j 2^-4 / vs_j;  out = 2^-4 O / l
//                         (64 keys at a time: the first half's product runs while
//                         the second half's P is made)
//
// as in w4_attn_dec.cu: both scales enter the exponent, so that no code is
// rounded and P is rounded relative to what it weighs.  Keys that are none
// (behind the end, of no page) have log2 vs = kNoKey and codes of zero.
//
// Twenty warps (three of them idle), one CTA an SM (where the keys and values were
// unpacked, ten: one that copies tiles stands for the converters):
//   warps 0-3, 4-7   the softmax of rows 0-127 and 128-255; they also load Q (of the
//                    next unit, while the last tile's products run), rescale O
//                    when m moves, and write the result
//   warps 8-15       load codes (a tile ahead, in registers) and write them as
//                    16-bit values in the MMA's layout: K rows by key, V
//                    transposed (rows by dimension, bytes of key pairs put
//                    together by PRMT); they also make the scales' factors
//   warp 16          issues the MMAs.  While the softmax works on one half, the
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
constexpr int kTcCta = 640;
constexpr int kConvWarp = 8, kConvWarps = 8, kIssueWarp = 16;
// registers a thread after the split: 2 * 128 + 2 * 72 + 80 = 480 = 5 * 96 launched
constexpr int kTcRegs = 96, kSoftRegs = 128, kConvRegs = 72, kIssueRegs = 80;
static_assert(2 * kSoftRegs + 2 * kConvRegs + kIssueRegs <= 5 * kTcRegs, "register split");
// a warp's 32 rows by 32 columns of the result on their way out: 64 bytes a row,
// rows 80 bytes apart (16-byte accesses of eight rows hit different banks)
constexpr int kOutRow = 80, kOutBytes = 32 * kOutRow;
// log2 vs is kept with this added (t and m, too): its negative is the exponent of what
// l adds, which stays in range for all vs, from 2^-100 (l) to 2^121 (normal numbers).
constexpr int kLogLift = 4;
constexpr float kUnlift = 1.f / (1 << kLogLift);

// Where codes become 16-bit values: by the CTA's own converter warps, tile by tile
// (kOwn), or once for all units by attn_unpack_kernel, whose tiles a warp copies
// (kTiles).  kUnpack: that kernel's use of the converters' code.
enum Source { kOwn = 0, kTiles = 1, kUnpack = 2 };
__host__ __device__ constexpr int tc_threads(int source) { return source == kTiles ? 320 : kTcCta; }

template <int D>
struct Tc {
  static constexpr int kStages = D == 128 ? 2 : 4;    // of K and of V
  // of the scales' factors: a slot is written again two tiles after the stage's
  // last use, when the softmax has read it
  static constexpr int kSlots = kStages + 2;
  static constexpr int kQ = kHalf * D * 2;            // bytes of a half's queries
  static constexpr int kTileBytes = kTcKeys * D * 2;  // of a stage of K or V
  // for a pair of keys ks', ks', log2 vs + 4, log2 vs + 4
  static constexpr int kFactors = 2 * kTcKeys * 4;
  static constexpr int kFactorsAt = 2 * kQ + 2 * kStages * kTileBytes;
  static constexpr int kOutAt = kFactorsAt + kSlots * kFactors;
  static constexpr int kBytes = kOutAt + 8 * kOutBytes;
  static constexpr int kSmem = kBytes + 1024;         // (for the alignment of the first)
  // an unpacked tile in the workspace: K and V as in a stage, the factors
  static constexpr int kRecord = 2 * kTileBytes + kFactors;
  // tensor memory columns: S (P in its first half) of both halves, then O
  static constexpr int kS = 0, kO = 2 * kTcKeys;
  // partial sums of a piece, in floats: [D / 4][rows] of 16 bytes, [rows] of (m, l)
  static constexpr int64_t kSlot = static_cast<int64_t>(kTcRows) * (D + 2);
};

struct TcBarriers {
  uint64_t q_full, join, fin, k_full[4], k_empty[4], v_full[4], v_empty[4], f_full[6], s_full[2], p_half[2],
      p_full[2], pv_half[2], pv_done[2];
};

// What the roles share, at an address known when compiled (no register holds one).
struct TcShared {
  TcBarriers bar;
  Piece piece;
  uint32_t tmem;
  int abort, never;  // (never: 0, for waits that go on after an abort)
  float join_m[kHalf], join_l[kHalf];
  // of each half's rows: they see keys below x; those from y on, and the sinks
  int2 sees[2][kTcRows];
  // a walk for each warp (registers are scarce): lane 0 moves it on; and the softmax
  // warps' next unit
  Walk<kTcRows, kTcKeys> ways[kIssueWarp + 1], next[kConvWarp];
};
__device__ __forceinline__ TcShared& tc_shared() {
  __shared__ __align__(16) char bytes[sizeof(TcShared)];
  return *reinterpret_cast<TcShared*>(bytes);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// D[128 x N] (+)= A[128 x 16] B[16 x N] with A in shared or tensor memory, B in
// shared; descriptors as their low words and the high word all share.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint32_t a, uint32_t b, uint32_t hi,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts32(uint32_t d_tmem, uint32_t a_tmem, uint32_t b, uint32_t hi,
                                         uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__host__ __device__ constexpr uint32_t idesc_f16_c(uint32_t ab_format, uint32_t n) {
  return (1u << 4) | (ab_format << 7) | (ab_format << 10) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}
// 32 lanes x 4 columns, a lane a row.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, float* v, int step) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) v[step * i] = __uint_as_float(r[i]);
}

// 16 lanes x 32 columns, as an MMA's accumulator lies in registers: lane 4 g + t of
// the warp has columns 8 n + 2 t, + 1 of rows g (v[4 n], v[4 n + 1]) and g + 8.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const float (&v)[16]) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// 16 lanes x 16 columns of packed pairs: lane 4 g + t has column 4 n + t of rows g
// (v[2 n]) and g + 8 (v[2 n + 1]).
__device__ __forceinline__ void tmem_st_pairs(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}
__device__ __forceinline__ void tmem_ld_pairs(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x128b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7])
      : "r"(taddr)
      : "memory");
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
template <int D, bool E4M3, bool BF16, int SOURCE>
struct AttnTc {
  using T = Tc<D>;
  const AttnArgs& a;
  uint32_t base;  // shared address of the tiles
  uint32_t tmem;
  uint8_t* record = nullptr;  // kUnpack: the tile's place in the workspace

  using Way = Walk<kTcRows, kTcKeys>;
  static __device__ __forceinline__ void sts4(uint32_t at, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
  }
  static __device__ __forceinline__ TcShared& sh() { return tc_shared(); }
  static __device__ __forceinline__ Way& way() { return sh().ways[threadIdx.x >> 5]; }
  static __device__ __forceinline__ Way& way_next() { return sh().next[threadIdx.x >> 5]; }
  __device__ __forceinline__ void start() const {
    if ((threadIdx.x & 31) == 0) way().start(a, sh().piece);
    __syncwarp();
  }
  // The unit after this one, in w_next; false if there is none.  (A shuffle orders no
  // memory: the lanes meet before they read what lane 0 wrote, here and in next().)
  __device__ __forceinline__ bool look_ahead() const {
    int more = 0;
    if ((threadIdx.x & 31) == 0) {
      way_next() = way();
      more = way_next().next(a);
    }
    __syncwarp();
    return __shfl_sync(0xffffffffu, more, 0) != 0;
  }
  // This warp's share of a unit's Q is in shared memory.
  __device__ __forceinline__ void q_loaded() const {
    asm volatile("cp.async.wait_all;" ::: "memory");
    done(sh().bar.q_full);
  }
  __device__ __forceinline__ bool next() const {
    __syncwarp();
    int more = 0;
    if ((threadIdx.x & 31) == 0) more = way().next(a);
    __syncwarp();
    return __shfl_sync(0xffffffffu, more, 0) != 0;
  }

  __device__ __forceinline__ uint32_t q_at(int half) const { return base + half * T::kQ; }
  __device__ __forceinline__ uint32_t k_at(int st) const { return base + 2 * T::kQ + st * T::kTileBytes; }
  __device__ __forceinline__ uint32_t v_at(int st) const {
    return base + 2 * T::kQ + (T::kStages + st) * T::kTileBytes;
  }
  __device__ __forceinline__ uint32_t factors(int slot) const {
    return base + T::kFactorsAt + slot * T::kFactors;
  }
  // A whole warp: it goes on or gives up as one.
  __device__ __forceinline__ bool wait(uint64_t& b, uint32_t parity) const {
    return __all_sync(0xffffffffu, mbar_wait(&b, parity & 1, &sh().abort, a.status));
  }
  // What is still in flight when a role ends (it gave up, then): its last phase of b,
  // waited for whoever gave up, so that no copy or product outlives the CTA's memory.
  __device__ __forceinline__ void settle(uint64_t& b, uint32_t parity) const {
    mbar_wait(&b, parity & 1, &sh().never, a.status);
  }
  // Both halves of the softmax meet (bounded, like every wait here).
  __device__ __forceinline__ bool meet(uint32_t& meets) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sh().bar.join);
    return wait(sh().bar.join, meets++);
  }
  __device__ __forceinline__ int rows_of(const Way& w) const {
    return min(kTcRows, w.s.n * (a.heads / a.c.heads) - w.rt * kTcRows);
  }

  // ---- warp 16.  The whole warp walks and waits; one elected lane issues.
  __device__ __forceinline__ void qk(int half, int q, uint32_t st, uint32_t lo, uint32_t hi) const {
    constexpr uint32_t kId = idesc_f16_c(BF16 ? 1u : 0u, kTcKeys);
    if (elect_one()) {
      const uint32_t qd = lo + q * (T::kQ >> 4), kd = lo + ((2 * T::kQ + st * T::kTileBytes) >> 4);
      const uint32_t d = tmem + T::kS + half * kTcKeys;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const uint32_t off = (i >> 2) * (kHalf * 128 >> 4) + 2 * (i & 3);
        mma_ss(d, qd + off, kd + off, hi, kId, i != 0);
      }
      mma_commit(&sh().bar.s_full[half]);
    }
    __syncwarp();
  }
  // The first (second) 64 keys' part of the product with V.
  __device__ __forceinline__ void pv(int half, int part, uint32_t st, bool add, uint32_t lo,
                                     uint32_t hi) const {
    constexpr uint32_t kId = idesc_f16_c(0u, D);
    if (elect_one()) {
      const uint32_t vd = lo + ((2 * T::kQ + (T::kStages + st) * T::kTileBytes + part * D * 128) >> 4);
      const uint32_t d = tmem + T::kO + half * D, p = tmem + T::kS + half * kTcKeys + 32 * part;
#pragma unroll
      for (int i = 0; i < kTcKeys / 32; ++i) mma_ts32(d, p + 8 * i, vd + 2 * i, hi, kId, i != 0 || add);
      mma_commit(part ? &sh().bar.pv_done[half] : &sh().bar.pv_half[half]);
    }
    __syncwarp();
  }
  __device__ __forceinline__ bool pv_parts(int half, uint32_t& count, uint32_t st, bool add, uint32_t lo,
                                           uint32_t hi) const {
    if (!wait(sh().bar.p_half[half], count)) return false;
    tc_fence_after();
    pv(half, 0, st, add, lo, hi);
    if (!wait(sh().bar.p_full[half], count++)) return false;
    tc_fence_after();
    pv(half, 1, st, true, lo, hi);
    return true;
  }
  __device__ __forceinline__ void commit(uint64_t& b) const {
    if (elect_one()) mma_commit(&b);
    __syncwarp();
  }

  __device__ void issue() const {
    issue_units();
    commit(sh().bar.fin);  // of all products
    settle(sh().bar.fin, 0);
    __syncwarp();
  }
  __device__ __forceinline__ void issue_units() const {
    Way& w = way();
    uint32_t units = 0, kc = 0, vc = 0, pc0 = 0, pc1 = 0;
    start();
    // descriptors differ in the low word (the address) alone
    const uint32_t hi = static_cast<uint32_t>(sw128_kmajor_desc(0) >> 32);
    const uint32_t lo = static_cast<uint32_t>(sw128_kmajor_desc(0)) | base >> 4;
    for (;;) {
      const int n = w.to - w.from;
      if (!wait(sh().bar.q_full, units++)) return;
      if (rows_of(w) > kHalf) {
        uint32_t st = kc % T::kStages;
        if (!wait(sh().bar.k_full[st], kc / T::kStages)) return;
        fence_async_shared();
        tc_fence_after();
        qk(0, 0, st, lo, hi);
        qk(1, 1, st, lo, hi);
        commit(sh().bar.k_empty[st]);
        ++kc;
        for (int i = 0; i < n; ++i) {
          const uint32_t vs = vc % T::kStages;
          st = kc % T::kStages;
          if (!wait(sh().bar.v_full[vs], vc / T::kStages)) return;
          fence_async_shared();
          if (!pv_parts(0, pc0, vs, i > 0, lo, hi)) return;
          if (i + 1 < n) {
            if (!wait(sh().bar.k_full[st], kc / T::kStages)) return;
            fence_async_shared();
            tc_fence_after();
            qk(0, 0, st, lo, hi);
          }
          if (!pv_parts(1, pc1, vs, i > 0, lo, hi)) return;
          commit(sh().bar.v_empty[vs]);
          ++vc;
          if (i + 1 < n) {
            qk(1, 1, st, lo, hi);
            commit(sh().bar.k_empty[st]);
            ++kc;
          }
        }
      } else {
        // even tiles through the first half, odd ones through the second
        for (int i = -2; i < n; ++i) {
          const bool odd = i & 1;
          if (i >= 0) {
            const uint32_t vs = vc % T::kStages;
            if (!wait(sh().bar.v_full[vs], vc / T::kStages)) return;
            fence_async_shared();
            if (!(odd ? pv_parts(1, pc1, vs, i > 1, lo, hi) : pv_parts(0, pc0, vs, i > 1, lo, hi))) return;
            commit(sh().bar.v_empty[vs]);
            ++vc;
          }
          if (i + 2 < n) {
            const uint32_t st = kc % T::kStages;
            if (!wait(sh().bar.k_full[st], kc / T::kStages)) return;
            fence_async_shared();
            tc_fence_after();
            qk(odd, 0, st, lo, hi);
            commit(sh().bar.k_empty[st]);
            ++kc;
          }
        }
      }
      if (!next()) return;
    }
  }

  // ---- warps 8-15
  // Codes of a tile as this thread loads them, and where.  A warp has 16 keys, and
  // each of its loads whole rows of them: parts of 128-byte lines cost as much as
  // lines (16 KB in 1014 cycles by halves, 225 whole).  K: a lane has 16 dimensions
  // of a key.  V: a lane has eight neighbouring keys by kW dimensions (lane c of a
  // row's 16: kW c ..), and dimension kW c + e is row c + 16 e of the MMA's V, so that
  // the lanes of a store hit different banks; O's columns lie in that order.
  // The loads are volatile so that they stay where they are written, a tile ahead of
  // their use.  Keys that are none load row 0 instead, and their codes are set to
  // zero where they are used.
  static constexpr int kTurns = D / 32;   // of four (eight) keys
  static constexpr int kW = D / 16, kVWords = kW / 4;
  static __device__ __forceinline__ void load16(const void* p, uint32_t (&v)[4]) {
    asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "l"(p));
  }
  static __device__ __forceinline__ void load8(const void* p, uint32_t& v0, uint32_t& v1) {
    asm volatile("ld.global.nc.v2.b32 {%0, %1}, [%2];" : "=r"(v0), "=r"(v1) : "l"(p));
  }
  static __device__ __forceinline__ uint32_t load4(const void* p) {
    uint32_t v;
    asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
  }
  static __device__ __forceinline__ int conv_warp() {
    return (threadIdx.x >> 5) - (SOURCE == kUnpack ? 0 : kConvWarp);
  }
  // 16 bytes of a stage (of an unpacked tile) at offset `at` from base.
  __device__ __forceinline__ void put(uint32_t at, const uint32_t (&o)[4]) const {
    if constexpr (SOURCE == kUnpack)
      *reinterpret_cast<uint4*>(record + at) = make_uint4(o[0], o[1], o[2], o[3]);
    else
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(o[0]), "r"(o[1]),
                   "r"(o[2]), "r"(o[3])
                   : "memory");
  }
  __device__ __forceinline__ void put_factors(uint32_t to, int key, bool none, float ks, float vs) const {
    const uint32_t f = to + 16 * (key >> 1) + 4 * (key & 1);
    const float x = none ? 0.f : (ks + (vs - vs)) * (a.scale * (BF16 ? 1.44269504f / kBf16Code : 1.44269504f));
    const float y = none ? kNoKey : lg2(counted(vs)) + kLogLift;
    if constexpr (SOURCE == kUnpack) {
      *reinterpret_cast<float*>(record + f) = x;
      *reinterpret_cast<float*>(record + f + 8) = y;
    } else {
      sts4(f, x);
      sts4(f + 8, y);
    }
  }
  // This lane's key of turn u, and its first dimension.
  static __device__ __forceinline__ int k_key(int u) {
    return 16 * conv_warp() + 512 / D * u + ((threadIdx.x & 31) * 16 / D);
  }
  static __device__ __forceinline__ int k_dim() { return (threadIdx.x & (D / 16 - 1)) * 16; }

  // A tile of the piece, and the pages of its unit's tiles 4 q .. 4 q + 3 (q = i / 4):
  // lane l has that of 16-key group l % 8 of tile 4 q + l / 8.
  struct At {
    int tile, len, h, i, pages;
  };
  __device__ __forceinline__ int pages_at(int q) const {
    const Way& w = way();
    const int lane = threadIdx.x & 31, i = 4 * q + (lane >> 3);
    const int key = tile_at(w.t, i) * kTcKeys + 16 * (lane & 7);
    const bool in = i < w.t.count && key < w.s.len;
    const int page = static_cast<int>(
        load4(in ? a.b.table + w.b * a.b.width + (key >> a.c.page_shift) : a.b.lens));
    return in ? page : -1;
  }
  // Row of codes (and scales) of a tile's key, -1 if it is none.
  __device__ __forceinline__ int64_t row_of(const At& t, int key) const {
    const int page = __shfl_sync(0xffffffffu, t.pages, 8 * (t.i & 3) + (key >> 4));
    const int pos = t.tile * kTcKeys + key;
    if (page < 0 || page >= a.c.pages || pos >= t.len) return -1;
    return ((static_cast<int64_t>(page) * a.c.heads + t.h) << a.c.page_shift) +
           (pos & ((1 << a.c.page_shift) - 1));
  }
  // Bits of `in`: the turns' keys, and (bit 8) the key of the scales.
  __device__ __forceinline__ void load_k(const At& t, uint32_t (&c)[kTurns][4], float& ks, float& vs,
                                         uint32_t& in) const {
    in = 0;
    const int64_t r0 = row_of(t, 16 * conv_warp());  // (16 neighbouring keys lie in one page)
    const int valid = r0 < 0 ? 0 : t.len - (t.tile * kTcKeys + 16 * conv_warp());
    const uint8_t* const p = a.c.k + (r0 < 0 ? 0 : r0) * D + k_dim();
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
      const int k = k_key(u) - 16 * conv_warp();
      load16(k < valid ? p + k * D : p, c[u]);
      in |= k < valid ? 1u << u : 0u;
    }
    const int64_t r = row_of(t, 32 * (conv_warp() & 3) + (threadIdx.x & 31));  // (a key a lane)
    ks = __uint_as_float(load4(a.c.k_scales + (r < 0 ? 0 : r)));
    vs = __uint_as_float(load4(a.c.v_scales + (r < 0 ? 0 : r)));
    in |= r >= 0 ? 256u : 0u;
  }
  // to: where the stage's K lies.
  __device__ __forceinline__ void store_k(uint32_t to, uint32_t (&c)[kTurns][4], uint32_t in) const {
    if ((in & ((1u << kTurns) - 1)) != (1u << kTurns) - 1) {
#pragma unroll
      for (int u = 0; u < kTurns; ++u)
        if (!(in >> u & 1)) c[u][0] = c[u][1] = c[u][2] = c[u][3] = 0;
    }
    // the lanes of the second 64 dimensions write their two chunks the other way
    // round: other banks than those of the first
    const int sub = k_dim() >> 6, ch = (k_dim() & 63) >> 3;
    to += sub * (kTcKeys * 128);
#pragma unroll
    for (int u = 0; u < kTurns; ++u) {
      const int key = k_key(u);
      uint32_t o[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (BF16) {
          codes4_bf16<E4M3>(c[u][2 * e], o[e][0], o[e][1]);
          codes4_bf16<E4M3>(c[u][2 * e + 1], o[e][2], o[e][3]);
        } else {
          codes4_f16<E4M3>(c[u][2 * e], o[e][0], o[e][1]);
          codes4_f16<E4M3>(c[u][2 * e + 1], o[e][2], o[e][3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t at = to + key * 128 + (((ch + (e ^ sub)) ^ (key & 7)) << 4);
        const uint32_t y[4] = {sub ? o[e ^ 1][0] : o[e][0], sub ? o[e ^ 1][1] : o[e][1],
                               sub ? o[e ^ 1][2] : o[e][2], sub ? o[e ^ 1][3] : o[e][3]};
        put(at, y);
      }
    }
  }
  // valid: of the eight keys, the first so many.
  __device__ __forceinline__ void load_v(const At& t, uint32_t (&c)[8][kVWords], int& valid) const {
    const int lane = threadIdx.x & 31, key0 = 16 * conv_warp() + 8 * (lane >> 4);
    const int64_t r0 = row_of(t, key0);
    valid = r0 < 0 ? 0 : min(t.len - (t.tile * kTcKeys + key0), 8);
    const uint8_t* const p = a.c.v + (r0 < 0 ? 0 : r0) * D + kW * (lane & 15);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint8_t* const q = u < valid ? p + u * D : p;
      if constexpr (D == 128) load8(q, c[u][0], c[u][1]);
      else c[u][0] = load4(q);
    }
  }
  __device__ __forceinline__ void store_v(uint32_t to, uint32_t (&c)[8][kVWords], int valid) const {
    if (valid < 8) {
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int q = 0; q < kVWords; ++q)
          if (u >= valid) c[u][q] = 0;
    }
    const int lane = threadIdx.x & 31, kg = 2 * conv_warp() + (lane >> 4);
    // (row c + 16 e: its low bits are c's)
    to += (kg >> 3) * (D * 128) + (lane & 15) * 128 + (((kg & 7) ^ (lane & 7)) << 4);
#pragma unroll
    for (int q = 0; q < kVWords; ++q)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t o[2][4];
#pragma unroll
        for (int p = 0; p < 4; ++p)
          codes4_f16<E4M3>(prmt(c[2 * p][q], c[2 * p + 1][q], hf ? 0x7362 : 0x5140), o[0][p], o[1][p]);
#pragma unroll
        for (int e = 0; e < 2; ++e) put(to + (4 * q + 2 * hf + e) * 2048, o[e]);
      }
  }
  // What this warp wrote is there.  The fence that lets the tensor cores see it is the
  // issuing warp's, after its wait: one warp's instead of eight.
  __device__ __forceinline__ void done(uint64_t& b) const {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&b);
  }

  __device__ void convert() const {
    Way& w = way();
    const int tid = threadIdx.x - 32 * kConvWarp;
    // Codes of K are loaded a tile before they are stored, pages before that; V
    // follows K by a tile.
    start();
    uint32_t ck[kTurns][4], cv[8][kVWords];
    float ks = 0.f, vs = 0.f;
    uint32_t in = 0;
    int valid = 0;
    int i = w.from;
    const uint32_t tiles = static_cast<uint32_t>(sh().piece.end - sh().piece.begin);
    int pages = pages_at(i >> 2);
    const auto here = [&]() {
      At t;
      t.tile = tile_at(w.t, i);
      t.len = w.s.len;
      t.h = w.h;
      t.i = i;
      t.pages = pages;
      return t;
    };
    const auto step = [&]() {  // on to the next tile
      if (++i >= w.to) {
        next();
        i = w.from;
        pages = pages_at(i >> 2);
      } else if ((i & 3) == 0) {
        pages = pages_at(i >> 2);
      }
    };
    At before, now = here();
    load_k(now, ck, ks, vs, in);
    if (tiles > 1) step();
    for (uint32_t kc = 0; kc <= tiles; ++kc) {
      before = now;
      if (kc < tiles) {
        const uint32_t st = kc % T::kStages, slot = kc % T::kSlots;
        if (!wait(sh().bar.k_empty[st], kc / T::kStages + 1)) return;
        store_k(k_at(st), ck, in);
        if (tid < kTcKeys) put_factors(factors(slot), tid, !(in & 256u), ks, vs);
        done(sh().bar.k_full[st]);
        if (tid < kTcKeys && (tid & 31) == 0) mbar_arrive(&sh().bar.f_full[slot]);
        if (kc + 1 < tiles) {
          now = here();
          load_k(now, ck, ks, vs, in);
          if (kc + 2 < tiles) step();
        }
      }
      if (kc > 0) {
        const uint32_t vc = kc - 1, st = vc % T::kStages;
        if (!wait(sh().bar.v_empty[st], vc / T::kStages + 1)) return;
        store_v(v_at(st), cv, valid);
        done(sh().bar.v_full[st]);
      }
      if (kc < tiles) load_v(before, cv, valid);
    }
  }

  // ---- kTiles: warp 8 copies the unpacked tiles instead
  __device__ void copy() const {
    uint32_t k = 0, v = 0;  // copied tiles of K (and factors), of V
    copy_tiles(k, v);
    for (uint32_t j = k > T::kStages ? k - T::kStages : 0; j < k; ++j)
      settle(sh().bar.k_full[j % T::kStages], j / T::kStages);
    for (uint32_t j = k > T::kSlots ? k - T::kSlots : 0; j < k; ++j)
      settle(sh().bar.f_full[j % T::kSlots], j / T::kSlots);
    for (uint32_t j = v > T::kStages ? v - T::kStages : 0; j < v; ++j)
      settle(sh().bar.v_full[j % T::kStages], j / T::kStages);
    __syncwarp();
  }
  __device__ __forceinline__ void copy_tiles(uint32_t& copied_k, uint32_t& copied_v) const {
    Way& w = way();
    start();
    const uint32_t tiles = static_cast<uint32_t>(sh().piece.end - sh().piece.begin);
    const uint8_t *now = nullptr, *before = nullptr;
    int i = w.from;
    for (uint32_t kc = 0; kc <= tiles; ++kc) {
      before = now;
      if (kc < tiles) {
        if (kc > 0 && ++i >= w.to) {
          next();
          i = w.from;
        }
        now = a.tiles + ((static_cast<int64_t>(w.b) * a.c.heads + w.h) * a.tiles_each +
                         tile_at(w.t, i)) * T::kRecord;
        const uint32_t st = kc % T::kStages, slot = kc % T::kSlots;
        if (!wait(sh().bar.k_empty[st], kc / T::kStages + 1)) return;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sh().bar.k_full[st], T::kTileBytes);
          bulk_g2s_a(k_at(st), now, T::kTileBytes, smem_addr(&sh().bar.k_full[st]));
          mbar_arrive_expect_tx(&sh().bar.f_full[slot], T::kFactors);
          bulk_g2s_a(factors(slot), now + 2 * T::kTileBytes, T::kFactors, smem_addr(&sh().bar.f_full[slot]));
        }
        __syncwarp();
        copied_k = kc + 1;
      }
      if (kc > 0) {
        const uint32_t vc = kc - 1, st = vc % T::kStages;
        if (!wait(sh().bar.v_empty[st], vc / T::kStages + 1)) return;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sh().bar.v_full[st], T::kTileBytes);
          bulk_g2s_a(v_at(st), before + T::kTileBytes, T::kTileBytes, smem_addr(&sh().bar.v_full[st]));
        }
        __syncwarp();
        copied_v = vc + 1;
      }
    }
  }

  // ---- kUnpack: the CTA's tile
  __device__ __forceinline__ void unpack(const Sequence& s, int b, int h, int tile) const {
    At t;
    t.tile = tile, t.len = s.len, t.h = h, t.i = 0, t.pages = -1;
    const int key = tile * kTcKeys + 16 * (threadIdx.x & 7);
    if (key < s.len) t.pages = __ldg(a.b.table + b * a.b.width + (key >> a.c.page_shift));
    uint32_t ck[kTurns][4], cv[8][kVWords], in;
    float ks, vs;
    int valid;
    load_k(t, ck, ks, vs, in);
    load_v(t, cv, valid);
    store_k(0, ck, in);
    if (threadIdx.x < kTcKeys) put_factors(2 * T::kTileBytes, threadIdx.x, !(in & 256u), ks, vs);
    store_v(T::kTileBytes, cv, valid);
  }

  // ---- warps 0-3 (half 0) and 4-7 (half 1)
  __device__ __forceinline__ void load_q(const Way& w, int half) const {
    const int nr = rows_of(w);
    const int group = a.heads / a.c.heads;
    constexpr int kChunks = D / 8;  // a thread: one chunk of every (128 / kChunks)-th row
    const int tid = threadIdx.x & 127, c = tid % kChunks;
    const int first = w.rt * kTcRows + half * kHalf;
    const int token0 = first / group, rest = first - token0 * group;
    // x / group by a product, exactly for x < 2^21 and group <= 2^16
    const float by = 1.f / static_cast<float>(group);
    const uint16_t* const q0 = static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(w.h) * group * D + 8 * c;
    const bool vec = ((reinterpret_cast<uintptr_t>(a.q) & 15) | (a.q_stride & 7)) == 0;
    const uint32_t to = q_at(half) + (c >> 3) * (kHalf * 128);
#pragma unroll
    for (int u = 0; u < kChunks; ++u) {
      const int r = tid / kChunks + 128 / kChunks * u;
      const bool in = half * kHalf + r < nr;
      const int x = rest + r, t = static_cast<int>((static_cast<float>(x) + 0.5f) * by);
      const uint16_t* const q = q0 + (static_cast<int64_t>(w.s.row0) + token0 + t) * a.q_stride +
                                static_cast<int64_t>(x - t * group) * D;
      const uint32_t at = to + r * 128 + (((c & 7) ^ (r & 7)) << 4);
      if (vec) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at),
                     "l"(in ? static_cast<const void*>(q) : a.q), "r"(in ? 16 : 0)
                     : "memory");
      } else {
        uint32_t y[4] = {0, 0, 0, 0};
        if (in) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            y[k] = static_cast<uint32_t>(q[2 * k]) | static_cast<uint32_t>(q[2 * k + 1]) << 16;
        }
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(y[0]), "r"(y[1]),
                     "r"(y[2]), "r"(y[3])
                     : "memory");
      }
    }
  }

  // Dimensions c .. c + 31 of O, a row a lane: of the converters' order, kW c' + e at
  // column c' + 16 e.
  __device__ __forceinline__ void load_sums(uint32_t o_at, int c, float (&y)[32]) const {
#pragma unroll
    for (int k = 0; k < 32 / kW; k += 4)
#pragma unroll
      for (int e = 0; e < kW; ++e) tmem_ld4(o_at + c / kW + k + 16 * e, y + kW * k + e, kW);
    tmem_wait_ld();
  }
  // 32 columns (from column c on) of the warp's rows, a row a lane, to the result:
  // through shared memory, so that a store covers 64 bytes of eight rows.
  __device__ __forceinline__ void store_out(const float (&y)[32], uint16_t* to, bool mine, int c) const {
    const int lane = threadIdx.x & 31;
    const uint32_t at = base + T::kOutAt + (threadIdx.x >> 5) * kOutBytes;
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t u[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (BF16) {
          const __nv_bfloat162 p = __floats2bfloat162_rn(y[8 * q + 2 * k], y[8 * q + 2 * k + 1]);
          u[k] = *reinterpret_cast<const uint32_t*>(&p);
        } else {
          const __half2 p = __floats2half2_rn(y[8 * q + 2 * k], y[8 * q + 2 * k + 1]);
          u[k] = *reinterpret_cast<const uint32_t*>(&p);
        }
      }
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + lane * kOutRow + 16 * q),
                   "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3])
                   : "memory");
    }
    __syncwarp();
    const uint64_t row = mine ? reinterpret_cast<uint64_t>(to + c) : 0;
    const bool vec = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = 8 * q + (lane >> 2);
      uint32_t u[4];
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                   : "r"(at + r * kOutRow + 16 * (lane & 3))
                   : "memory");
      uint16_t* const p = reinterpret_cast<uint16_t*>(__shfl_sync(0xffffffffu, row, r));
      if (p == nullptr) continue;
      uint16_t* const dst = p + 8 * (lane & 3);
      if (vec) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) dst[k] = static_cast<uint16_t>(u[k >> 1] >> (16 * (k & 1)));
      }
    }
  }

  // A lane's four rows of the warp's 32: g, g + 8, g + 16, g + 24.
  static __device__ __forceinline__ int row_at(int k) { return 8 * k + ((threadIdx.x & 31) >> 2); }

  static __device__ __forceinline__ float4 lds4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
  }
  // O times shrink (a row's own); the products so far are done.
  __device__ __forceinline__ void rescale_sums(uint32_t o_at, const float (&shrink)[4]) const {
    tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float y[2][16];
      tmem_ld_frag(o_at + c, y[0]);
      tmem_ld_frag(o_at + c + (16u << 16), y[1]);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        y[0][e] *= shrink[e >> 1 & 1];
        y[1][e] *= shrink[2 + (e >> 1 & 1)];
      }
      tmem_st_frag(o_at + c, y[0]);
      tmem_st_frag(o_at + c + (16u << 16), y[1]);
    }
  }
  // The tile's probabilities of chunks begin .. end - 1 times shrink: exactly, it is a
  // power of two (but for those that fall below fp16's subnormals).
  __device__ __forceinline__ void rescale_tile(uint32_t s_at, int begin, int end,
                                               const float (&shrink)[4]) const {
    if (begin >= end) return;
    tmem_wait_st();
#pragma unroll 1
    for (int c = begin; c < end; ++c) {
      uint32_t p[2][8];
      tmem_ld_pairs(s_at + 16 * c, p[0]);
      tmem_ld_pairs(s_at + 16 * c + (16u << 16), p[1]);
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        uint32_t& v = p[e >> 3][e & 7];
        const float by = shrink[2 * (e >> 3) + (e & 1)];
        float2 y = __half22float2(*reinterpret_cast<const __half2*>(&v));
        const __half2 h = __floats2half2_rn(y.x * by, y.y * by);
        v = *reinterpret_cast<const uint32_t*>(&h);
      }
      tmem_st_pairs(s_at + 16 * c, p[0]);
      tmem_st_pairs(s_at + 16 * c + (16u << 16), p[1]);
    }
  }

  // Adds the drafts among keys at .. at + 31 that each row sees.
  __device__ __forceinline__ void drafts(int at, int first_row, uint32_t (&see)[4]) const {
    const Way& w = way();
    const int lane = threadIdx.x & 31;
    const int nr = rows_of(w);
    const int group = a.heads / a.c.heads;
    const int j = at + lane - w.s.prefix;
    const bool in = j >= 0 && j < w.s.n && j < a.mask_width;
    // the warp's rows' tokens
    const int last = min(first_row + 31, nr - 1);
    if (first_row > last) return;
    const int t0 = token_of(first_row), t1 = token_of(last);
#pragma unroll 2
    for (int t = t0; t <= t1; ++t) {
      const bool bit = in && __ldg(a.mask + (static_cast<int64_t>(w.s.row0) + t) * a.mask_width + j) != 0;
      const uint32_t bits = __ballot_sync(0xffffffffu, bit);
      // rows of this token: t * group <= flat < (t + 1) * group
      const int from = t * group - w.rt * kTcRows - first_row;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = row_at(k) - from;
        if (r >= 0 && r < group) see[k] |= bits;
      }
    }
  }
  // Token (row of the sequence) of the unit's row r.
  __device__ __forceinline__ int token_of(int r) const {
    return (way().rt * kTcRows + r) / (a.heads / a.c.heads);
  }

  __device__ void softmax() const {
    softmax_units();
    asm volatile("cp.async.wait_all;" ::: "memory");
    tmem_wait_st();
  }
  __device__ __forceinline__ void softmax_units() const {
    Way& w = way();
    const int half = threadIdx.x >> 7, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // 32 lanes a warp, at bit 16
    const uint32_t s_at = tmem + lanes + T::kS + half * kTcKeys;
    const uint32_t o_at = tmem + lanes + T::kO + half * D;
    uint32_t sc = 0, first_tile = 0, meets = 0;  // S tiles of this half so far; tiles of the piece
    start();
    if (half == 0 || rows_of(w) > kHalf) load_q(w, half);
    q_loaded();
    for (;;) {
      const int nr = rows_of(w), n = w.to - w.from;
      const bool full = nr > kHalf;
      const bool more = look_ahead();

      // what the warp's rows see, a row a lane (rows that are none: all)
      const int first_row = (full ? half * kHalf : 0) + 32 * (warp & 3);
      int2 own = make_int2(0x7fffffff, 0);  // keys below x, from y on
      {
        const int r = first_row + lane;
        const int token = r < nr ? token_of(r) : -1;
        int pos = w.s.prefix + token;
        if (a.mask && a.window > 0 && first_row < nr) {
          const int t1 = token_of(min(first_row + 31, nr - 1));
          for (int t = token_of(first_row); t <= t1; ++t) {
            const int at = draft_position(a, w.s, t);
            if (t == token) pos = at;
          }
        }
        if (r < nr) {
          const Visible v = visible(pos, a.mask ? max(w.s.prefix, 0) : min(w.s.len, pos + 1), a.window, a.sinks);
          own = make_int2(v.hi, v.lo);
        }
      }
      __syncwarp();
      sh().sees[half][first_row + lane] = own;
      __syncwarp();
      const int hi_all = __reduce_min_sync(0xffffffffu, own.x);
      const int lo_all = __reduce_max_sync(0xffffffffu, own.y);

      // m: whole numbers (the maximum rounded down: the largest p is 1 at least), so
      // that rescaling is exact; l: of even and odd keys
      float m[4];
      float2 l[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) m[k] = -INFINITY, l[k] = make_float2(0.f, 0.f);
      bool begun = false;
      for (int i = full ? 0 : half; i < n; i += full ? 1 : 2) {
        const int key0 = tile_at(w.t, w.from + i) * kTcKeys;
        const uint32_t fc = first_tile + i, slot = fc % T::kSlots;
        if (!wait(sh().bar.s_full[half], sc)) return;
        if (!wait(sh().bar.f_full[slot], fc / T::kSlots)) return;
        tc_fence_after();
        if (full && i + 1 == n) {
          // this half's last product with Q is done: the next unit's Q
          if (more && (half == 0 || rows_of(way_next()) > kHalf)) load_q(way_next(), half);
        }
        const bool all = key0 + kTcKeys <= hi_all && (key0 >= lo_all || key0 + kTcKeys <= a.sinks);
        uint32_t f = factors(slot) + 16 * (lane & 3);
        // 32 keys at a time (a loop: the code of all roles has to stay in the
        // instruction cache)
#pragma unroll 1
        for (int c = 0; c < 4; ++c, f += 256) {
          float x[2][16];
          tmem_ld_frag(s_at + 32 * c, x[0]);
          tmem_ld_frag(s_at + 32 * c + (16u << 16), x[1]);
          float4 u[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) u[q] = lds4(f + 64 * q);
          tmem_wait_ld();
          float top[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            top[k] = -INFINITY;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float *const e = &x[k >> 1][4 * q + 2 * (k & 1)];
              const float2 t = fma2(make_float2(e[0], e[1]), make_float2(u[q].x, u[q].y),
                                    make_float2(u[q].z, u[q].w));
              e[0] = t.x, e[1] = t.y;
            }
          }
          if (!all) {
            const int at = key0 + 32 * c;
            uint32_t see[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int2 v = sh().sees[half][first_row + row_at(k)];
              see[k] = below(v.x - at) & (~below(v.y - at) | below(a.sinks - at));
            }
            if (a.mask && at + 32 > w.s.prefix) drafts(at, first_row, see);
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint32_t bits = see[k] >> (8 * q + 2 * (lane & 3));
                if (!(bits & 1)) x[k >> 1][4 * q + 2 * (k & 1)] = -INFINITY;
                if (!(bits & 2)) x[k >> 1][4 * q + 2 * (k & 1) + 1] = -INFINITY;
              }
          }
          bool grows = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              top[k] = max3(top[k], x[k >> 1][4 * q + 2 * (k & 1)], x[k >> 1][4 * q + 2 * (k & 1) + 1]);
            grows |= top[k] > m[k] + (kSlack + 1.f) && top[k] > 0.5f * kNoKey;
          }
          if (__any_sync(0xffffffffu, grows)) {
            float shrink[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              top[k] = fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 1));
              top[k] = floorf(fmaxf(top[k], __shfl_xor_sync(0xffffffffu, top[k], 2)));
              const bool up = top[k] > m[k] + kSlack && top[k] > 0.5f * kNoKey;
              shrink[k] = up ? ex2(m[k] - top[k]) : 1.f;
              if (up) m[k] = top[k];
              l[k].x *= shrink[k];
              l[k].y *= shrink[k];
            }
            // O holds the sums of the tiles before and, from the third chunk on, of
            // this one's first half
            if (c >= 2) {
              if (!wait(sh().bar.pv_half[half], sc)) return;
              rescale_sums(o_at, shrink);
              rescale_tile(s_at, 2, c, shrink);
            } else {
              if (begun) {
                if (!wait(sh().bar.pv_done[half], sc - 1)) return;
                rescale_sums(o_at, shrink);
              }
              rescale_tile(s_at, 0, c, shrink);
            }
          }
          float2 neg[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float y = m[k] == -INFINITY ? 0.f : kTcLift - m[k];
            neg[k] = make_float2(y, y);
          }
          uint32_t p[2][8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 r = make_float2(ex2(fminf(-u[q].z, 126.f)), ex2(fminf(-u[q].w, 126.f)));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float *const e = &x[k >> 1][4 * q + 2 * (k & 1)];
              float2 t = add2(make_float2(e[0], e[1]), neg[k]);
              t.x = ex2(t.x);
              t.y = ex2(t.y);
              l[k] = fma2(t, r, l[k]);
              const __half2 h = __floats2half2_rn(t.x, t.y);
              p[k >> 1][2 * q + (k & 1)] = *reinterpret_cast<const uint32_t*>(&h);
            }
          }
          tmem_st_pairs(s_at + 16 * c, p[0]);
          tmem_st_pairs(s_at + 16 * c + (16u << 16), p[1]);
          if (c == 1) {
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh().bar.p_half[half]);
          }
        }
        begun = true;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh().bar.p_full[half]);
        ++sc;
      }
      first_tile += n;
      // (before the result is written, so that the next unit's first scores are
      // computed meanwhile; a unit of one half still needs Q's memory)
      if (more && full) q_loaded();
      if (begun) {
        if (!wait(sh().bar.pv_done[half], sc - 1)) return;
        tc_fence_after();
      }
      // a row a lane: row r of the warp's is row_at(r / 8) of lanes 4 (r % 8) ..
      float row_m = 0.f, row_l = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float sum = l[k].x + l[k].y;
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const float mk = __shfl_sync(0xffffffffu, m[k], 4 * (lane & 7));
        const float lk = __shfl_sync(0xffffffffu, sum, 4 * (lane & 7));
        if (lane >> 3 == k) row_m = mk, row_l = lk;
      }
      if (!finish(full, half, nr, begun, row_m, row_l, o_at, meets)) return;
      if (!full && more) {
        if (half == 0 || rows_of(way_next()) > kHalf) load_q(way_next(), half);
        q_loaded();
      }
      if (!more) return;
      __syncwarp();
      if (lane == 0) w = way_next();
      __syncwarp();
    }
  }

  // The unit's sums: written out, or left for the kernel that adds them up.
  __device__ __forceinline__ bool finish(bool full, int half, int nr, bool begun, float m, float l,
                                         uint32_t o_at, uint32_t& meets) const {
    const Way& w = way();
    const Piece& piece = sh().piece;
    const int tid = threadIdx.x & 127;
    const int group = a.heads / a.c.heads;
    const int r = (full ? half * kHalf : 0) + tid;  // this thread's row of the unit
    const bool mine = r < nr;
    const int flat = w.rt * kTcRows + (mine ? r : 0), token = flat / group;
    const int64_t u0 = w.unit_begin(), u1 = u0 + w.t.count;
    const bool begins = u0 >= piece.begin, whole = begins && u1 <= piece.end;
    float other_f = 0.f, mine_f = 1.f;
    // the queries' memory, as [row][D / 4] of 16 bytes
    const auto scratch = [&](int c) { return base + 16 * (tid * (D / 4) + (c ^ (tid & 7))); };
    if (!full) {
      // the second half's sums through the queries' shared memory: both halves'
      // products are done
      if (!meet(meets)) return false;
      if (half == 1) {
        if (begun) {
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float y[32];
            load_sums(o_at, c, y);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(scratch(c / 4 + k)),
                           "f"(y[4 * k]), "f"(y[4 * k + 1]), "f"(y[4 * k + 2]), "f"(y[4 * k + 3])
                           : "memory");
          }
        }
        sh().join_m[tid] = begun ? m : -INFINITY;
        sh().join_l[tid] = begun ? l : 0.f;
        tc_fence_before();
      }
      if (!meet(meets)) return false;
      if (half == 1) return meet(meets);  // (the first half has read it)
    }
    float om = -INFINITY, ol = 0.f;
    if (!full) {
      om = sh().join_m[tid];
      ol = sh().join_l[tid];
    }
    const bool two = !full && w.to - w.from > 1;
    const float top = fmaxf(m, om), from = top == -INFINITY ? 0.f : top;
    mine_f = ex2(m - from);
    other_f = ex2(om - from);
    const float sum_l = full ? l : l * mine_f + ol * other_f;
    const float inv = sum_l == 0.f ? 0.f : kUnlift / sum_l;
    uint16_t* const to = static_cast<uint16_t*>(a.out) +
                         ((static_cast<int64_t>(w.s.row0) + token) * a.heads + w.h * group +
                          flat - token * group) * D;
    float4* const part = reinterpret_cast<float4*>(
        a.partials + static_cast<int64_t>(gridDim.x) * kCutInts + (2 * static_cast<int64_t>(blockIdx.x) + begins) * T::kSlot);
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      float y[32];
      load_sums(o_at, c, y);
      if (!full) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
          if (two) z = lds4(scratch(c / 4 + k));
          y[4 * k] = fmaf(other_f, z.x, y[4 * k] * mine_f);
          y[4 * k + 1] = fmaf(other_f, z.y, y[4 * k + 1] * mine_f);
          y[4 * k + 2] = fmaf(other_f, z.z, y[4 * k + 2] * mine_f);
          y[4 * k + 3] = fmaf(other_f, z.w, y[4 * k + 3] * mine_f);
        }
      }
      if (whole) {
#pragma unroll
        for (int k = 0; k < 32; ++k) y[k] *= inv;
        store_out(y, to, mine, c);
      } else {
        if (mine) {
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
    if (!whole && begins && threadIdx.x == 0) {
      Cut cut;
      cut.b = w.b, cut.h = w.h, cut.rt = w.rt;
      cut.last_cta = piece_of(piece.total, piece.pieces, u1 - 1);
      reinterpret_cast<Cut*>(a.partials)[blockIdx.x] = cut;
    }
    tc_fence_before();
    return full || meet(meets);
  }
};

template <int D, bool E4M3, bool BF16, int SOURCE>
__global__ void __launch_bounds__(tc_threads(SOURCE), 1)
    attn_tc_kernel(const __grid_constant__ AttnArgs a, int least) {
  extern __shared__ uint8_t raw[];
  TcShared& sh = tc_shared();
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  if (tid == 0) {
    Cut none;
    none.b = none.h = none.rt = 0;
    none.last_cta = -1;
    reinterpret_cast<Cut*>(a.partials)[blockIdx.x] = none;
  }
  constexpr int kIssue = SOURCE == kTiles ? kConvWarp + 1 : kIssueWarp;
  plan_piece<kTcRows, kTcKeys, tc_threads(SOURCE)>(a, least, &sh.piece);
  if (sh.piece.begin == sh.piece.end) return;
  if (tid == 0) {
    sh.abort = sh.never = 0;
    TcBarriers& bar = sh.bar;
    mbar_init(&bar.q_full, kConvWarp);
    mbar_init(&bar.join, kConvWarp);
    mbar_init(&bar.fin, 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.k_full[i], SOURCE == kTiles ? 1 : kConvWarps);
      mbar_init(&bar.k_empty[i], 1);
      mbar_init(&bar.v_full[i], SOURCE == kTiles ? 1 : kConvWarps);
      mbar_init(&bar.v_empty[i], 1);
    }
    for (int i = 0; i < 6; ++i) mbar_init(&bar.f_full[i], SOURCE == kTiles ? 1 : 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.s_full[i], 1);
      mbar_init(&bar.p_half[i], 4);
      mbar_init(&bar.p_full[i], 4);
      mbar_init(&bar.pv_half[i], 1);
      mbar_init(&bar.pv_done[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == kIssue) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const AttnTc<D, E4M3, BF16, SOURCE> r{a, (smem_addr(raw) + 1023) & ~1023u, sh.tmem};
  if constexpr (SOURCE == kTiles) {  // (registers are plenty)
    if (warp < kConvWarp) r.softmax();
    else if (warp == kIssue) r.issue();
    else r.copy();
  } else if (warp < kConvWarp) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    r.softmax();
  } else if (warp < kIssueWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    r.convert();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == kIssueWarp) r.issue();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kIssue) {
    tc_fence_after();
    tmem_dealloc(sh.tmem, 512);
  }
}

// The visible tiles of all sequences as 16-bit values in the workspace, a CTA a tile:
// where many units share them, each would be converted many times over.
template <int D, bool E4M3, bool BF16>
__global__ void __launch_bounds__(32 * kConvWarps) attn_unpack_kernel(const __grid_constant__ AttnArgs a) {
  const int64_t line = blockIdx.x / a.tiles_each;
  const int tile = static_cast<int>(blockIdx.x - line * a.tiles_each);
  const int b = static_cast<int>(line / a.c.heads), h = static_cast<int>(line - static_cast<int64_t>(b) * a.c.heads);
  const Sequence s = sequence(a.c, a.b, b);
  if (s.n == 0 || (tile > 0 && tile * kTcKeys >= s.len)) return;
  const int lo = a.window > 0 ? max(0, s.prefix - a.window + 1) : 0;
  if ((tile + 1) * kTcKeys <= lo && tile * kTcKeys >= a.sinks) return;
  const AttnTc<D, E4M3, BF16, kUnpack> r{a, 0, 0,
                                         a.tiles + static_cast<int64_t>(blockIdx.x) * Tc<D>::kRecord};
  r.unpack(s, b, h, tile);
}

// Adds up the units that were cut between CTAs, in the order of the CTAs: a
// block takes a share of the rows of the unit that began in CTA blockIdx.x.
constexpr int kReduceThreads = 256;
template <int D>
__global__ void __launch_bounds__(kReduceThreads) attn_tc_reduce_kernel(AttnArgs a, int ctas) {
  const int c0 = blockIdx.x;
  const Cut cut = reinterpret_cast<const Cut*>(a.partials)[c0];
  if (cut.last_cta < 0) return;
  const float* const partials = a.partials + static_cast<int64_t>(ctas) * kCutInts;
  const Sequence s = sequence(a.c, a.b, cut.b);
  const int group = a.heads / a.c.heads;
  const int r0 = cut.rt * kTcRows, nr = min(kTcRows, s.n * group - r0);
  // 32 rows by 32 columns a block (few units cut many times still make many blocks): a
  // warp takes a chunk of four columns, a row a lane; then, through shared memory, 64
  // bytes of a row
  __shared__ uint2 out[32][9];
  __shared__ uint64_t to[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = 32 * blockIdx.y, r = first + lane, c = 8 * blockIdx.z + warp;
  if (first >= nr) return;
  if (warp == 0) {
    const int flat = r0 + min(r, nr - 1), token = flat / group;
    to[lane] = reinterpret_cast<uint64_t>(static_cast<uint16_t*>(a.out) +
                                          ((static_cast<int64_t>(s.row0) + token) * a.heads + cut.h * group +
                                           flat - token * group) * D + 32 * blockIdx.z);
  }
  if (r < nr) {
    float top = -INFINITY, sum_l = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kAhead = 8;
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
        const float up = fmaxf(top, ml[k].x);
        const float from = up == -INFINITY ? 0.f : up;
        const float f = ex2(top - from), fk = ex2(ml[k].x - from);
        top = up;
        sum_l = sum_l * f + fk * ml[k].y;
        y.x = y.x * f + fk * x[k].x;
        y.y = y.y * f + fk * x[k].y;
        y.z = y.z * f + fk * x[k].z;
        y.w = y.w * f + fk * x[k].w;
      }
    }
    const float inv = sum_l == 0.f ? 0.f : kUnlift / sum_l;
    uint2 u;
    if (a.bf16) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(y.x * inv, y.y * inv);
      const __nv_bfloat162 q = __floats2bfloat162_rn(y.z * inv, y.w * inv);
      u = make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
    } else {
      const __half2 p = __floats2half2_rn(y.x * inv, y.y * inv);
      const __half2 q = __floats2half2_rn(y.z * inv, y.w * inv);
      u = make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
    }
    out[lane][warp] = u;
  }
  __syncthreads();
  const bool vec = (reinterpret_cast<uintptr_t>(a.out) & 7) == 0;
  const int i = threadIdx.x >> 3, e = threadIdx.x & 7;
  if (first + i < nr) {
    const uint2 u = out[i][e];
    uint16_t* const p = reinterpret_cast<uint16_t*>(to[i]) + 4 * e;
    if (vec) {
      *reinterpret_cast<uint2*>(p) = u;
    } else {
      p[0] = static_cast<uint16_t>(u.x), p[1] = static_cast<uint16_t>(u.x >> 16);
      p[2] = static_cast<uint16_t>(u.y), p[3] = static_cast<uint16_t>(u.y >> 16);
    }
  }
}

template <int D, bool E4M3, bool BF16, int SOURCE>
cudaError_t launch_tc_source(const AttnArgs& a, int sms, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<D, E4M3, BF16, SOURCE>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<D>::kSmem);
  if (e != cudaSuccess) return e;
  attn_tc_kernel<D, E4M3, BF16, SOURCE><<<sms, tc_threads(SOURCE), Tc<D>::kSmem, s>>>(a, 2);
  return cudaGetLastError();
}
template <int D, bool E4M3, bool BF16>
cudaError_t launch_tc_kernel(const AttnArgs& a, int sms, cudaStream_t s) {
  cudaError_t e;
  if (a.tiles) {
    const int64_t ctas = static_cast<int64_t>(a.b.sequences) * a.c.heads * a.tiles_each;
    attn_unpack_kernel<D, E4M3, BF16><<<static_cast<unsigned>(ctas), 32 * kConvWarps, 0, s>>>(a);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = launch_tc_source<D, E4M3, BF16, kTiles>(a, sms, s);
  } else {
    e = launch_tc_source<D, E4M3, BF16, kOwn>(a, sms, s);
  }
  if (e != cudaSuccess) return e;
  attn_tc_reduce_kernel<D><<<dim3(sms, kTcRows / 32, D / 32), kReduceThreads, 0, s>>>(a, sms);
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

int64_t attn_tc_tile_bytes(int dim) { return dim == 128 ? Tc<128>::kRecord : Tc<64>::kRecord; }

cudaError_t launch_attn_tc(const AttnArgs& a, int sms, cudaStream_t s) {
  return a.c.dim == 128 ? launch_tc_dim<128>(a, sms, s) : launch_tc_dim<64>(a, sms, s);
}

}  // namespace w4
