// w4_attn_plan.cuh — how the attention kernels share out their work, decided on
// the device from the batch's arrays alone, so that no length is read by the
// host and a captured graph follows them.
//
// A unit is a tile of RT rows (a row: one query head of one token; the heads of
// a key head are neighbouring rows, so that they share its keys) of one
// sequence and key head.  It visits tiles of TK keys: those that any of its
// rows may see.  All units' tiles, in order, are one line, cut into equal
// pieces, one for each CTA: a long sequence is spread over many CTAs, many
// short ones are shared out evenly.  A unit cut between CTAs is added up from
// partial sums in the order of its CTAs.
#pragma once
#include "w4_cache.cuh"
#include "w4_ptx.cuh"

namespace w4 {
namespace {

// The key tiles of a unit: the first `ns`, then t0, t0 + 1, ...; `count` in all
// (one at least: a unit that sees nothing still writes its rows).
struct Tiles {
  int ns, t0, count;
};
template <int RT, int TK>
__device__ __forceinline__ Tiles unit_tiles(const AttnArgs& a, const Sequence& s, int group, int rt) {
  Tiles t;
  const int first = rt * RT / group;
  const int last = min(s.n - 1, (rt * RT + RT - 1) / group);
  const int hi = a.mask ? s.len : min(s.len, s.prefix + last + 1);
  t.ns = t.t0 = 0;
  t.count = 1;
  if (hi <= 0) return t;
  const int lo = a.window > 0 ? max(0, (a.mask ? s.prefix : s.prefix + first) - a.window + 1) : 0;
  t.t0 = lo / TK;
  t.ns = min((min(a.sinks, lo) + TK - 1) / TK, t.t0);
  t.count = t.ns + (hi + TK - 1) / TK - t.t0;
  return t;
}
__device__ __forceinline__ int tile_at(const Tiles& t, int i) { return i < t.ns ? i : t.t0 + i - t.ns; }

template <int RT>
__device__ __forceinline__ int row_tiles(const Sequence& s, int group) {
  return (s.n * group + RT - 1) / RT;
}

// Tiles of a sequence under one key head.
template <int RT, int TK>
__device__ __forceinline__ int64_t head_tiles(const AttnArgs& a, const Sequence& s, int group) {
  int64_t n = 0;
  const int nrt = row_tiles<RT>(s, group);
  for (int rt = 0; rt < nrt; ++rt) n += unit_tiles<RT, TK>(a, s, group, rt).count;
  return n;
}

// Where a CTA's piece begins and how long it is.
struct Piece {
  int64_t total;  // tiles of all units
  int64_t begin, end;
  int pieces;     // CTAs that have one
  int b, h, rt;   // the unit that `begin` lies in
  int at;         // tiles of it before `begin`
  Sequence s;     // its sequence
};

__device__ __forceinline__ int64_t piece_begin(int64_t total, int pieces, int i) {
  return div_nn(total * i, pieces);
}
// The piece that tile x of the line lies in.
__device__ __forceinline__ int piece_of(int64_t total, int pieces, int64_t x) {
  return static_cast<int>(div_nn((x + 1) * pieces - 1, total));
}

// Filled in by all NT threads of the CTA (shared memory, and a barrier at the
// end).  least: tiles a piece has at least while there are fewer than that for
// every CTA.
template <int RT, int TK, int NT>
__device__ __forceinline__ void plan_piece(const AttnArgs& a, int least, Piece* p) {
  constexpr int W = NT / 32;
  __shared__ int64_t sums[W];
  __shared__ int64_t whole;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = a.heads / a.c.heads, B = a.b.sequences;
  int64_t mine = 0;
  Sequence s;
  const auto cost = [&](int i) -> int64_t {
    s = sequence(a.c, a.b, i);
    return head_tiles<RT, TK>(a, s, group);
  };
  for (int i = tid; i < B; i += NT) mine += cost(i);
  int64_t all = mine;
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  if (lane == 0) sums[warp] = all;
  __syncthreads();
  if (tid == 0) {
    all = 0;
    for (int i = 0; i < W; ++i) all += sums[i];
    all *= a.c.heads;
    whole = all;
    p->total = all;
    const int64_t most = div_nn(all + least - 1, least);
    p->pieces = most < gridDim.x ? static_cast<int>(most) : static_cast<int>(gridDim.x);
    const int c = blockIdx.x;
    p->begin = p->end = 0;
    if (c < p->pieces) {
      p->begin = piece_begin(all, p->pieces, c);
      p->end = piece_begin(all, p->pieces, c + 1);
    }
  }
  __syncthreads();
  if (p->begin == p->end) return;
  // the sequence that `begin` lies in: running sums over the sequences
  const int64_t begin = p->begin;
  int64_t run = 0;
  for (int base = 0; base < B; base += NT) {
    const int i = base + tid;
    const int64_t per_head = B <= NT ? mine : i < B ? cost(i) : 0;  // (s stays the one of i)
    const int64_t w = per_head * a.c.heads;
    int64_t to = w;  // inclusive sum
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, to, o);
      if (lane >= o) to += up;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = to;
    __syncthreads();
    int64_t before = run;
    for (int k = 0; k < W; ++k) {
      if (k < warp) before += sums[k];
      run += sums[k];
    }
    to += before;
    if (w > 0 && begin >= to - w && begin < to) {
      int64_t off = begin - (to - w);
      p->b = i;
      p->h = static_cast<int>(div_nn(off, per_head));
      off -= p->h * per_head;
      p->s = s;
      int rt = 0;
      for (;; ++rt) {
        const int n = unit_tiles<RT, TK>(a, s, group, rt).count;
        if (off < n) break;
        off -= n;
      }
      p->rt = rt;
      p->at = static_cast<int>(off);
    }
  }
  __syncthreads();
}

// A CTA's walk over the units of its piece; every thread walks by itself.
template <int RT, int TK>
struct Walk {
  int64_t x, end;  // next tile of the line, end of the piece
  int b, h, rt;
  Sequence s;
  Tiles t;
  int from, to;    // the piece's tiles of this unit

  __device__ __forceinline__ void start(const AttnArgs& a, const Piece& p) {
    x = p.begin;
    end = p.end;
    b = p.b;
    h = p.h;
    rt = p.rt;
    s = p.s;
    t = unit_tiles<RT, TK>(a, s, a.heads / a.c.heads, rt);
    from = p.at;
    clip();
  }
  __device__ __forceinline__ void clip() {
    to = static_cast<int>(min(static_cast<int64_t>(t.count), from + (end - x)));
  }
  // The line's tile where this unit begins.
  __device__ __forceinline__ int64_t unit_begin() const { return x - from; }
  // On to the next unit; false at the end of the piece.
  __device__ __forceinline__ bool next(const AttnArgs& a) {
    x += to - from;
    if (x >= end) return false;
    const int group = a.heads / a.c.heads;
    if (++rt >= row_tiles<RT>(s, group)) {
      rt = 0;
      if (++h >= a.c.heads) {
        h = 0;
        do {
          s = sequence(a.c, a.b, ++b);
        } while (s.n == 0 && b + 1 < a.b.sequences);
      }
    }
    t = unit_tiles<RT, TK>(a, s, group, rt);
    from = 0;
    clip();
    return true;
  }
};

}  // namespace
}  // namespace w4
