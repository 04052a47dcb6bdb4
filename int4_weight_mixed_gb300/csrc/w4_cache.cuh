// w4_cache.cuh — device-side access to the paged key-value cache: which
// sequence a row belongs to, where a position lies, what a row sees.
#pragma once
#include <cuda_fp16.h>

#include "w4_internal.h"

namespace w4 {
namespace {

// Number of sequences that end at or before `row` (starts[b + 1] <= row): the
// row's sequence, or the count of sequences for a row behind the last one.
// All lanes of a warp; 32 probes a step, so 1024 sequences take two.  Ends
// whatever the array holds.
__device__ __forceinline__ int find_sequence(const BatchView& b, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = b.sequences;
  while (lo < hi) {
    const int step = (hi - lo + 31) >> 5;
    const int64_t j = lo + static_cast<int64_t>(lane) * step;
    const bool past = j < hi && __ldg(b.starts + j + 1) <= row;
    const int c = __popc(__ballot_sync(0xffffffffu, past));
    if (c == 0) return lo;
    const int last = lo + (c - 1) * step;
    lo = last + 1;
    hi = min(last + step, hi);
  }
  return lo;
}

// A sequence's rows and positions, whatever the arrays hold: its rows lie
// within the rows there are, its length within its line of the table.
struct Sequence {
  int row0;    // first row
  int n;       // rows
  int len;     // positions, the rows' own among them
  int prefix;  // position of row 0 (negative: its first rows have none)
};
__device__ __forceinline__ Sequence sequence(const CacheView& c, const BatchView& b, int i) {
  Sequence s;
  const int s0 = __ldg(b.starts + i), s1 = __ldg(b.starts + i + 1), len = __ldg(b.lens + i);
  s.row0 = min(max(s0, 0), b.rows);
  s.n = min(max(s1, s.row0), b.rows) - s.row0;
  s.len = static_cast<int>(min(static_cast<int64_t>(max(len, 0)), b.width << c.page_shift));
  s.prefix = s.len - s.n;
  return s;
}

// Index of (position, head 0) among all [pages][heads][page size] rows of
// codes, -1 where the table names no page.
__device__ __forceinline__ int64_t place(const CacheView& c, const BatchView& b, int seq, int pos) {
  const int page = __ldg(b.table + seq * b.width + (pos >> c.page_shift));
  if (page < 0 || page >= c.pages) return -1;
  return ((static_cast<int64_t>(page) * c.heads) << c.page_shift) +
         (pos & ((1 << c.page_shift) - 1));
}

// Two codes (the low two bytes of v) as fp16: both kinds are exact there.
template <bool E4M3>
__device__ __forceinline__ float2 codes2_f32(uint32_t v) {
  if constexpr (E4M3) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
  } else {
    return make_float2(static_cast<float>(static_cast<int8_t>(v & 0xff)),
                       static_cast<float>(static_cast<int8_t>(v >> 8 & 0xff)));
  }
}

// What the row at `pos` sees of the keys before `limit` (exclusive): those
// below `sinks` and those from `lo` on.
struct Visible {
  int lo, sinks, hi;
};
__device__ __forceinline__ Visible visible(int pos, int limit, int window, int sinks) {
  Visible v;
  v.hi = limit;
  v.lo = window > 0 ? max(0, pos - window + 1) : 0;
  v.sinks = window > 0 ? sinks : 0;
  return v;
}

// Position of row i of a tree of drafts: one step past the prefix for each
// draft that it sees but itself.  A row that sees none stands at the first.
// All lanes of a warp.
__device__ __forceinline__ int draft_position(const AttnArgs& a, const Sequence& s, int i) {
  const uint8_t* m = a.mask + (static_cast<int64_t>(s.row0) + i) * a.mask_width;
  const int n = static_cast<int>(min(static_cast<int64_t>(s.n), a.mask_width));
  int c = 0;
  for (int t = threadIdx.x & 31; t < n; t += 32) c += m[t] != 0;
  c = __reduce_add_sync(0xffffffffu, c);
  return s.prefix + max(c - 1, 0);
}

}  // namespace
}  // namespace w4
