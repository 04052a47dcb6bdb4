// w4_tc_ep.cu — the tensor-core kernels of a product with an epilogue of its
// own (activation, gate, residual; see w4_epilogue.cuh), one CTA per tile;
// the CTA-pair variant is compiled in w4_tc_ep2.cu.
#include "w4_tc_kernel.cuh"

namespace w4 {

cudaError_t launch_tc_pair(const TcPlan& plan, const CUtensorMap& amap, const CUtensorMap& smap,
                           const CUtensorMap& zmap, const EpArgs& args, cudaStream_t s);

namespace {

constexpr int kRedWarps = 8;  // warps of a CTA
constexpr int kRedAhead = 8;  // slots whose loads are in flight together

// Split tiles: the sum of their contributors' partial sums, in K order (the
// plain product's), and the epilogue.  A warp has a block of eight rows by 32
// columns, laid out as the main kernel's drain leaves it (CTA pairs: the LEAN
// one's).  The plain product's
// kernels let the last contributor of a tile add the others', slot by slot;
// here the whole GPU does, eight slots in flight a warp, and the main kernel is
// rid of that code, whose registers its main loop spilled (M=64 4096 x 14336
// bf16 g128 with a residual 31.4 -> 25.2 us, M=100 1024 x 8192 int8 on 128-row
// tiles 52 -> 17, M=64 28672 x 4096 48.0 -> 45.9).  Bound by latency: a launch
// and one or two rounds of loads from L2.
template <int MODE, bool PAIR>
__global__ void __launch_bounds__(32 * kRedWarps)
    tc_reduce_kernel(const TcPlan p, const EpArgs args) {
  constexpr int NCTA = PAIR ? 2 : 1;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const int blocks = NCTA * p.nt * (p.bm / 8) * 4;  // of a tile
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kRedWarps + warp;
  if (item >= static_cast<int64_t>(p.tiles) * blocks) return;
  Work w;
  w.kb = p.kb_total;
  w.T = static_cast<int64_t>(p.tiles) * p.kb_total;
  w.G = p.grid / NCTA;
  Unit u;
  u.tile = static_cast<int>(div_nn(item, blocks));
  u.cfirst = 0;
  u.nslots = p.ksplit;
  if (p.decomp != kSplitK) {
    u.cfirst = static_cast<int>(sk_owner(u.tile * w.kb, w.T, w.G));
    u.nslots = static_cast<int>(sk_owner((u.tile + 1) * w.kb - 1, w.T, w.G)) - u.cfirst + 1;
  }
  if (u.nslots == 1) return;  // the main kernel stored it
  int b = static_cast<int>(item - static_cast<int64_t>(u.tile) * blocks);
  const int q = b & 3, nblk = p.bm / 8;
  b >>= 2;
  const int rank = b / (p.nt * nblk);
  b -= rank * p.nt * nblk;
  const int t = b / nblk, cc = (b - t * nblk) * 8;
  int mt, nt;
  tile_coords(p, u.tile, mt, nt);
  const int64_t m0 = static_cast<int64_t>(mt) * p.bm + cc;
  const int64_t n0 =
      ((static_cast<int64_t>(nt) * NCTA + rank) * p.nt + t) * kTileN + q * 32;
  if (m0 >= args.M || n0 >= args.N) return;
  const size_t slot_elems = static_cast<size_t>(p.nt) * kTileN * p.bm;
  const size_t off = PAIR ? static_cast<size_t>(b) * 1024 + q * 256 + lane * 4
                          : static_cast<size_t>(t * p.bm + cc) * kTileN + (q * 32 + lane) * 8;
  // lane l: the slot of contributor s0 + l of the 32 from s0 on
  auto slot_of = [&](int sl) {
    return sl < u.nslots ? (slot_index(p, w, u, sl) * NCTA + rank) * slot_elems : 0;
  };
  size_t held = slot_of(lane);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the main kernel is complete
  const uint4 side = ep_side8<MODE>(args, m0, n0);
  const uint32_t* part = static_cast<const uint32_t*>(args.partials) + off;
  uint32_t d[8];
  for (int s0 = 0; s0 < u.nslots; s0 += kRedAhead) {
    if (s0 != 0 && s0 % 32 == 0) held = slot_of(s0 + lane);
    uint32_t x[kRedAhead][8];
#pragma unroll
    for (int j = 0; j < kRedAhead; ++j) {
      const size_t at = static_cast<size_t>(__shfl_sync(
          0xffffffffu, static_cast<unsigned long long>(held), (s0 + j) & 31));
      if (s0 + j < u.nslots) {
        if (PAIR) ld_cg_halves(part + at, 128, x[j]);
        else ld_cg_v8(part + at, x[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < kRedAhead; ++j) {
      if (s0 + j >= u.nslots) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (s0 + j == 0) d[i] = x[j][i];
        else if (MODE == kW4A8) d[i] += x[j][i];
        else d[i] = __float_as_uint(__fadd_rn(__uint_as_float(d[i]), __uint_as_float(x[j][i])));
      }
    }
  }
  store_block8<MODE>(args, m0, n0, d, side);
}

template <int MODE>
cudaError_t launch_reduce(const TcPlan& plan, const EpArgs& args, cudaStream_t s) {
  const int64_t items =
      static_cast<int64_t>(plan.tiles) * (plan.pair ? 2 : 1) * plan.nt * (plan.bm / 8) * 4;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((items + kRedWarps - 1) / kRedWarps));
  cfg.blockDim = dim3(32 * kRedWarps);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (!plan.pair) return cudaLaunchKernelEx(&cfg, &tc_reduce_kernel<MODE, false>, plan, args);
  return cudaLaunchKernelEx(&cfg, &tc_reduce_kernel<MODE, true>, plan, args);
}

}  // namespace

cudaError_t launch_tc(const TcPlan& plan, const CUtensorMap& amap, const CUtensorMap& smap,
                      const CUtensorMap& zmap, const EpArgs& given, cudaStream_t s) {
  EpArgs args = given;
  args.reduce = tc_reduces(plan);
  const cudaError_t e = plan.pair ? launch_tc_pair(plan, amap, smap, zmap, args, s)
                        : tc_mma2(plan) ? launch_tc_t<true, false>(plan, amap, smap, zmap, args, s)
                                        : launch_tc_t<false, false>(plan, amap, smap, zmap, args, s);
  if (e != cudaSuccess || !args.reduce) return e;
  switch (plan.mode) {
    case kW4A16_F16: return launch_reduce<kW4A16_F16>(plan, args, s);
    case kW4A16_BF16: return launch_reduce<kW4A16_BF16>(plan, args, s);
    case kW4A8F8: return launch_reduce<kW4A8F8>(plan, args, s);
    default: return launch_reduce<kW4A8>(plan, args, s);
  }
}

}  // namespace w4
