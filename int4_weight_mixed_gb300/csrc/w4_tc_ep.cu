// w4_tc_ep.cu — the tensor-core kernels of a product with an epilogue of its
// own (activation, gate, residual; see w4_epilogue.cuh), one CTA per tile;
// the CTA-pair variant is compiled in w4_tc_ep2.cu.
#include "w4_tc_kernel.cuh"

namespace w4 {

cudaError_t launch_tc_pair(const TcPlan& plan, const CUtensorMap& amap, const CUtensorMap& smap,
                           const CUtensorMap& zmap, const EpArgs& args, cudaStream_t s);

cudaError_t launch_tc(const TcPlan& plan, const CUtensorMap& amap, const CUtensorMap& smap,
                      const CUtensorMap& zmap, const EpArgs& args, cudaStream_t s) {
  if (plan.pair) return launch_tc_pair(plan, amap, smap, zmap, args, s);
  if (!tc_mma2(plan)) return launch_tc_t<false, false>(plan, amap, smap, zmap, args, s);
  return launch_tc_t<true, false>(plan, amap, smap, zmap, args, s);
}

}  // namespace w4
