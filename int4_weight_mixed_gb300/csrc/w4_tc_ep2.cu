// w4_tc_ep2.cu — the CTA-pair tensor-core kernels of a product with an
// epilogue of its own (see w4_tc3.cu and w4_epilogue.cuh).
#include "w4_tc_kernel.cuh"

namespace w4 {

cudaError_t launch_tc_pair(const TcPlan& plan, const CUtensorMap& amap, const CUtensorMap& smap,
                           const CUtensorMap& zmap, const EpArgs& args, cudaStream_t s) {
  if (plan.nt != 1) return cudaErrorInvalidValue;
  return launch_tc_t<true, true>(plan, amap, smap, zmap, args, s);
}

}  // namespace w4
