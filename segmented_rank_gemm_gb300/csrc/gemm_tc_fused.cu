// gemm_tc_fused.cu -- the base GEMM's variants with bias, activation, factor and residual in the
// epilogue (include/lora_layer.h: lora_forward_fused), in a translation unit of their own.
#include "gemm_tc.cuh"

namespace lora {

cudaError_t launch_planned_fused(const GemmArgs& a, const GemmPlan& plan, const CUtensorMap& tmap_x,
                                 const CUtensorMap& tw, const CUtensorMap& tb, cudaStream_t stream) {
  return launch_planned<true>(a, plan, tmap_x, tw, tb, stream);
}

}  // namespace lora
