// gemm_tc_gelu.cu -- the base GEMM's variants with an epilogue (include/lora_layer.h:
// lora_forward_fused) of this activation.
#include "gemm_tc.cuh"

namespace lora {

LORA_FUSED_VARIANTS(LORA_ACT_GELU)

}  // namespace lora
