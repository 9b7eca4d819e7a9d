// gemm_tc_none.cu -- the base GEMM's variants with an epilogue (include/lora_layer.h:
// lora_forward_fused) without an activation.
#include "gemm_tc.cuh"

namespace lora {

LORA_FUSED_VARIANTS(LORA_ACT_NONE)

}  // namespace lora
