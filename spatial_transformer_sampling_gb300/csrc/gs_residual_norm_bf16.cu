// gs_residual_norm_bf16.cu -- norms around a gated branch, __nv_bfloat16.
#include "gs_residual_norm.cuh"

namespace gs {
GS_RESNORM_INST(__nv_bfloat16)
}  // namespace gs
