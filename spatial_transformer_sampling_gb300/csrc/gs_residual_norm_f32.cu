// gs_residual_norm_f32.cu -- norms around a gated branch, float.
#include "gs_residual_norm.cuh"

namespace gs {
GS_RESNORM_INST(float)
}  // namespace gs
