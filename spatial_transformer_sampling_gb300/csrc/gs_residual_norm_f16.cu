// gs_residual_norm_f16.cu -- norms around a gated branch, __half.
#include "gs_residual_norm.cuh"

namespace gs {
GS_RESNORM_INST(__half)
}  // namespace gs
