// The residual norm's gradient by pairs of elements (bf16).
#include "gs_residual_norm.cuh"

namespace gs {
GS_RESNORM_BACKWARD(__nv_bfloat16, 2)
}
