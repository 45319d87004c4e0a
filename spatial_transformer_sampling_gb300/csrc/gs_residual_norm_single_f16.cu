// The residual norm's gradient by single elements (fp16).
#include "gs_residual_norm.cuh"

namespace gs {
GS_RESNORM_BACKWARD(__half, 1)
}
