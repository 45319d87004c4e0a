// The residual norm's gradient by pairs of elements (fp32).
#include "gs_residual_norm.cuh"

namespace gs {
GS_RESNORM_BACKWARD(float, 2)
}
