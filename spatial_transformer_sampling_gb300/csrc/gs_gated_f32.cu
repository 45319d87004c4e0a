// gs_gated_f32.cu -- the gated projections of a feed-forward block, float.
#include "gs_gated_launch.cuh"

namespace gs {
GS_GATED_INST(float)
}  // namespace gs
