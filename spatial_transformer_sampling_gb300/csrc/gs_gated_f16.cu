// gs_gated_f16.cu -- the gated projections of a feed-forward block, __half.
#include "gs_gated_launch.cuh"

namespace gs {
GS_GATED_INST(__half)
}  // namespace gs
