// gs_gated_bf16.cu -- the gated projections of a feed-forward block, __nv_bfloat16.
#include "gs_gated_launch.cuh"

namespace gs {
GS_GATED_INST(__nv_bfloat16)
}  // namespace gs
