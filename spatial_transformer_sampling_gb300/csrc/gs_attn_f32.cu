// gs_attn_f32.cu -- float instantiations of the attention kernels (one
// translation unit per dtype so the build compiles them in parallel).
#include "gs_attn.cuh"

namespace gs {
template size_t attn_ws_bytes<float>(const AttnArgs &, bool);
template cudaError_t launch_attn<float>(const AttnArgs &, const AttnPtrs &, void *, cudaStream_t);
template cudaError_t launch_attn_backward<float>(const AttnArgs &, const AttnPtrs &, void *,
                                               cudaStream_t);
}  // namespace gs
