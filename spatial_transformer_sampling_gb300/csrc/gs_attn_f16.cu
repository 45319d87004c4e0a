// gs_attn_f16.cu -- __half instantiations of the attention kernels (one
// translation unit per dtype so the build compiles them in parallel).
#include "gs_attn.cuh"

namespace gs {
template size_t attn_ws_bytes<__half>(const AttnArgs &, bool);
template cudaError_t launch_attn<__half>(const AttnArgs &, const AttnPtrs &, void *, cudaStream_t);
template cudaError_t launch_attn_backward<__half>(const AttnArgs &, const AttnPtrs &, void *,
                                               cudaStream_t);
}  // namespace gs
