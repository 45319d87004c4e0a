// gs_attn_bf16.cu -- __nv_bfloat16 instantiations of the attention kernels (one
// translation unit per dtype so the build compiles them in parallel).
#include "gs_attn.cuh"

namespace gs {
template size_t attn_ws_bytes<__nv_bfloat16>(const AttnArgs &, bool);
template cudaError_t launch_attn<__nv_bfloat16>(const AttnArgs &, const AttnPtrs &, void *, cudaStream_t);
template cudaError_t launch_attn_backward<__nv_bfloat16>(const AttnArgs &, const AttnPtrs &, void *,
                                               cudaStream_t);
}  // namespace gs
