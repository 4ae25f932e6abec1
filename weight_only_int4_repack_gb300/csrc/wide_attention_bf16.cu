// Attention of many rows, queries and outputs in bf16.
#include "wide_attention.cuh"

namespace w4a16 {
namespace wide {

cudaError_t launch_bf16(Which which, const Params &p, cudaStream_t s) {
    return p.c.type == W4A16_TYPE_E4M3 ? launch_dims<__nv_bfloat16, E4M3>(which, p, s) : launch_dims<__nv_bfloat16, __nv_bfloat16>(which, p, s);
}

}  // namespace wide
}  // namespace w4a16
