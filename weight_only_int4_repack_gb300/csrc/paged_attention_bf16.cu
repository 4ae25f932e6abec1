// Paged attention, queries and outputs in bf16.
#include "paged_attention.cuh"

namespace w4a16 {
namespace attn {

cudaError_t launch_bf16(const Params &p, int sms, cudaStream_t s) {
    return p.c.type == W4A16_TYPE_E4M3 ? launch_dims<__nv_bfloat16, E4M3>(p, sms, s) : launch_dims<__nv_bfloat16, __nv_bfloat16>(p, sms, s);
}

}  // namespace attn
}  // namespace w4a16
