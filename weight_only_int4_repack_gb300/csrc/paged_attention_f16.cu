// Paged attention, queries and outputs in f16.
#include "paged_attention.cuh"

namespace w4a16 {
namespace attn {

cudaError_t launch_f16(const Params &p, int sms, cudaStream_t s) {
    return p.c.type == W4A16_TYPE_E4M3 ? launch_dims<__half, E4M3>(p, sms, s) : launch_dims<__half, __half>(p, sms, s);
}

}  // namespace attn
}  // namespace w4a16
