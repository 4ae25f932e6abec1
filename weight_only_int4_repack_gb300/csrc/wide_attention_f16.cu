// Attention of many rows, queries and outputs in f16.
#include "wide_attention.cuh"

namespace w4a16 {
namespace wide {

cudaError_t launch_f16(Which which, const Params &p, cudaStream_t s) {
    return p.c.type == W4A16_TYPE_E4M3 ? launch_dims<__half, E4M3>(which, p, s) : launch_dims<__half, __half>(which, p, s);
}

}  // namespace wide
}  // namespace w4a16
