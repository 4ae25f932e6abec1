// Paged attention for sums, queries in bf16.
#include "paged_attention.cuh"

namespace w4a16 {
namespace attn {

cudaError_t launch_sums_bf16(const Params &p, int sms, cudaStream_t s) {
    return launch_caches<true, __nv_bfloat16>(p, sms, s);
}

}  // namespace attn
}  // namespace w4a16
