// Paged attention for sums, queries in fp16.
#include "paged_attention.cuh"

namespace w4a16 {
namespace attn {

cudaError_t launch_sums_f16(const Params &p, int sms, cudaStream_t s) {
    return launch_caches<true, __half>(p, sms, s);
}

}  // namespace attn
}  // namespace w4a16
