// Internal declarations of the operators between the projections (and what the entry
// points of all share). Not installed; the public interface is include/w4a16.h.
#pragma once

#include "w4a16_internal.h"

namespace w4a16 {

// Device address of the error word on the current device (nullptr: no device).
unsigned int *device_error_ptr();
// Whether calls are launched as programmatic dependents (w4a16_set_launch_overlap).
bool launch_overlap();

// Whether an operator between the projections is launched as a programmatic dependent
// of the work before it. These kernels wait for that work before they touch memory, so
// all that overlaps is the launch: about 2 us less between two calls on a stream (a
// decoding step of four layers of width 5120, call by call: 369 us against 396). In a
// graph, where launches cost less, the same edges made the step slower (324 us against
// 320), so captured calls have them with w4a16_set_launch_overlap(1) only.
bool as_dependent(cudaStream_t s);

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }
inline w4a16_status from_cuda(cudaError_t e) { return e == cudaSuccess ? W4A16_OK : W4A16_ERR_CUDA; }

// What w4a16_kv_cache promises (include/w4a16.h), checked on the host.
w4a16_status check_cache(const w4a16_kv_cache *c);

}  // namespace w4a16
