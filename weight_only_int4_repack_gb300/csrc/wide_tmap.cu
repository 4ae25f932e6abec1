// Tensor maps of queries and of a cache's pages for the attention of many rows, made by each call.
#include <cudaTypedefs.h>

#include <array>
#include <cstring>

#include "wide_attention.cuh"

namespace w4a16 {
namespace wide {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr) : nullptr;
    }();
    return fn;
}

}  // namespace

// Boxes of 64 elements x box[1] x box[2] x box[3] of a tensor of 16-bit elements whose innermost dimension is contiguous,
// 128-byte swizzle. Strides in elements; that of a dimension of one entry says nothing.
bool tensor_map(CUtensorMap *out, const void *base, const std::array<long long, 4> &dims, const std::array<long long, 3> &strides,
                const std::array<int, 4> &box) {
    const auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t d[4], s[3];
    cuuint32_t b[4], each[4] = {1, 1, 1, 1};
    for (int i = 0; i < 4; ++i) {
        if (dims[i] <= 0 || box[i] <= 0 || box[i] > 256) return false;
        d[i] = (cuuint64_t)dims[i], b[i] = (cuuint32_t)box[i];
    }
    for (int i = 0; i < 3; ++i) s[i] = dims[i + 1] > 1 ? (cuuint64_t)strides[i] * 2 : 16;
    for (int i = 0; i < 3; ++i)
        if (s[i] == 0 || s[i] % 16) return false;
    std::memset(out, 0, sizeof(*out));
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT16, 4, const_cast<void *>(base), d, s, b, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace wide
}  // namespace w4a16
