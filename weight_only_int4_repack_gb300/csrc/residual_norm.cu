// Residual stream and norms between two blocks of a decoder layer:
//     t = [rms(y) * post_gamma | y] * [gate],  h' = h + alpha * t,  n = rms(h') * gamma
// with rms(x) = x / sqrt(mean x^2 + eps). Streaming work, bound by HBM: every
// element of h, y (and a full gate) is read once and every element of h' and n
// written once; the row between the passes stays in registers.
// Measured (GB300, in a CUDA graph): 8192 rows of 5120, bf16 with the stream in fp32,
// both norms and a gate (503 MB) 80.1 us, 6.3 TB/s, 94% of the copy rate; one row 2.2 us.
// Rows above 16384 wide with the stream in fp32 spill 68 bytes a thread.
#include <cmath>

#include "decode_ops.h"
#include "elem.cuh"
#include "ptx.cuh"

namespace w4a16 {
namespace {

struct NormParams {
    const void *h, *y, *post, *gate, *gamma;
    void *h_out, *n_out;
    long long h_row, y_row, gate_row, ho_row, no_row;
    int K;
    float alpha, eps;
    bool overlap;
};

constexpr int kMaxK = 32768;

// Sum over the CTA, the same in every thread and in the same order on every run.
__device__ __forceinline__ float cta_sum(float x, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = threadIdx.x % 32 < blockDim.x / 32 ? red[threadIdx.x % 32] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Eight elements as they are in memory.
template <typename T>
struct Raw {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); ++i) w[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void get(float (&f)[8]) const {
        elem::Vec<T, 8>::load(reinterpret_cast<const T *>(w), f);
    }
};

// One CTA per row; thread t holds the 8-element groups t, t + blockDim, ... All that
// the row needs from HBM is asked for before the first sum.
template <typename T, typename H, int V, int kMost>
__global__ void __launch_bounds__(kMost) residual_norm_kernel(const NormParams p) {
    using VT = elem::Vec<T, 8>;
    using VH = elem::Vec<H, 8>;
    __shared__ float red[2][32];
    if (p.overlap) ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const long long row = blockIdx.x;
    const int groups = p.K / 8, threads = blockDim.x;
    const T *y = static_cast<const T *>(p.y) + row * p.y_row;
    const H *h = static_cast<const H *>(p.h) + row * p.h_row;
    const T *gate = static_cast<const T *>(p.gate) + row * p.gate_row;
    Raw<T> ry[V], rg[V];
    Raw<H> rh[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int g = threadIdx.x + v * threads;
        if (g < groups) {
            ry[v].load(y + 8 * g);
            rh[v].load(h + 8 * g);
            if (p.gate) rg[v].load(gate + 8 * g);
        }
    }
    float r = 1.f;
    if (p.post) {
        float ss = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (threadIdx.x + v * threads < groups) {
                float f[8];
                ry[v].get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
            }
        r = 1.0f / sqrtf(cta_sum(ss, red[0]) / (float)p.K + p.eps);
    }
    float x[V][8], ss = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int g = threadIdx.x + v * threads;
        if (g >= groups) break;
        float f[8];
        ry[v].get(x[v]);
        if (p.post) {
            VT::load(static_cast<const T *>(p.post) + 8 * g, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[v][e] *= r * f[e];
        }
        if (p.gate) {
            rg[v].get(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[v][e] *= f[e];
        }
        rh[v].get(f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[v][e] = fmaf(p.alpha, x[v][e], f[e]);
            ss = fmaf(x[v][e], x[v][e], ss);
        }
        VH::store(static_cast<H *>(p.h_out) + row * p.ho_row + 8 * g, x[v]);
    }
    if (!p.gamma) return;
    r = 1.0f / sqrtf(cta_sum(ss, red[1]) / (float)p.K + p.eps);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int g = threadIdx.x + v * threads;
        if (g >= groups) break;
        float f[8];
        VT::load(static_cast<const T *>(p.gamma) + 8 * g, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[v][e] *= r * f[e];
        VT::store(static_cast<T *>(p.n_out) + row * p.no_row + 8 * g, x[v]);
    }
}

template <typename T, typename H>
cudaError_t launch(const NormParams &p, int M, cudaStream_t s) {
    // Few rows: as many threads as there are groups, for the shortest way through a row. Many rows: fewer
    // threads with more loads in flight each, and more rows on an SM at different stages.
    const int groups = p.K / 8;
    const bool many = M > 2 * sm_count() && groups > 256 && groups <= 1024;
    const int v = many ? (groups > 512 ? 4 : 2) : groups <= 1024 ? 1 : groups <= 2048 ? 2 : 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)M, 1, 1);
    cfg.blockDim = dim3((unsigned)((groups + v - 1) / v + 31) / 32 * 32, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = as_dependent(s) ? 1 : 0;
    if (many)
        return v == 4 ? cudaLaunchKernelEx(&cfg, residual_norm_kernel<T, H, 4, 256>, p)
                      : cudaLaunchKernelEx(&cfg, residual_norm_kernel<T, H, 2, 256>, p);
    if (v == 1) return cudaLaunchKernelEx(&cfg, residual_norm_kernel<T, H, 1, 1024>, p);
    if (v == 2) return cudaLaunchKernelEx(&cfg, residual_norm_kernel<T, H, 2, 1024>, p);
    return cudaLaunchKernelEx(&cfg, residual_norm_kernel<T, H, 4, 1024>, p);
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" w4a16_status w4a16_residual_rmsnorm(const void *h, w4a16_type h_type, long long h_row, const void *y,
                                               w4a16_type type, long long y_row, const void *post_gamma,
                                               const void *gate, long long gate_row, float alpha, const void *gamma,
                                               float eps, void *h_out, long long ho_row, void *n_out,
                                               long long no_row, int M, int K, void *stream) {
    if (M < 0 || K <= 0) return W4A16_ERR_INVALID_ARG;
    if (type != W4A16_TYPE_F16 && type != W4A16_TYPE_BF16) return W4A16_ERR_INVALID_ARG;
    if (h_type != type && h_type != W4A16_TYPE_F32)
        return h_type == W4A16_TYPE_F16 || h_type == W4A16_TYPE_BF16 ? W4A16_ERR_UNSUPPORTED : W4A16_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || std::isinf(eps) || std::isnan(alpha)) return W4A16_ERR_INVALID_ARG;
    if (K % 8 != 0 || K > kMaxK) return W4A16_ERR_UNSUPPORTED;
    if (M == 0) return W4A16_OK;
    if ((gamma == nullptr) != (n_out == nullptr)) return W4A16_ERR_INVALID_ARG;
    if (!h || !y || !h_out) return W4A16_ERR_INVALID_ARG;
    const int hv = h_type == W4A16_TYPE_F32 ? 4 : 8;  // elements of 16 bytes
    for (const void *p : {h, y, (const void *)h_out, (const void *)n_out, post_gamma, gate, gamma})
        if (!aligned(p, 16)) return W4A16_ERR_INVALID_ARG;
    if (M > 1 && (h_row < K || ho_row < K || y_row < K || (n_out && no_row < K) || (gate && gate_row && gate_row < K)))
        return W4A16_ERR_INVALID_ARG;
    if (h_row % hv || ho_row % hv || y_row % 8 || (n_out && no_row % 8) || (gate && gate_row % 8))
        return W4A16_ERR_INVALID_ARG;
    NormParams p{h, y, post_gamma, gate, gamma, h_out, n_out, h_row, y_row, gate_row, ho_row, no_row, K, alpha, eps, launch_overlap()};
    cudaStream_t s = (cudaStream_t)stream;
    if (type == W4A16_TYPE_F16)
        return from_cuda(h_type == W4A16_TYPE_F32 ? launch<__half, float>(p, M, s) : launch<__half, __half>(p, M, s));
    return from_cuda(h_type == W4A16_TYPE_F32 ? launch<__nv_bfloat16, float>(p, M, s)
                                              : launch<__nv_bfloat16, __nv_bfloat16>(p, M, s));
}

extern "C" w4a16_status w4a16_residual_rmsnorm_block(const w4a16_residual_rmsnorm_args *args) {
    if (!args) return W4A16_ERR_INVALID_ARG;
    const w4a16_residual_rmsnorm_args &a = *args;
    return w4a16_residual_rmsnorm(a.h, (w4a16_type)a.h_type, a.h_row, a.y, (w4a16_type)a.type, a.y_row, a.post_gamma,
                                  a.gate, a.gate_row, a.alpha, a.gamma, a.eps, a.h_out, a.ho_row, a.n_out, a.no_row,
                                  a.M, a.K, a.stream);
}
