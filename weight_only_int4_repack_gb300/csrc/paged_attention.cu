// Attention of one new token of each request over its pages of the cache.
//     s_j = scale * q . K_j (capped),  out = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m)
// Bound by HBM: each visible key and value is read once.
//
// One CTA per request and query head. Its warps take every eighth token, each with
// its own running maximum, sum and output, joined in shared memory at the end.
#include <cmath>

#include "elem.cuh"
#include "ptx.cuh"
#include "w4a16_internal.h"

namespace w4a16 {
namespace {

using elem::E4M3;

struct AttnParams {
    const void *q;
    void *out;
    long long q_row, q_head, o_row, o_head, table_stride;
    w4a16_kv_cache c;
    const int32_t *table, *lens;
    float *lse;
    int max_pages, batch, heads, window;
    float scale, softcap;
    unsigned int *err;
};

constexpr int kWarps = 8;

template <typename T, typename C>
__global__ void __launch_bounds__(32 * kWarps) paged_attention_kernel(const AttnParams p) {
    __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][256];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int head = blockIdx.x % p.heads, b = blockIdx.x / p.heads;
    const int kvh = head / (p.heads / p.c.kv_heads);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = p.c.head_dim;
    const long long most = (long long)p.max_pages * p.c.page_size;
    long long len = p.lens[b];
    if (len > most || len < 0) {
        if (threadIdx.x == 0) atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG);
        len = len < 0 ? 0 : most;
    }
    const long long first = p.window > 0 && len > p.window ? len - p.window : 0;
    const float ks = p.c.k_scale ? p.c.k_scale[kvh] : 1.f, vs = p.c.v_scale ? p.c.v_scale[kvh] : 1.f;
    // Lane l holds the elements 8l .. 8l+7.
    const bool in = 8 * lane < D;
    float q[8] = {}, o[8] = {}, m = -INFINITY, l = 0.f;
    if (in) elem::Vec<T, 8>::load(static_cast<const T *>(p.q) + b * p.q_row + head * p.q_head + 8 * lane, q);
    for (long long j = first + warp; j < len; j += kWarps) {
        const int page = p.table[b * p.table_stride + j / p.c.page_size];
        if (page < 0 || page >= p.c.pages) {
            if (lane == 0) atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG);
            continue;
        }
        const long long tok = j % p.c.page_size;
        float k[8] = {}, v[8] = {};
        if (in) {
            elem::Vec<C, 8>::load(static_cast<const C *>(p.c.k) + page * p.c.k_page + tok * p.c.k_token +
                                      kvh * p.c.k_head + 8 * lane, k);
            elem::Vec<C, 8>::load(static_cast<const C *>(p.c.v) + page * p.c.v_page + tok * p.c.v_token +
                                      kvh * p.c.v_head + 8 * lane, v);
        }
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(q[e], k[e], s);
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= p.scale * ks;
        if (p.softcap > 0.f) s = p.softcap * tanhf(s / p.softcap);
        const float m2 = fmaxf(m, s), keep = m2 == -INFINITY ? 1.f : expf(m - m2);
        const float e2 = m2 == -INFINITY ? 0.f : expf(s - m2);
        l = l * keep + e2;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = o[e] * keep + e2 * v[e];
        m = m2;
    }
    if (lane == 0) sm_m[warp] = m, sm_l[warp] = l;
    if (in)
#pragma unroll
        for (int e = 0; e < 8; ++e) sm_o[warp][8 * lane + e] = o[e];
    __syncthreads();
    if (warp) return;
    float top = -INFINITY, total = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm_m[w]);
    float r[8] = {};
    for (int w = 0; w < kWarps; ++w) {
        const float f = top == -INFINITY ? 0.f : expf(sm_m[w] - top);
        total += f * sm_l[w];
        if (in)
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] += f * sm_o[w][8 * lane + e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = total > 0.f || total != total ? r[e] * vs / total : 0.f;
    if (in) elem::Vec<T, 8>::store(static_cast<T *>(p.out) + b * p.o_row + head * p.o_head + 8 * lane, r);
    if (p.lse && lane == 0) p.lse[(long long)b * p.heads + head] = total > 0.f ? top + logf(total) : -INFINITY;
}

template <typename T, typename C>
cudaError_t launch(const AttnParams &p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.batch * p.heads), 1, 1);
    cfg.blockDim = dim3(32 * kWarps, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = launch_overlap() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, paged_attention_kernel<T, C>, p);
}

template <typename T>
cudaError_t launch_type(const AttnParams &p, cudaStream_t s) {
    return p.c.type == W4A16_TYPE_E4M3 ? launch<T, E4M3>(p, s) : launch<T, T>(p, s);
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

size_t w4a16_paged_attention_workspace_bytes(int batch, int heads, int kv_heads, int head_dim) {
    if (batch <= 0 || heads <= 0 || kv_heads <= 0 || head_dim <= 0 || heads % kv_heads) return 0;
    return 256;
}

w4a16_status w4a16_paged_attention(const void *q, w4a16_type type, long long q_row, long long q_head,
                                   const w4a16_kv_cache *cache, const int32_t *table, long long table_stride,
                                   int max_pages, const int32_t *lens, int batch, int heads, float scale, int window,
                                   float softcap, void *out, long long o_row, long long o_head, float *lse, void *ws,
                                   size_t ws_bytes, void *stream) {
    w4a16_status st = check_cache(cache);
    if (st != W4A16_OK) return st;
    if (type != W4A16_TYPE_F16 && type != W4A16_TYPE_BF16) return W4A16_ERR_INVALID_ARG;
    if (cache->type != type && cache->type != W4A16_TYPE_E4M3) return W4A16_ERR_UNSUPPORTED;
    if (batch < 0 || heads <= 0 || heads % cache->kv_heads || max_pages <= 0 || table_stride < max_pages || window < 0)
        return W4A16_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f) return W4A16_ERR_INVALID_ARG;
    if ((long long)batch * heads > (1 << 24)) return W4A16_ERR_UNSUPPORTED;
    if (batch == 0) return W4A16_OK;
    if (!q || !out || !table || !lens) return W4A16_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(lse, 4))
        return W4A16_ERR_INVALID_ARG;
    for (long long s : {q_row, q_head, o_row, o_head})
        if (s < 0 || s % 8) return W4A16_ERR_INVALID_ARG;
    if (!ws || !aligned(ws, 256) ||
        ws_bytes < w4a16_paged_attention_workspace_bytes(batch, heads, cache->kv_heads, cache->head_dim))
        return W4A16_ERR_WORKSPACE;
    const AttnParams p{q, out, q_row, q_head, o_row, o_head, table_stride, *cache, table, lens, lse,
                       max_pages, batch, heads, window, scale, softcap, device_error_ptr()};
    if (!p.err) return W4A16_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    return from_cuda(type == W4A16_TYPE_F16 ? launch_type<__half>(p, s) : launch_type<__nv_bfloat16>(p, s));
}

}  // extern "C"
