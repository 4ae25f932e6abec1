// Rotary positions of a step's queries and keys, and its keys and values into the
// paged cache. For the pair (a, b) of a head's first rot_dim elements and the
// angle t = position * inv_freq:
//     (x_a, x_b) -> m * (x_a cos t - x_b sin t, x_b cos t + x_a sin t)
// A pair is (2i, 2i+1) or (i, i + rot_dim/2). Streaming work, bound by HBM: each
// element of q, k and v is read once and written once.
//
// The angle: a position times a frequency passes 2^24 times the spacing that fp32
// has near it, so the product is taken modulo one turn in 64-bit fixed point.
// F = frac(inv_freq / 2 pi) * 2^64 (fp64, once per frequency); position * F modulo
// 2^64 is one integer multiplication and drops whole turns exactly; its upper 32
// bits, signed, are the angle in units of 2^-32 turns.
#include <cmath>

#include "elem.cuh"
#include "ptx.cuh"
#include "w4a16_internal.h"

namespace w4a16 {
namespace {

using elem::E4M3;

struct RopeParams {
    const void *q, *k, *v, *bias;
    void *q_out;
    long long q_row, q_head, k_row, k_head, v_row, v_head, qo_row, qo_head;
    const int32_t *positions;
    const float *inv_freq;
    const int64_t *slots;
    w4a16_kv_cache c;
    int rows, heads, rot;
    float mscale;
    unsigned int *err;
};

constexpr int kThreads = 256;
constexpr int kMaxHalf = 128;  // rot_dim / 2 at most

// cos and sin of frequency i at `pos`, times mscale.
__device__ __forceinline__ float2 rotation(float inv_freq, int pos, float mscale) {
    double turns = (double)inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= floor(turns);
    const unsigned long long F = __double2ull_rd(turns * 18446744073709551616.0);
    const unsigned long long part = (unsigned long long)(long long)pos * F;
    const float half_turns = (float)(int)(part >> 32) * 4.656612873077393e-10f;  // 2^-31
    float s, c;
    sincospif(half_turns, &s, &c);
    return make_float2(c * mscale, s * mscale);
}

// One CTA per row. A head's work is cut into units: rot/2/VEC units that each turn
// VEC pairs, then units that copy VEC elements.
template <typename T, typename C, int VEC, bool kPairs>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeParams p) {
    using VT = elem::Vec<T, VEC>;
    using VC = elem::Vec<C, VEC>;
    __shared__ float2 cs[kMaxHalf];
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const long long row = blockIdx.x;
    const int half = p.rot / 2, D = p.c.head_dim;
    const int pos = p.positions[row];
    for (int i = threadIdx.x; i < half; i += kThreads) cs[i] = rotation(p.inv_freq[i], pos, p.mscale);
    long long slot = p.slots[row];
    if (slot >= (long long)p.c.pages * p.c.page_size) {
        if (threadIdx.x == 0) atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG);
        slot = -1;
    }
    const long long page = slot < 0 ? 0 : slot / p.c.page_size;
    const long long token = slot < 0 ? 0 : slot % p.c.page_size;
    __syncthreads();

    const int turn_units = half / VEC, units = turn_units + (D - p.rot) / VEC;
    const int v_units = D / VEC;
    const int nq = p.heads * units, nk = p.c.kv_heads * units, nv = p.c.kv_heads * v_units;
    for (int j = threadIdx.x; j < nq + nk + nv; j += kThreads) {
        const bool is_q = j < nq, is_v = j >= nq + nk;
        const int i = is_q ? j : is_v ? j - nq - nk : j - nq;
        const int per = is_v ? v_units : units;
        const int head = i / per, u = i - head * per;
        if (!is_q && slot < 0) continue;
        const T *src = is_q ? static_cast<const T *>(p.q) + row * p.q_row + head * p.q_head
                     : is_v ? static_cast<const T *>(p.v) + row * p.v_row + head * p.v_head
                            : static_cast<const T *>(p.k) + row * p.k_row + head * p.k_head;
        const int bias_head = is_q ? head : is_v ? p.heads + p.c.kv_heads + head : p.heads + head;
        const T *bias = p.bias ? static_cast<const T *>(p.bias) + bias_head * D : nullptr;
        const bool turn = !is_v && u < turn_units;
        // The unit's two groups of VEC elements (copies have one).
        const int lo = is_v ? u * VEC : turn ? (kPairs ? 2 * VEC * u : VEC * u) : p.rot + (u - turn_units) * VEC;
        const int hi = kPairs ? lo + VEC : lo + half;
        float a[VEC], b[VEC];
        VT::load(src + lo, a);
        if (turn) VT::load(src + hi, b);
        if (bias) {
            float f[VEC];
            VT::load(bias + lo, f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) a[e] += f[e];
            if (turn) {
                VT::load(bias + hi, f);
#pragma unroll
                for (int e = 0; e < VEC; ++e) b[e] += f[e];
            }
        }
        if (turn) {
            const float2 *w = cs + u * VEC;
            if (kPairs) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {  // pair e of the 2*VEC elements a, b
                    float &x = (2 * e < VEC) ? a[2 * e % VEC] : b[2 * e % VEC];
                    float &y = (2 * e < VEC) ? a[2 * e % VEC + 1] : b[2 * e % VEC + 1];
                    const float x1 = x * w[e].x - y * w[e].y;
                    y = y * w[e].x + x * w[e].y;
                    x = x1;
                }
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float x1 = a[e] * w[e].x - b[e] * w[e].y;
                    b[e] = b[e] * w[e].x + a[e] * w[e].y;
                    a[e] = x1;
                }
            }
        }
        if (is_q) {
            T *dst = static_cast<T *>(p.q_out) + row * p.qo_row + head * p.qo_head;
            VT::store(dst + lo, a);
            if (turn) VT::store(dst + hi, b);
        } else {
            C *dst = is_v ? static_cast<C *>(p.c.v) + page * p.c.v_page + token * p.c.v_token + head * p.c.v_head
                          : static_cast<C *>(p.c.k) + page * p.c.k_page + token * p.c.k_token + head * p.c.k_head;
            const float *scale = is_v ? p.c.v_scale : p.c.k_scale;
            if (scale) {
                const float s = scale[head];
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    a[e] = a[e] / s;
                    if (turn) b[e] = b[e] / s;
                }
            }
            VC::store(dst + lo, a);
            if (turn) VC::store(dst + hi, b);
        }
    }
}

template <typename T, typename C, int VEC>
cudaError_t launch(const RopeParams &p, bool pairs, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.rows, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = launch_overlap() ? 1 : 0;
    return pairs ? cudaLaunchKernelEx(&cfg, rope_append_kernel<T, C, VEC, true>, p)
                 : cudaLaunchKernelEx(&cfg, rope_append_kernel<T, C, VEC, false>, p);
}

template <typename T>
cudaError_t launch_type(const RopeParams &p, bool pairs, bool wide, cudaStream_t s) {
    if (p.c.type == W4A16_TYPE_E4M3)
        return wide ? launch<T, E4M3, 8>(p, pairs, s) : launch<T, E4M3, 2>(p, pairs, s);
    return wide ? launch<T, T, 8>(p, pairs, s) : launch<T, T, 2>(p, pairs, s);
}

}  // namespace

w4a16_status check_cache(const w4a16_kv_cache *c) {
    if (!c || !c->k || !c->v || c->pages <= 0 || c->page_size <= 0 || c->kv_heads <= 0 || c->head_dim <= 0)
        return W4A16_ERR_INVALID_ARG;
    if (c->type != W4A16_TYPE_F16 && c->type != W4A16_TYPE_BF16 && c->type != W4A16_TYPE_E4M3)
        return W4A16_ERR_INVALID_ARG;
    const bool e4m3 = c->type == W4A16_TYPE_E4M3;
    const int per16 = e4m3 ? 16 : 8;  // elements of 16 bytes
    if (!e4m3 && (c->k_scale || c->v_scale)) return W4A16_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
        return W4A16_ERR_INVALID_ARG;
    for (long long stride : {c->k_page, c->k_token, c->k_head, c->v_page, c->v_token, c->v_head})
        if (stride < 0 || stride % per16) return W4A16_ERR_INVALID_ARG;
    for (long long stride : {c->k_page, c->k_token, c->k_head, c->v_page, c->v_token, c->v_head})
        if (stride >= (1LL << 31)) return W4A16_ERR_UNSUPPORTED;
    if (c->head_dim % per16 || c->head_dim > 256) return W4A16_ERR_UNSUPPORTED;
    if ((long long)c->pages * c->page_size > (1LL << 40)) return W4A16_ERR_UNSUPPORTED;
    return W4A16_OK;
}

}  // namespace w4a16

using namespace w4a16;

extern "C" {

w4a16_status w4a16_rope_frequencies(float *inv_freq, int rot_dim, double base, int scaling, double factor,
                                    double context, double low, double high) {
    if (!inv_freq || rot_dim <= 0 || rot_dim % 2 || !(base > 0) || std::isinf(base) || scaling < 0 || scaling > 3)
        return W4A16_ERR_INVALID_ARG;
    if (scaling && (!(factor >= 1) || std::isinf(factor))) return W4A16_ERR_INVALID_ARG;
    if (scaling == 2 && rot_dim < 4) return W4A16_ERR_INVALID_ARG;
    if (scaling == 3 && (!(context > 0) || !(high > low))) return W4A16_ERR_INVALID_ARG;
    if (scaling == 2) base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == 1) f /= factor;
        if (scaling == 3) {
            const double turns = context * f / (2.0 * 3.14159265358979323846);
            const double keep = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
            f = f * keep + f / factor * (1.0 - keep);
        }
        inv_freq[i] = (float)f;
    }
    return W4A16_OK;
}

w4a16_status w4a16_rope_append(const void *q, const void *k, const void *v, w4a16_type type, long long q_row,
                               long long q_head, long long k_row, long long k_head, long long v_row, long long v_head,
                               const void *bias, const int32_t *positions, const float *inv_freq, int rot_dim,
                               int interleaved, float mscale, void *q_out, long long qo_row, long long qo_head,
                               const w4a16_kv_cache *cache, const int64_t *slots, int rows, int heads, void *stream) {
    w4a16_status st = check_cache(cache);
    if (st != W4A16_OK) return st;
    if (type != W4A16_TYPE_F16 && type != W4A16_TYPE_BF16) return W4A16_ERR_INVALID_ARG;
    if (cache->type != type && cache->type != W4A16_TYPE_E4M3) return W4A16_ERR_UNSUPPORTED;
    if (rows < 0 || heads <= 0 || (interleaved != 0 && interleaved != 1)) return W4A16_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > cache->head_dim) return W4A16_ERR_INVALID_ARG;
    if (rot_dim % 4) return W4A16_ERR_UNSUPPORTED;
    if (rows == 0) return W4A16_OK;
    if (!q || !k || !v || !q_out || !positions || !slots || (rot_dim && !inv_freq)) return W4A16_ERR_INVALID_ARG;
    if (!aligned(positions, 4) || !aligned(inv_freq, 4) || !aligned(slots, 8)) return W4A16_ERR_INVALID_ARG;
    bool wide = rot_dim % 16 == 0;
    for (const void *p : {q, k, v, (const void *)q_out, bias}) {
        if (!aligned(p, 4)) return W4A16_ERR_INVALID_ARG;
        wide = wide && aligned(p, 16);
    }
    for (long long s : {q_row, q_head, k_row, k_head, v_row, v_head, qo_row, qo_head}) {
        if (s < 0 || s % 2) return W4A16_ERR_INVALID_ARG;
        wide = wide && s % 8 == 0;
    }
    RopeParams p{q, k, v, bias, q_out, q_row, q_head, k_row, k_head, v_row, v_head, qo_row, qo_head,
                 positions, inv_freq, slots, *cache, rows, heads, rot_dim, mscale, device_error_ptr()};
    if (!p.err) return W4A16_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    return from_cuda(type == W4A16_TYPE_F16 ? launch_type<__half>(p, interleaved != 0, wide, s)
                                            : launch_type<__nv_bfloat16>(p, interleaved != 0, wide, s));
}

}  // extern "C"
