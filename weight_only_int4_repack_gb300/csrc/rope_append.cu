// Rotary positions of a step's queries and keys, and its keys and values into the
// paged cache. For the pair (a, b) of a head's first rot_dim elements and the
// angle t = position * inv_freq:
//     (x_a, x_b) -> m * (x_a cos t - x_b sin t, x_b cos t + x_a sin t)
// A pair is (2i, 2i+1) or (i, i + rot_dim/2). Streaming work, bound by HBM: each
// element of q, k and v is read once and written once.
//
// The angle: a position times a frequency passes 2^24 times the spacing that fp32
// has near it, so the product is taken modulo one turn in 64-bit fixed point.
// F = inv_freq / (2 pi) * 2^64 modulo 2^64, one integer product of the frequency's
// 24-bit mantissa and the first 64 bits of 1 / (2 pi); position * F modulo 2^64 is
// another one and drops whole turns exactly; its upper 32 bits, signed, are the angle
// in units of 2^-32 turns. No fp64, of which the GPU has little.
#include <cmath>
#include <type_traits>

#include "decode_ops.h"
#include "elem.cuh"
#include "ptx.cuh"

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
    int rows, heads, rot, at_once;
    float mscale;
    unsigned int *err;
    bool overlap;
};

constexpr int kThreads = 128;
constexpr int kMaxHalf = 128;  // rot_dim / 2 at most

// cos and sin of frequency `inv_freq` at `pos`, times mscale.
__device__ __forceinline__ float2 rotation(float inv_freq, int pos, float mscale) {
    const uint32_t bits = __float_as_uint(inv_freq), exponent = (bits >> 23) & 0xffu;
    if (exponent == 0xffu) return make_float2(NAN, NAN);  // an infinite frequency has no angle, and NaN none either
    const unsigned long long mant = (bits & 0x7fffffu) | (exponent ? 0x800000u : 0u);
    const unsigned long long kTurn = 0x28BE60DB9391054Aull;  // 2^64 / (2 pi)
    // mant * kTurn * 2^(exponent - 150), modulo 2^64
    const unsigned long long lo = mant * kTurn, hi = __umul64hi(mant, kTurn);
    const int s = 150 - (int)(exponent ? exponent : 1u);
    unsigned long long F = s <= 0 ? (s > -64 ? lo << -s : 0ull)
                         : s < 64 ? (lo >> s) | (hi << (64 - s)) : s < 128 ? hi >> (s - 64) : 0ull;
    if (bits >> 31) F = 0ull - F;
    const unsigned long long part = (unsigned long long)(long long)pos * F;
    const float half_turns = (float)(int)(part >> 32) * 4.656612873077393e-10f;  // 2^-31
    float s1, c1;
    sincospif(half_turns, &s1, &c1);
    return make_float2(c1 * mscale, s1 * mscale);
}

// x / scale for an 8-bit cache, from the rounded reciprocal: the product's remainder is exact as a fused product, and
// corrects it to the rounded quotient (Markstein, IBM Journal of Research and Development 34, 1990), as long as it
// does not underflow (scales from 2^-60 on). Quotients beyond the type's range, infinite ones among them, saturate
// as they are. A division in its place took 59.1 us for the 16384 rows below, the product alone 53.0.
__device__ __forceinline__ float quotient(float x, float scale, float inverse) {
    const float q = x * inverse;
    return fabsf(q) < 1024.f ? fmaf(fmaf(-q, scale, x), inverse, q) : q;
}

// The row's place in the cache: false where its keys and values are not written.
struct Place {
    long long page, token;
};
__device__ __forceinline__ bool place_of(const RopeParams &p, long long slot, Place &at) {
    if (slot < 0) return false;
    if (slot >= (long long)p.c.pages * p.c.page_size) {
        atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG);
        return false;
    }
    if (slot < (1ll << 31)) {
        const unsigned int page = (unsigned int)slot / (unsigned int)p.c.page_size;
        at.page = page, at.token = (unsigned int)slot - page * (unsigned int)p.c.page_size;
    } else {
        at.page = slot / p.c.page_size, at.token = slot % p.c.page_size;
    }
    return true;
}

// rot_dim a multiple of 16, everything 16-byte aligned. A CTA takes p.at_once rows.
//
// A unit is 16 elements of a head as two groups a and b of 8, a lane's: eight pairs
// between a and b (halves), or four in each (neighbours), always those of frequencies
// 8u..8u+7; or elements behind rot_dim, and of v, which only get their bias. A warp's
// lanes cover several heads, a pass, and go through the CTA's rows with it: which
// heads, where they lie and their bias are found once for all rows. The rows' angles
// and cache places are worked out once for all heads, in shared memory. (A warp for
// each row, which finds the heads anew for every one, took 60.7 us for 16384 rows of
// 36 heads of 128 with an 8-bit cache, where this takes 52.2.)
// Measured (GB300, in a CUDA graph): that case (294 MB) 52.3 to 53.5 us, 5.5 TB/s, 83% of the
// copy rate; 4099 rows of 56 heads in bf16 (118 MB) 22.6 us, 78%: what a CTA does before
// its first row and the last round of CTAs weigh more there; one row 3.1 us. 64 registers
// are not quite enough: fp16 forms spill 8 to 36 bytes a thread, bf16 forms 64 to 184; the
// 4099 rows take 3% less time in fp16.
constexpr int kWideWarps = 16, kRowsAtOnce = 8;

template <typename T, typename C, bool kPairs>
__global__ void __launch_bounds__(32 * kWideWarps, 2) rope_append_wide_kernel(const RopeParams p) {
    using VT = elem::Vec<T, 8>;
    using VC = elem::Vec<C, 8>;
    // Row r's cos and sin of frequencies 8u + 2e, 8u + 2e + 1 at [r][e * turning units + u]: lanes side by side.
    __shared__ float4 cs[kRowsAtOnce][kMaxHalf / 2];
    __shared__ long long k_at[kRowsAtOnce], v_at[kRowsAtOnce];  // offsets in the pools; k_at < 0: not written
    if (p.overlap) ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int row0 = blockIdx.x * p.at_once, rows = min(p.at_once, p.rows - row0);
    const int D = p.c.head_dim, half = p.rot / 2, kv = p.c.kv_heads;
    const int units = (D + 15) / 16, heads_at = 32 / units, turning = p.rot / 16;
    const int sub = lane / units, u = lane - sub * units;
    const int q_passes = (p.heads + heads_at - 1) / heads_at, kv_passes = (kv + heads_at - 1) / heads_at;

    for (int pass = warp; pass < q_passes + 2 * kv_passes; pass += warps) {  // one at least: warps <= passes
        // Which heads, and where the lane's groups lie in them (b may lie behind the head).
        const bool q = pass < q_passes, v = pass >= q_passes + kv_passes;
        const int head = (pass - (q ? 0 : v ? q_passes + kv_passes : q_passes)) * heads_at + sub;
        const bool in = sub < heads_at && head < (q ? p.heads : kv);
        const bool turns = !v && u < turning;
        const int a_at = kPairs || !turns ? 16 * u : 8 * u, b_at = kPairs || !turns ? a_at + 8 : a_at + half;
        const bool two = b_at < D;
        const long long src_row = q ? p.q_row : v ? p.v_row : p.k_row;
        const T *src = (q ? static_cast<const T *>(p.q) + head * p.q_head
                          : v ? static_cast<const T *>(p.v) + head * p.v_head : static_cast<const T *>(p.k) + head * p.k_head) +
                       row0 * src_row + a_at;
        const int ab = b_at - a_at;
        uint4 ra[2], rb[2];  // two rows on their way
        auto load = [&](int x) {
            if (!in) return;
            ra[x] = __ldcs(reinterpret_cast<const uint4 *>(src));
            if (two) rb[x] = __ldcs(reinterpret_cast<const uint4 *>(src + ab));
            src += src_row;
        };
        load(0);
        if (rows > 1) load(1);
        uint4 fa = make_uint4(0, 0, 0, 0), fb = fa;
        if (p.bias && in) {
            const T *bias = static_cast<const T *>(p.bias) + (head + (q ? 0 : v ? p.heads + kv : p.heads)) * D;
            fa = *reinterpret_cast<const uint4 *>(bias + a_at);
            if (two) fb = *reinterpret_cast<const uint4 *>(bias + b_at);
        }
        T *q_out = static_cast<T *>(p.q_out) + row0 * p.qo_row + head * p.qo_head + a_at;
        C *pool = v ? static_cast<C *>(p.c.v) + head * p.c.v_head + a_at : static_cast<C *>(p.c.k) + head * p.c.k_head + a_at;
        const float *scales = v ? p.c.v_scale : p.c.k_scale;
        const float scale = !q && scales && in ? scales[head] : 1.0f, inverse = 1.0f / scale;

        if (pass == warp) {  // the first loads are on their way
            for (int i = threadIdx.x; i < rows * half; i += blockDim.x) {
                const int r = i / half, f = i - r * half, e = f & 7;
                reinterpret_cast<float2 *>(cs[r])[((e >> 1) * turning + (f >> 3)) * 2 + (e & 1)] =
                    rotation(p.inv_freq[f], p.positions[row0 + r], p.mscale);
            }
            if (threadIdx.x < rows) {
                Place at{0, 0};
                const bool writes = place_of(p, p.slots[row0 + threadIdx.x], at);
                k_at[threadIdx.x] = writes ? at.page * p.c.k_page + at.token * p.c.k_token : -1;
                v_at[threadIdx.x] = at.page * p.c.v_page + at.token * p.c.v_token;
            }
            __syncthreads();
        }
        // The lane's rows, for queries (0), keys (1) or values (2).
        auto go = [&](auto kind) {
            constexpr int kKind = decltype(kind)::value;
            const T *from = src;
            const long long *at = kKind == 2 ? v_at : k_at;
            for (int r0 = 0; r0 < rows; r0 += 2) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int r = r0 + y;
                    if (r >= rows) break;
                    float a[8], b[8];
                    VT::load(reinterpret_cast<const T *>(&ra[y]), a);
                    VT::load(reinterpret_cast<const T *>(&rb[y]), b);
                    if (r + 2 < rows) {
                        ra[y] = __ldcs(reinterpret_cast<const uint4 *>(from));
                        if (two) rb[y] = __ldcs(reinterpret_cast<const uint4 *>(from + ab));
                        from += src_row;
                    }
                    if (p.bias) {
                        float f[8];
                        VT::load(reinterpret_cast<const T *>(&fa), f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) a[e] += f[e];
                        VT::load(reinterpret_cast<const T *>(&fb), f);
#pragma unroll
                        for (int e = 0; e < 8; ++e) b[e] += f[e];
                    }
                    if (kKind < 2 && turns) {
                        const float4 *w = cs[r] + u;
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const float4 x = w[(e >> 1) * turning];  // cos, sin of two frequencies
                            if (kPairs) {
                                float *g = e < 4 ? a : b;
                                const int i = 2 * e & 7;
                                const float y0 = g[i], y2 = g[i + 2];
                                g[i] = y0 * x.x - g[i + 1] * x.y, g[i + 1] = g[i + 1] * x.x + y0 * x.y;
                                g[i + 2] = y2 * x.z - g[i + 3] * x.w, g[i + 3] = g[i + 3] * x.z + y2 * x.w;
                            } else {
                                const float y0 = a[e], y1 = a[e + 1];
                                a[e] = y0 * x.x - b[e] * x.y, b[e] = b[e] * x.x + y0 * x.y;
                                a[e + 1] = y1 * x.z - b[e + 1] * x.w, b[e + 1] = b[e + 1] * x.z + y1 * x.w;
                            }
                        }
                    }
                    if (kKind == 0) {
                        VT::store(q_out, a);
                        if (two) VT::store(q_out + ab, b);
                        q_out += p.qo_row;
                    } else if (k_at[r] >= 0) {
                        if (sizeof(C) == 1) {
#pragma unroll
                            for (int e = 0; e < 8; ++e) a[e] = quotient(a[e], scale, inverse), b[e] = quotient(b[e], scale, inverse);
                        }
                        VC::store(pool + at[r], a);
                        if (two) VC::store(pool + at[r] + ab, b);
                    }
                }
            }
        };
        if (!in) continue;
        if (q) go(std::integral_constant<int, 0>());
        else if (!v) go(std::integral_constant<int, 1>());
        else go(std::integral_constant<int, 2>());
    }
}

// Any alignment of 4 bytes and rot_dim a multiple of 4: two elements at a time, one CTA
// per row. Measured: 4099 rows of 28 heads of 80 in fp16, 40 turned (37 MB) 21 us, 26% of
// the copy rate, bound by instructions and latency. A head's work is rot/4 units that turn two pairs each, then units that copy
// two elements.
template <typename T, typename C, bool kPairs>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeParams p) {
    using VT = elem::Vec<T, 2>;
    using VC = elem::Vec<C, 2>;
    __shared__ float2 cs[kMaxHalf];
    if (p.overlap) ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const long long row = blockIdx.x;
    const int half = p.rot / 2, D = p.c.head_dim;
    const int pos = p.positions[row];
    for (int i = threadIdx.x; i < half; i += kThreads) cs[i] = rotation(p.inv_freq[i], pos, p.mscale);
    Place at{0, 0};
    const bool writes = place_of(p, p.slots[row], at);
    __syncthreads();

    const int turn_units = half / 2, units = turn_units + (D - p.rot) / 2, v_units = D / 2;
    const int nq = p.heads * units, nk = p.c.kv_heads * units, nv = p.c.kv_heads * v_units;
    for (int j = threadIdx.x; j < nq + nk + nv; j += kThreads) {
        const bool is_q = j < nq, is_v = j >= nq + nk;
        const int i = is_q ? j : is_v ? j - nq - nk : j - nq;
        const int per = is_v ? v_units : units;
        const int head = i / per, u = i - head * per;
        if (!is_q && !writes) continue;
        const T *src = is_q ? static_cast<const T *>(p.q) + row * p.q_row + head * p.q_head
                     : is_v ? static_cast<const T *>(p.v) + row * p.v_row + head * p.v_head
                            : static_cast<const T *>(p.k) + row * p.k_row + head * p.k_head;
        const int bias_head = is_q ? head : is_v ? p.heads + p.c.kv_heads + head : p.heads + head;
        const T *bias = p.bias ? static_cast<const T *>(p.bias) + bias_head * D : nullptr;
        const bool turn = !is_v && u < turn_units;
        // The unit's two groups of two elements (copies have one).
        const int lo = is_v ? 2 * u : turn ? (kPairs ? 4 * u : 2 * u) : p.rot + (u - turn_units) * 2;
        const int hi = kPairs ? lo + 2 : lo + half;
        float a[2], b[2] = {0.f, 0.f};
        VT::load(src + lo, a);
        if (turn) VT::load(src + hi, b);
        if (bias) {
            float f[2];
            VT::load(bias + lo, f);
            a[0] += f[0], a[1] += f[1];
            if (turn) {
                VT::load(bias + hi, f);
                b[0] += f[0], b[1] += f[1];
            }
        }
        if (turn) {
            const float2 w0 = cs[2 * u], w1 = cs[2 * u + 1];
            if (kPairs) {
                const float xa = a[0], xb = b[0];
                a[0] = xa * w0.x - a[1] * w0.y, a[1] = a[1] * w0.x + xa * w0.y;
                b[0] = xb * w1.x - b[1] * w1.y, b[1] = b[1] * w1.x + xb * w1.y;
            } else {
                const float x0 = a[0], x1 = a[1];
                a[0] = x0 * w0.x - b[0] * w0.y, a[1] = x1 * w1.x - b[1] * w1.y;
                b[0] = b[0] * w0.x + x0 * w0.y, b[1] = b[1] * w1.x + x1 * w1.y;
            }
        }
        if (is_q) {
            T *dst = static_cast<T *>(p.q_out) + row * p.qo_row + head * p.qo_head;
            VT::store(dst + lo, a);
            if (turn) VT::store(dst + hi, b);
        } else {
            C *dst = is_v ? static_cast<C *>(p.c.v) + at.page * p.c.v_page + at.token * p.c.v_token + head * p.c.v_head
                          : static_cast<C *>(p.c.k) + at.page * p.c.k_page + at.token * p.c.k_token + head * p.c.k_head;
            const float *scale = is_v ? p.c.v_scale : p.c.k_scale;
            if (scale) {
                const float s = scale[head], r = 1.0f / s;
                a[0] = quotient(a[0], s, r), a[1] = quotient(a[1], s, r);
                b[0] = quotient(b[0], s, r), b[1] = quotient(b[1], s, r);
            }
            VC::store(dst + lo, a);
            if (turn) VC::store(dst + hi, b);
        }
    }
}

template <typename T, typename C>
cudaError_t launch(RopeParams p, bool pairs, bool wide, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = as_dependent(s) ? 1 : 0;
    if (!wide) {
        cfg.gridDim = dim3((unsigned)p.rows, 1, 1);
        return pairs ? cudaLaunchKernelEx(&cfg, rope_append_kernel<T, C, true>, p)
                     : cudaLaunchKernelEx(&cfg, rope_append_kernel<T, C, false>, p);
    }
    // A warp for each pass. As many rows at once as take the fewest rounds of the CTAs that the SMs hold (64
    // registers a thread), where what a CTA does once costs about as much as one and a half rows.
    const int heads_at = 32 / ((p.c.head_dim + 15) / 16);
    const int passes = (p.heads + heads_at - 1) / heads_at + 2 * ((p.c.kv_heads + heads_at - 1) / heads_at);
    const int threads = 32 * (passes < kWideWarps ? passes : kWideWarps);
    const long long held = (long long)sm_count() * (1024 / threads);
    double least = 0.;
    for (int n = 1; n <= kRowsAtOnce; ++n) {
        const long long ctas = ((long long)p.rows + n - 1) / n, rounds = (ctas + held - 1) / held;
        if (n == 1 || rounds * (n + 1.5) < least) least = rounds * (n + 1.5), p.at_once = n;
    }
    cfg.gridDim = dim3((unsigned)((p.rows + p.at_once - 1) / p.at_once), 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    return pairs ? cudaLaunchKernelEx(&cfg, rope_append_wide_kernel<T, C, true>, p)
                 : cudaLaunchKernelEx(&cfg, rope_append_wide_kernel<T, C, false>, p);
}

template <typename T>
cudaError_t launch_type(const RopeParams &p, bool pairs, bool wide, cudaStream_t s) {
    return p.c.type == W4A16_TYPE_E4M3 ? launch<T, E4M3>(p, pairs, wide, s) : launch<T, T>(p, pairs, wide, s);
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
                 positions, inv_freq, slots, *cache, rows, heads, rot_dim, 1, mscale, device_error_ptr(), launch_overlap()};
    if (!p.err) return W4A16_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    return from_cuda(type == W4A16_TYPE_F16 ? launch_type<__half>(p, interleaved != 0, wide, s)
                                            : launch_type<__nv_bfloat16>(p, interleaved != 0, wide, s));
}

w4a16_status w4a16_rope_append_block(const w4a16_rope_append_args *args) {
    if (!args) return W4A16_ERR_INVALID_ARG;
    const w4a16_rope_append_args &a = *args;
    return w4a16_rope_append(a.q, a.k, a.v, (w4a16_type)a.type, a.q_row, a.q_head, a.k_row, a.k_head, a.v_row, a.v_head,
                             a.bias, a.positions, a.inv_freq, a.rot_dim, a.interleaved, a.mscale, a.q_out, a.qo_row,
                             a.qo_head, a.cache, a.slots, a.rows, a.heads, a.stream);
}

}  // extern "C"
