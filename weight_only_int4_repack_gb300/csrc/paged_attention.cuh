// Attention of one new token of each request over its pages of the cache.
//     s_j = scale * q . K_j (capped),  out = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m)
// Bound by HBM: each visible key and value is read once, for all query heads that
// share it.
//
// Work. A tile is kWarps * 16 tokens of one request, kv head and block of 8 * NT
// query heads. All tiles, request after request and head after head, form one line
// that is cut into equal parts, one for each CTA, so lengths may differ as they
// like and a single long request still fills the GPU. What a CTA has of a head's
// tokens is a segment; a head whose tokens lie in several CTAs leaves one partial
// result (maximum, sum, unnormalised output) for each, and the CTA that finishes
// last joins them in the order of the tokens, so results do not depend on timing.
//
// A segment. Warp w takes the w-th 16 tokens of each tile and keeps its own running
// maximum, sum and output; the warps meet once, at the segment's end. Each warp
// feeds a ring of its own with 16-byte asynchronous copies (no CTA barrier in the
// loop). Tokens are the rows of the matrix instruction and query heads its columns
// (m16n8k16: S^T = K Q^T, O^T = V^T P^T), so heads are padded to 8, not to 16, and
// scores and outputs of one head stay in the same threads.
#pragma once

#include <cmath>

#include "elem.cuh"
#include "ptx.cuh"
#include "w4a16_internal.h"

namespace w4a16 {
namespace attn {

using elem::E4M3;

struct Params {
    const void *q;
    void *out;
    long long q_row, q_head, o_row, o_head, table_stride;
    w4a16_kv_cache c;
    const int32_t *table, *lens;
    float *lse;
    unsigned int *counters;  // [CTAs], zero between calls
    float *partial;          // [CTAs][2][rows * (kDim + 2)]
    int max_pages, batch, heads, group, head_blocks, window;
    float scale, softcap;
    unsigned int *err;
};

constexpr int kSlice = 16;  // tokens that a warp takes at a time

template <typename T, typename C, int DT, int NT>
struct Config {
    static constexpr int kDim = DT;                        // head_dim, rounded up
    static constexpr int kRows = 8 * NT;                   // query heads of a block
    static constexpr int kBytes = sizeof(C);
    static constexpr int kRowBytes = DT * kBytes;          // a token's keys (or values) in the ring
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kSliceBytes = kSlice * kRowBytes; // keys or values of a slice
    static constexpr int kWarps = kSliceBytes > 4096 ? 4 : 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kTile = kWarps * kSlice;
    static constexpr int kStagesFit = 196608 / (kWarps * 2 * kSliceBytes);
    static constexpr int kStages = kStagesFit > 6 ? 6 : kStagesFit;
    static constexpr int kRing = kStages * 2 * kSliceBytes;  // one warp's
    static constexpr int kMerge = kWarps * kRows * (DT + 2) * 4;
    static constexpr int kSmem = kWarps * kRing > kMerge ? kWarps * kRing : kMerge;
    static constexpr int kPartial = kRows * (DT + 2);        // floats of a partial result
    static_assert(kPartial <= 16 * (128 + 2), "the workspace holds partial results of this size");
};

// ------------------------------------------------------------------ instructions
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
template <typename M>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes to shared memory, or 16 zero bytes where `real` is false.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool real) {
    const int n = real ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Byte offset of 16-byte chunk `chunk` of ring row `row`: chunks change places so
// that the eight rows of an 8x8 matrix lie in eight different bank groups.
template <int kChunks>
__device__ __forceinline__ uint32_t place(int row, int chunk) {
    const int turn = kChunks >= 8 ? (row & 7) : ((row >> 1) & 3);
    return (uint32_t)(row * kChunks + (chunk ^ turn)) * 16;
}

// A request's visible tokens [lo, hi).
struct Range {
    long long lo, hi;
};
__device__ __forceinline__ Range visible(const Params &p, int b) {
    const long long most = (long long)p.max_pages * p.c.page_size;
    Range r;
    r.hi = min(max((long long)p.lens[b], 0ll), most);
    r.lo = p.window > 0 && r.hi > p.window ? r.hi - p.window : 0;
    return r;
}
template <int kTile>
__device__ __forceinline__ long long tiles_of(const Range &r) {
    return r.hi > r.lo ? (r.hi + kTile - 1) / kTile - r.lo / kTile : 0;
}

// Where the 16 tokens of a slice are: lane l (and l + 16) knows that of token l. The
// page number is loaded a slice ahead of its use, so its latency is not waited for.
struct Places {
    int page;          // -1: not a visible token
    unsigned int at;   // the token's place in its page
};
__device__ __forceinline__ Places look_up(const Params &p, const int32_t *table, long long t0, const Range &r, int lane) {
    const long long tok = t0 + (lane & 15);
    Places x{-1, 0u};
    if (tok >= r.lo && tok < r.hi) {  // lengths fit 31 bits
        const unsigned int j = (unsigned int)tok / (unsigned int)p.c.page_size;
        x.page = __ldg(table + j);
        x.at = (unsigned int)tok - j * (unsigned int)p.c.page_size;
    }
    return x;
}

// One warp's copies of a slice into ring stage `dst`. Returns the mask of its rows
// that hold visible tokens of valid pages; the others become zeros.
template <typename K, typename C>
__device__ __forceinline__ uint32_t load_slice(const Params &p, const Places &x, const Range &r, long long t0, int kvh,
                                               uint32_t dst, int lane) {
    constexpr int kLanes = K::kChunks < 8 ? K::kChunks : 8;  // lanes on a row
    constexpr int kRowsAt = 32 / kLanes;
    const int chunks = p.c.head_dim * K::kBytes / 16;
    const int sub = lane % kLanes;
    const long long tok = t0 + (lane & 15);
    const bool good = x.page >= 0 && x.page < p.c.pages;
    if (!good && tok >= r.lo && tok < r.hi) atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG);
    const uint32_t mask = __ballot_sync(0xffffffffu, good) & 0xffffu;
    const int page_ok = good ? x.page : 0;
    const C *kh = static_cast<const C *>(p.c.k) + kvh * p.c.k_head + sub * (16 / K::kBytes);
    const C *vh = static_cast<const C *>(p.c.v) + kvh * p.c.v_head + sub * (16 / K::kBytes);
#pragma unroll
    for (int i = 0; i < kSlice / kRowsAt; ++i) {
        const int row = i * kRowsAt + lane / kLanes;
        const bool ok = (mask >> row) & 1u;
        const long long page = __shfl_sync(0xffffffffu, page_ok, row);
        const long long at = __shfl_sync(0xffffffffu, x.at, row);
        const C *k = kh + page * p.c.k_page + at * p.c.k_token;
        const C *v = vh + page * p.c.v_page + at * p.c.v_token;
#pragma unroll
        for (int c = 0; c < K::kChunks / kLanes; ++c) {
            const int chunk = c * kLanes + sub;
            if (chunk < chunks) {
                const uint32_t o = place<K::kChunks>(row, chunk);
                copy16(dst + o, k + c * kLanes * (16 / K::kBytes), ok);
                copy16(dst + K::kSliceBytes + o, v + c * kLanes * (16 / K::kBytes), ok);
            }
        }
    }
    return mask;
}

// Running state of a warp over its slices of a segment. M is the operand type.
template <typename K, typename M, int NT>
struct State {
    uint32_t q[K::kDim / 16][NT][2];
    float o[K::kDim / 16][NT][4];
    float m[NT][2], l[NT][2];  // maximum and sum of the thread's two heads (l: of its own rows)
};

// Weights are drawn up by 2^kUp before they become operands of 16 bits, so that
// fp16 holds those down to 2^-(kUp + 14) of the largest with full precision.
constexpr float kUp = 12.f;

template <typename T, typename C, int DT, int NT>
__global__ void __launch_bounds__(Config<T, C, DT, NT>::kThreads, 1) paged_attention_kernel(const Params p) {
    using K = Config<T, C, DT, NT>;
    constexpr bool k8 = sizeof(C) == 1;
    using M = typename std::conditional<k8, __half, T>::type;  // operand type
    constexpr int kSteps = DT / 16;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long sums[32];
    __shared__ long long first_base;
    __shared__ int first_request;
    __shared__ uint32_t masks[K::kWarps][K::kStages];
    __shared__ int is_last;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x, ctas = gridDim.x;
    const int D = p.c.head_dim;
    const int items = p.c.kv_heads * p.head_blocks;  // of a request

    // Where this CTA's part of the line begins.
    const int per = (p.batch + K::kThreads - 1) / K::kThreads;
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += tiles_of<K::kTile>(visible(p, b));
    long long upto = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, x);
        if (lane >= x) upto += y;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    long long total = 0;
    for (int w = 0; w < K::kWarps; ++w) {
        if (w == warp) upto += total;
        total += sums[w];
    }
    total *= items;
    const int active = (int)min((long long)ctas, total);  // CTAs with work: each has a tile at least
    const long long t_begin = cta < active ? total * cta / active : 0, t_end = cta < active ? total * (cta + 1) / active : 0;
    long long before = (upto - mine) * items;
    if (t_begin < t_end && before <= t_begin && t_begin < upto * items) {
        for (int b = b0; b < b1; ++b) {
            const long long n = tiles_of<K::kTile>(visible(p, b)) * items;
            if (t_begin < before + n) {
                first_request = b;
                first_base = before;
                break;
            }
            before += n;
        }
    }
    // Requests without tokens, and lengths out of range.
    for (int b = cta; b < p.batch; b += ctas) {
        const Range r = visible(p, b);
        if (tid == 0 && (p.lens[b] < 0 || p.lens[b] > (long long)p.max_pages * p.c.page_size))
            atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG);
        if (r.hi > r.lo) continue;
        for (int i = tid; i < p.heads * D; i += K::kThreads)
            static_cast<T *>(p.out)[b * p.o_row + (i / D) * p.o_head + i % D] = T(0.f);
        if (p.lse)
            for (int i = tid; i < p.heads; i += K::kThreads) p.lse[(long long)b * p.heads + i] = -INFINITY;
    }
    if (D < DT)  // the ring's columns beyond head_dim stay zero
        for (int i = tid; i < K::kWarps * K::kRing / 16; i += K::kThreads)
            reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();

    const uint32_t ring = ptx::smem_u32(smem) + warp * K::kRing;
    long long t = t_begin, base = first_base;
    int b = first_request;
    while (t < t_end) {
        Range r = visible(p, b);
        long long n = tiles_of<K::kTile>(r);
        while (t >= base + n * items) {
            base += n * items;
            r = visible(p, ++b);
            n = tiles_of<K::kTile>(r);
        }
        const int item = (int)((t - base) / n);
        const long long item_begin = base + item * n, item_end = item_begin + n;
        const long long seg_end = min(t_end, item_end);
        const int count = (int)(seg_end - t);  // tiles of the segment
        const int kvh = item / p.head_blocks, h0 = kvh * p.group + (item % p.head_blocks) * K::kRows;
        const int rows = min(K::kRows, (kvh + 1) * p.group - h0);
        const long long tok0 = (r.lo / K::kTile + (t - item_begin)) * K::kTile + warp * kSlice;
        const int32_t *table = p.table + b * p.table_stride;

        State<K, M, NT> st;
        // Queries as the B operand: column n = head lane/4, two k of each half. With 8-bit keys the k of a
        // step are taken in the order in which four consecutive bytes of a row come out of the ring.
        float q_scale = 1.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int head = nt * 8 + lane / 4;
            const T *q = static_cast<const T *>(p.q) + b * p.q_row + (h0 + head) * p.q_head;
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
                const int k0 = ks * 16 + (k8 ? 4 : 2) * (lane % 4);
                const bool in = head < rows && ks * 16 < D;
                const bool in2 = in && (k8 || ks * 16 + 8 < D);
                st.q[ks][nt][0] = in ? *reinterpret_cast<const uint32_t *>(q + k0) : 0u;
                st.q[ks][nt][1] = in2 ? *reinterpret_cast<const uint32_t *>(q + k0 + (k8 ? 2 : 8)) : 0u;
                st.o[ks][nt][0] = st.o[ks][nt][1] = st.o[ks][nt][2] = st.o[ks][nt][3] = 0.f;
            }
            st.m[nt][0] = st.m[nt][1] = -INFINITY;
            st.l[nt][0] = st.l[nt][1] = 0.f;
        }
        if constexpr (k8 && !std::is_same<T, __half>::value) {
            // bf16 queries against 8-bit keys: keys become fp16 (exact), queries fp16 after a power of two that
            // brings the block's largest below 2; what that loses is 2^-25 of the largest.
            float big = 0.f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float2 f = elem::pair_to_f32<T>(st.q[ks][nt][x]);
                        big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, x));
            const int e = big > 0.f && big < INFINITY ? ilogbf(big) : 0;
            const float down = ldexpf(1.f, -max(e, -120));
            q_scale = ldexpf(1.f, max(e, -120));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float2 f = elem::pair_to_f32<T>(st.q[ks][nt][x]);
                        st.q[ks][nt][x] = elem::pair_from_f32<__half>(f.x * down, f.y * down);
                    }
        }
        const float k_scale = p.scale * q_scale * (k8 && p.c.k_scale ? p.c.k_scale[kvh] : 1.f);
        constexpr float kLog2e = 1.4426950408889634f;

        // Fill the ring, then one slice out and one in.
        const int fill = min(count, K::kStages - 1);
        Places ahead = look_up(p, table, tok0, r, lane);
#pragma unroll 1
        for (int i = 0; i < K::kStages - 1; ++i) {
            if (i < fill) {
                const Places now = ahead;
                const long long t0 = tok0 + (long long)i * K::kTile;
                ahead = look_up(p, table, t0 + K::kTile, r, lane);
                const uint32_t mask = load_slice<K, C>(p, now, r, t0, kvh, ring + i * 2 * K::kSliceBytes, lane);
                if (lane == 0) masks[warp][i] = mask;
            }
            copies_commit();
        }
        int stage = 0;
#pragma unroll 1
        for (int i = 0; i < count; ++i) {
            copies_wait<K::kStages - 2>();
            __syncwarp();
            const uint32_t sk = ring + stage * 2 * K::kSliceBytes, sv = sk + K::kSliceBytes;
            const uint32_t mask = masks[warp][stage];
            // Scores: 16 tokens x 8 NT heads.
            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
            if constexpr (!k8) {
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks) {
                    if (ks * 16 >= D) break;
                    uint32_t a[4];
                    ldsm4(a, sk + place<K::kChunks>(lane & 15, ks * 2 + (lane >> 4)));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma<M>(s[nt], a, st.q[ks][nt][0], st.q[ks][nt][1]);
                }
            } else {
#pragma unroll
                for (int k2 = 0; k2 < kSteps / 2; ++k2) {  // two steps for each four matrices
                    if (k2 * 32 >= D) break;
                    uint32_t w[4];
                    ldsm4(w, sk + place<K::kChunks>(lane & 15, k2 * 2 + (lane >> 4)));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t a[4] = {elem::e4m3_to_half2((uint16_t)w[2 * x]), elem::e4m3_to_half2((uint16_t)w[2 * x + 1]),
                                               elem::e4m3_to_half2((uint16_t)(w[2 * x] >> 16)),
                                               elem::e4m3_to_half2((uint16_t)(w[2 * x + 1] >> 16))};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma<M>(s[nt], a, st.q[2 * k2 + x][nt][0], st.q[2 * k2 + x][nt][1]);
                    }
                }
            }
            // Scores in units of log2: rows lane/4 and lane/4 + 8, heads 2*(lane%4) and the next.
            const bool up = (mask >> (lane / 4)) & 1u, low = (mask >> (lane / 4 + 8)) & 1u;
            uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float y = s[nt][x] * k_scale;
                    if (p.softcap > 0.f) y = p.softcap * tanhf(y / p.softcap);
                    s[nt][x] = (x < 2 ? up : low) ? y * kLog2e : -INFINITY;
                }
                float top[2], keep[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float y = fmaxf(s[nt][x], s[nt][x + 2]);
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
                    y = fmaxf(y, st.m[nt][x]);
                    top[x] = y == -INFINITY ? 0.f : y;  // no token so far: all weights are 0
                    keep[x] = exp2_approx(st.m[nt][x] - top[x]);
                    st.m[nt][x] = y;
                }
                float w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) w[x] = exp2_approx(s[nt][x] - top[x & 1] + kUp);
#pragma unroll
                for (int x = 0; x < 2; ++x) st.l[nt][x] = st.l[nt][x] * keep[x] + (w[x] + w[x + 2]);
                if (__any_sync(0xffffffffu, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
                    for (int dt = 0; dt < kSteps; ++dt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) st.o[dt][nt][x] *= keep[x & 1];
                }
                // Weights as two operands, the value and what its rounding left: one of 16 bits would be as
                // coarse as the output's own rounding.
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t h = elem::pair_from_f32<M>(w[2 * x], w[2 * x + 1]);
                    const float2 f = elem::pair_to_f32<M>(h);
                    ph[nt][x] = transpose8x8(h);
                    pl[nt][x] = transpose8x8(elem::pair_from_f32<M>(w[2 * x] - f.x, w[2 * x + 1] - f.y));
                }
            }
            // Outputs: 16 elements of the head at a time.
            if constexpr (!k8) {
#pragma unroll
                for (int dt = 0; dt < kSteps; ++dt) {
                    if (dt * 16 >= D) break;
                    uint32_t a[4];
                    ldsm4_t(a, sv + place<K::kChunks>((lane & 7) + ((lane >> 4) << 3), dt * 2 + ((lane >> 3) & 1)));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma<M>(st.o[dt][nt], a, ph[nt][0], ph[nt][1]);
                        mma<M>(st.o[dt][nt], a, pl[nt][0], pl[nt][1]);
                    }
                }
            } else {
#pragma unroll
                for (int d2 = 0; d2 < kSteps / 2; ++d2) {
                    if (d2 * 32 >= D) break;
                    uint32_t w[4];
                    ldsm4_t(w, sv + place<K::kChunks>(lane & 15, d2 * 2 + (lane >> 4)));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        // Bytes: (d, d+1) of one token, (d, d+1) of the next; rows r and r + 8 become d = 2r, 2r + 1.
                        const uint32_t e0 = __byte_perm(w[2 * x], 0, 0x3120), e1 = __byte_perm(w[2 * x + 1], 0, 0x3120);
                        const uint32_t a[4] = {elem::e4m3_to_half2((uint16_t)e0), elem::e4m3_to_half2((uint16_t)(e0 >> 16)),
                                               elem::e4m3_to_half2((uint16_t)e1), elem::e4m3_to_half2((uint16_t)(e1 >> 16))};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma<M>(st.o[2 * d2 + x][nt], a, ph[nt][0], ph[nt][1]);
                            mma<M>(st.o[2 * d2 + x][nt], a, pl[nt][0], pl[nt][1]);
                        }
                    }
                }
            }
            __syncwarp();  // all lanes have read the stage that is filled next time
            const int next = i + K::kStages - 1;
            if (next < count) {
                const int to = stage == 0 ? K::kStages - 1 : stage - 1;
                const Places now = ahead;
                const long long t0 = tok0 + (long long)next * K::kTile;
                ahead = look_up(p, table, t0 + K::kTile, r, lane);
                const uint32_t got = load_slice<K, C>(p, now, r, t0, kvh, ring + to * 2 * K::kSliceBytes, lane);
                if (lane == 0) masks[warp][to] = got;
            }
            copies_commit();
            stage = stage + 1 == K::kStages ? 0 : stage + 1;
        }
        copies_wait<0>();
        __syncthreads();

        // The warps' results meet in shared memory (the ring is empty): [warp][row][DT], then maxima, sums.
        float *mo = reinterpret_cast<float *>(smem);
        float *mm = mo + K::kWarps * K::kRows * DT, *ml = mm + K::kWarps * K::kRows;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int row = nt * 8 + 2 * (lane % 4) + x;
                float l = st.l[nt][x];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                if (lane < 4) mm[warp * K::kRows + row] = st.m[nt][x], ml[warp * K::kRows + row] = l;
#pragma unroll
                for (int dt = 0; dt < kSteps; ++dt) {
                    float *o = mo + (warp * K::kRows + row) * DT + dt * 16;
                    o[k8 ? 2 * (lane / 4) : lane / 4] = st.o[dt][nt][x];
                    o[k8 ? 2 * (lane / 4) + 1 : lane / 4 + 8] = st.o[dt][nt][x + 2];
                }
            }
        __syncthreads();
        const int c_first = (int)(((item_begin + 1) * active - 1) / total), c_last = (int)((item_end * active - 1) / total);
        const bool whole = c_first == c_last;
        float *part = p.partial + ((long long)cta * 2 + (cta == c_first)) * K::kPartial;
        const float v_scale = k8 && p.c.v_scale ? p.c.v_scale[kvh] : 1.f;
        constexpr float kLn2 = 0.6931471805599453f;
        // A joined row: o / l, and its lse.
        auto finish = [&](int row, int d, float4 o, float m, float l) {
            const float f = l > 0.f || l != l ? v_scale / l : 0.f;
            T *out = static_cast<T *>(p.out) + b * p.o_row + (h0 + row) * p.o_head + d;
            *reinterpret_cast<uint2 *>(out) =
                make_uint2(elem::pair_from_f32<T>(o.x * f, o.y * f), elem::pair_from_f32<T>(o.z * f, o.w * f));
            if (p.lse && d == 0)
                p.lse[(long long)b * p.heads + h0 + row] = l > 0.f || l != l ? (m + log2f(l) - kUp) * kLn2 : -INFINITY;
        };
        for (int i = tid; i < rows * (DT / 4); i += K::kThreads) {
            const int row = i / (DT / 4), d = i % (DT / 4) * 4;
            if (d >= D) continue;
            float m = -INFINITY, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < K::kWarps; ++w) m = fmaxf(m, mm[w * K::kRows + row]);
            const float top = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int w = 0; w < K::kWarps; ++w) {
                const float f = exp2_approx(mm[w * K::kRows + row] - top);
                const float4 x = *reinterpret_cast<const float4 *>(mo + (w * K::kRows + row) * DT + d);
                l += f * ml[w * K::kRows + row];
                o.x += f * x.x, o.y += f * x.y, o.z += f * x.z, o.w += f * x.w;
            }
            if (whole) {
                finish(row, d, o, m, l);
            } else {
                __stcg(reinterpret_cast<float4 *>(part + row * DT + d), o);
                if (d == 0) __stcg(part + K::kRows * DT + 2 * row, m), __stcg(part + K::kRows * DT + 2 * row + 1, l);
            }
        }
        if (!whole) {
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const unsigned int parts = (unsigned int)(c_last - c_first + 1);
                const bool last = atomicAdd(p.counters + c_first, 1u) == parts - 1;
                if (last) p.counters[c_first] = 0u;  // ready for the next call
                is_last = last;
            }
            __syncthreads();
            if (is_last) {
                __threadfence();
                const float *first = p.partial + ((long long)c_first * 2 + 1) * K::kPartial;
                for (int i = tid; i < rows * (DT / 4); i += K::kThreads) {
                    const int row = i / (DT / 4), d = i % (DT / 4) * 4;
                    if (d >= D) continue;
                    float m = -INFINITY, l = 0.f;
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int c = c_first; c <= c_last; ++c) {
                        const float *x = c == c_first ? first : p.partial + (long long)c * 2 * K::kPartial;
                        const float m2 = __ldcg(x + K::kRows * DT + 2 * row), l2 = __ldcg(x + K::kRows * DT + 2 * row + 1);
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(x + row * DT + d));
                        const float mx = fmaxf(m, m2), top = mx == -INFINITY ? 0.f : mx;
                        const float f1 = exp2_approx(m - top), f2 = exp2_approx(m2 - top);
                        l = l * f1 + l2 * f2;
                        o.x = o.x * f1 + y.x * f2, o.y = o.y * f1 + y.y * f2;
                        o.z = o.z * f1 + y.z * f2, o.w = o.w * f1 + y.w * f2;
                        m = mx;
                    }
                    finish(row, d, o, m, l);
                }
            }
        }
        t = seg_end;
        __syncthreads();  // the merge area becomes the ring again
        if (D < DT && t < t_end) {
            for (int i = tid; i < K::kWarps * K::kRing / 16; i += K::kThreads)
                reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
            __syncthreads();
        }
    }
}

template <typename T, typename C, int DT, int NT>
cudaError_t launch(Params p, int ctas, cudaStream_t s) {
    using K = Config<T, C, DT, NT>;
    auto kernel = paged_attention_kernel<T, C, DT, NT>;
    cudaError_t e = ensure_max_dyn_smem((const void *)kernel, K::kSmem);
    if (e != cudaSuccess) return e;
    p.head_blocks = (p.group + K::kRows - 1) / K::kRows;
    const long long tiles = ((long long)p.max_pages * p.c.page_size + K::kTile - 1) / K::kTile * p.batch *
                            p.c.kv_heads * p.head_blocks;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles < ctas ? tiles : ctas), 1, 1);
    cfg.blockDim = dim3(K::kThreads, 1, 1);
    cfg.dynamicSmemBytes = K::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = launch_overlap() ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T, typename C>
cudaError_t launch_dims(const Params &p, int ctas, cudaStream_t s) {
    const bool two = p.group > 8;
    if (p.c.head_dim <= 64) return two ? launch<T, C, 64, 2>(p, ctas, s) : launch<T, C, 64, 1>(p, ctas, s);
    if (p.c.head_dim <= 128) return two ? launch<T, C, 128, 2>(p, ctas, s) : launch<T, C, 128, 1>(p, ctas, s);
    return launch<T, C, 256, 1>(p, ctas, s);
}

// Defined in paged_attention_f16.cu and paged_attention_bf16.cu.
cudaError_t launch_f16(const Params &p, int ctas, cudaStream_t s);
cudaError_t launch_bf16(const Params &p, int ctas, cudaStream_t s);

}  // namespace attn
}  // namespace w4a16
