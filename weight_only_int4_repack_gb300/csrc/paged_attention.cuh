// Attention of one new token of each request over its pages of the cache.
//     s_j = scale * q . K_j (capped),  out = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m)
// Bound by HBM: each visible key and value is read once, for all query heads that
// share it.
//
// Work. A tile is kWarps slices of 16 or 32 tokens of one request, kv head and block
// of 8 * NT query heads. All tiles, request after request and head after head, form one line
// that is cut into equal parts, one for each CTA, so lengths may differ as they
// like and a single long request still fills the GPU. What a CTA has of a head's
// tokens is a segment; a head whose tokens lie in several CTAs leaves one partial
// result (maximum, sum, unnormalised output) for each, and the CTA that finishes
// last joins them in the order of the tokens, so results do not depend on timing.
// Many partial results are joined in two rounds, groups first.
//
// A segment. Warp w takes the w-th slice of each tile and keeps its own running
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
    unsigned int *counters;  // [3][kMaxCtas], zero between calls
    float *partial;          // [CTAs][2][kMaxPartial]
    int max_pages, batch, heads, group, head_blocks, window;
    float scale, softcap;
    unsigned int *err;
};

constexpr int kMaxCtas = 1024;
constexpr int kMaxPartial = 16 * (128 + 4);  // floats of the largest partial result (8 * (256 + 4) is less)
constexpr int kPerSm = 2;                    // CTAs on an SM: one streams while the other begins or ends a segment

template <typename T, typename C, int DT, int NT>
struct Config {
    static constexpr int kDim = DT;                        // head_dim, rounded up
    static constexpr int kRows = 8 * NT;                   // query heads of a block
    static constexpr int kBytes = sizeof(C);
    static constexpr int kRowBytes = DT * kBytes;          // a token's keys (or values) in the ring
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kTok = kRowBytes <= 128 ? 32 : 16;  // tokens of a slice
    static constexpr int kTiles = kTok / 16;
    static constexpr int kSliceBytes = kTok * kRowBytes;   // keys or values of a slice
    static constexpr int kWarps = kSliceBytes > 4096 ? 2 : 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kTile = kWarps * kTok;
    static constexpr int kStagesFit = 98304 / (kWarps * 2 * kSliceBytes);
    static constexpr int kStages = kStagesFit > 6 ? 6 : kStagesFit;
    static constexpr int kRing = kStages * 2 * kSliceBytes;  // one warp's
    static constexpr int kMerge = kWarps * kRows * (DT + 2) * 4;
    static constexpr int kSmem = kWarps * kRing > kMerge ? kWarps * kRing : kMerge;
    // A partial result: outputs, then maxima and sums, then room for those of a joined group.
    static constexpr int kPartial = kRows * (DT + 4);
    static_assert(kPartial <= kMaxPartial, "the workspace holds partial results of this size");
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

// Where a slice's tokens are: lane l knows that of token l (with 16 tokens, so does
// lane l + 16). The page number is loaded a slice ahead of its use, so that its
// latency is not waited for.
struct Places {
    int page;          // -1: not a visible token
    unsigned int at;   // the token's place in its page
};
template <int kTok>
__device__ __forceinline__ Places look_up(const Params &p, const int32_t *table, int t0, int lo, int hi, int lane) {
    const int tok = t0 + lane % kTok;
    Places x{-1, 0u};
    if (tok >= lo && tok < hi) {
        const unsigned int j = (unsigned int)tok / (unsigned int)p.c.page_size;
        x.page = __ldg(table + j);
        x.at = (unsigned int)tok - j * (unsigned int)p.c.page_size;
    }
    return x;
}

// One warp's copies of a slice into ring stage `dst`. Returns the mask of its rows
// that hold visible tokens of valid pages; the others become zeros. k, v: the lane's
// 16 bytes of the kv head's first token.
template <typename K, typename C>
__device__ __forceinline__ uint32_t load_slice(const Params &p, const Places &x, bool in_range, const C *k, const C *v,
                                               uint32_t dst, int lane) {
    constexpr int kLanes = K::kChunks < 8 ? K::kChunks : 8;  // lanes on a row
    constexpr int kRowsAt = 32 / kLanes;
    const int chunks = p.c.head_dim * K::kBytes / 16;
    const int sub = lane % kLanes;
    const bool good = x.page >= 0 && x.page < p.c.pages;
    if (!good && in_range) atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG);
    const uint32_t mask = __ballot_sync(0xffffffffu, good) & (K::kTok == 32 ? 0xffffffffu : 0xffffu);
    const int page_ok = good ? x.page : 0;
#pragma unroll
    for (int i = 0; i < K::kTok / kRowsAt; ++i) {
        const int row = i * kRowsAt + lane / kLanes;
        const bool ok = (mask >> row) & 1u;
        const long long page = __shfl_sync(0xffffffffu, page_ok, row);
        const long long at = __shfl_sync(0xffffffffu, x.at, row);
        const C *kr = k + page * p.c.k_page + at * p.c.k_token;
        const C *vr = v + page * p.c.v_page + at * p.c.v_token;
#pragma unroll
        for (int c = 0; c < K::kChunks / kLanes; ++c) {
            const int chunk = c * kLanes + sub;
            if (chunk < chunks) {
                const uint32_t o = place<K::kChunks>(row, chunk);
                copy16(dst + o, kr + c * kLanes * (16 / K::kBytes), ok);
                copy16(dst + K::kSliceBytes + o, vr + c * kLanes * (16 / K::kBytes), ok);
            }
        }
    }
    return mask;
}

// A running maximum, sum and unnormalised output of 4 elements, and another one
// taken in. Maxima are in units of log2.
struct Joined {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    __device__ __forceinline__ void take(float m2, float l2, const float4 &y) {
        const float mx = fmaxf(m, m2), top = mx == -INFINITY ? 0.f : mx;
        const float f1 = exp2_approx(m - top), f2 = exp2_approx(m2 - top);
        l = l * f1 + l2 * f2;
        o.x = o.x * f1 + y.x * f2, o.y = o.y * f1 + y.y * f2;
        o.z = o.z * f1 + y.z * f2, o.w = o.w * f1 + y.w * f2;
        m = mx;
    }
};

// Weights are drawn up by 2^kUp before they become operands of 16 bits, so that
// fp16 holds those down to 2^-(kUp + 14) of the largest with full precision.
constexpr float kUp = 12.f;

template <typename T, typename C, int DT, int NT>
__global__ void __launch_bounds__(Config<T, C, DT, NT>::kThreads, kPerSm) paged_attention_kernel(const Params p) {
    using K = Config<T, C, DT, NT>;
    constexpr bool k8 = sizeof(C) == 1;
    using M = typename std::conditional<k8, __half, T>::type;  // operand type
    // Weights become one operand of 16 bits and, with 16-bit caches, a second one for what the first's rounding
    // left: alone it would be as coarse as the output's own rounding. With 8-bit values, whose own rounding is
    // 2^-4, that second product is not spent.
    constexpr bool kTwo = !k8;
    constexpr int kSteps = DT / 16, MT = K::kTiles;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long sums[K::kWarps];
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
#pragma unroll
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
    constexpr int kLanes = K::kChunks < 8 ? K::kChunks : 8;
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
        const int lo = (int)r.lo, hi = (int)r.hi;  // lengths fit 31 bits
        // The warp's first token. Slices behind the last one may begin beyond 31 bits: taken modulo 2^32 they
        // turn negative and so lie outside [lo, hi).
        int tok = (int)((unsigned int)(r.lo / K::kTile + (t - item_begin)) * K::kTile + warp * K::kTok);
        const int32_t *table = p.table + b * p.table_stride;
        const C *kp = static_cast<const C *>(p.c.k) + kvh * p.c.k_head + lane % kLanes * (16 / K::kBytes);
        const C *vp = static_cast<const C *>(p.c.v) + kvh * p.c.v_head + lane % kLanes * (16 / K::kBytes);

        // Fill the ring.
        Places ahead = look_up<K::kTok>(p, table, tok, lo, hi, lane);
        int loaded = 0;
        auto load_next = [&](int stage) {
            if (loaded < count) {
                const Places now = ahead;
                const int mine = tok + lane % K::kTok;
                const bool in = mine >= lo && mine < hi;
                tok = (int)((unsigned int)tok + K::kTile);
                ahead = look_up<K::kTok>(p, table, tok, lo, hi, lane);
                const uint32_t mask = load_slice<K, C>(p, now, in, kp, vp, ring + stage * 2 * K::kSliceBytes, lane);
                if (lane == 0) masks[warp][stage] = mask;
                ++loaded;
            }
            copies_commit();
        };
#pragma unroll 1
        for (int i = 0; i < K::kStages - 1; ++i) load_next(i);

        // Queries as the B operand: column n = head lane/4, two k of each half. With 8-bit keys the k of a
        // step are taken in the order in which four consecutive bytes of a row come out of the ring.
        uint32_t q[kSteps][NT][2];
        float o[kSteps][NT][4];
        float m[NT][2], l[NT][2];  // maximum and sum of the thread's two heads (l: of its own rows)
        float q_scale = 1.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int head = nt * 8 + lane / 4;
            const T *qh = static_cast<const T *>(p.q) + b * p.q_row + (h0 + head) * p.q_head;
            // A scale of 0 or below turns into queries that are 0 or negated, and a positive scale.
            const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) {
                const int k0 = ks * 16 + (k8 ? 4 : 2) * (lane % 4);
                const bool in = head < rows && ks * 16 < D && p.scale != 0.f;
                const bool in2 = in && (k8 || ks * 16 + 8 < D);
                q[ks][nt][0] = in ? *reinterpret_cast<const uint32_t *>(qh + k0) ^ flip : 0u;
                q[ks][nt][1] = in2 ? *reinterpret_cast<const uint32_t *>(qh + k0 + (k8 ? 2 : 8)) ^ flip : 0u;
                o[ks][nt][0] = o[ks][nt][1] = o[ks][nt][2] = o[ks][nt][3] = 0.f;
            }
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
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
                        const float2 f = elem::pair_to_f32<T>(q[ks][nt][x]);
                        big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, x));
            const int e = big > 0.f && big < INFINITY ? max(ilogbf(big), -120) : 0;
            const float down = ldexpf(1.f, -e);
            q_scale = ldexpf(1.f, e);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float2 f = elem::pair_to_f32<T>(q[ks][nt][x]);
                        q[ks][nt][x] = elem::pair_from_f32<__half>(f.x * down, f.y * down);
                    }
        }
        // Scores in units of log2 are the products times `unit`.
        constexpr float kLog2e = 1.4426950408889634f;
        const float to_score = (p.scale != 0.f ? fabsf(p.scale) : 1.f) * q_scale * (k8 && p.c.k_scale ? p.c.k_scale[kvh] : 1.f);
        const float unit = p.softcap > 0.f ? 1.f : to_score * kLog2e;

        int stage = 0;
#pragma unroll 1
        for (int i = 0; i < count; ++i) {
            copies_wait<K::kStages - 2>();
            __syncwarp();
            const uint32_t sk = ring + stage * 2 * K::kSliceBytes, sv = sk + K::kSliceBytes;
            const uint32_t mask = masks[warp][stage];
            // Products: MT * 16 tokens x 8 NT heads; rows lane/4 and lane/4 + 8, heads 2*(lane%4) and the next.
            float s[MT][NT][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
#pragma unroll
            for (int ks = 0; ks < kSteps; ks += k8 ? 2 : 1) {
                if (ks * 16 >= D) break;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t w[4];
                    if constexpr (!k8) {
                        ldsm4(w, sk + place<K::kChunks>(mt * 16 + (lane & 15), ks * 2 + (lane >> 4)));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma<M>(s[mt][nt], w, q[ks][nt][0], q[ks][nt][1]);
                    } else {
                        ldsm4(w, sk + place<K::kChunks>(mt * 16 + (lane & 15), ks + (lane >> 4)));
#pragma unroll
                        for (int x = 0; x < 2; ++x) {  // two steps for each four matrices
                            const uint32_t a[4] = {elem::e4m3_to_half2((uint16_t)w[2 * x]),
                                                   elem::e4m3_to_half2((uint16_t)w[2 * x + 1]),
                                                   elem::e4m3_to_half2((uint16_t)(w[2 * x] >> 16)),
                                                   elem::e4m3_to_half2((uint16_t)(w[2 * x + 1] >> 16))};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma<M>(s[mt][nt], a, q[ks + x][nt][0], q[ks + x][nt][1]);
                        }
                    }
                }
            }
            if (p.softcap > 0.f) {
                const float in = to_score / p.softcap, out = p.softcap * kLog2e;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) s[mt][nt][x] = out * tanhf(s[mt][nt][x] * in);
            }
            if (mask != (K::kTok == 32 ? 0xffffffffu : 0xffffu)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (!((mask >> (mt * 16 + lane / 4 + (x < 2 ? 0 : 8))) & 1u))
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) s[mt][nt][x] = -INFINITY;
            }
            // Maxima over the slice's tokens, and what the past is worth under the new ones.
            float keep[NT][2], off[NT][2];
            bool moved = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float y = fmaxf(s[0][nt][x], s[0][nt][x + 2]);
#pragma unroll
                    for (int mt = 1; mt < MT; ++mt) y = fmaxf(y, fmaxf(s[mt][nt][x], s[mt][nt][x + 2]));
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                    y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
                    y = fmaxf(y, m[nt][x]);
                    const float top = y == -INFINITY ? 0.f : y;  // no token so far: all weights are 0
                    keep[nt][x] = exp2_approx((m[nt][x] - top) * unit);
                    off[nt][x] = kUp - top * unit;
                    moved |= m[nt][x] != y;
                    m[nt][x] = y;
                }
            if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    l[nt][0] *= keep[nt][0], l[nt][1] *= keep[nt][1];
#pragma unroll
                    for (int dt = 0; dt < kSteps; ++dt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[dt][nt][x] *= keep[nt][x & 1];
                }
            }
            uint32_t ph[MT][NT][2], pl[kTwo ? MT : 1][kTwo ? NT : 1][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) w[x] = exp2_approx(fmaf(s[mt][nt][x], unit, off[nt][x & 1]));
                    l[nt][0] += w[0] + w[2], l[nt][1] += w[1] + w[3];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t h = elem::pair_from_f32<M>(w[2 * x], w[2 * x + 1]);
                        ph[mt][nt][x] = transpose8x8(h);
                        if constexpr (kTwo) {
                            const float2 f = elem::pair_to_f32<M>(h);
                            pl[mt][nt][x] = transpose8x8(elem::pair_from_f32<M>(w[2 * x] - f.x, w[2 * x + 1] - f.y));
                        }
                    }
                }
            // Outputs: 16 elements of the head at a time.
#pragma unroll
            for (int dt = 0; dt < kSteps; dt += k8 ? 2 : 1) {
                if (dt * 16 >= D) break;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t w[4];
                    if constexpr (!k8) {
                        ldsm4_t(w, sv + place<K::kChunks>(mt * 16 + (lane & 7) + ((lane >> 4) << 3), dt * 2 + ((lane >> 3) & 1)));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma<M>(o[dt][nt], w, ph[mt][nt][0], ph[mt][nt][1]);
                            mma<M>(o[dt][nt], w, pl[mt][nt][0], pl[mt][nt][1]);
                        }
                    } else {
                        ldsm4_t(w, sv + place<K::kChunks>(mt * 16 + (lane & 15), dt + (lane >> 4)));
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            // Bytes: (d, d+1) of one token, (d, d+1) of the next; rows r, r + 8 become d = 2r, 2r + 1.
                            const uint32_t e0 = __byte_perm(w[2 * x], 0, 0x3120), e1 = __byte_perm(w[2 * x + 1], 0, 0x3120);
                            const uint32_t a[4] = {elem::e4m3_to_half2((uint16_t)e0), elem::e4m3_to_half2((uint16_t)(e0 >> 16)),
                                                   elem::e4m3_to_half2((uint16_t)e1), elem::e4m3_to_half2((uint16_t)(e1 >> 16))};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma<M>(o[dt + x][nt], a, ph[mt][nt][0], ph[mt][nt][1]);
                        }
                    }
                }
            }
            __syncwarp();  // all lanes have read the stage that is filled next time
            load_next(stage == 0 ? K::kStages - 1 : stage - 1);
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
                float sum = l[nt][x];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                if (lane < 4) mm[warp * K::kRows + row] = m[nt][x] * unit, ml[warp * K::kRows + row] = sum;
#pragma unroll
                for (int dt = 0; dt < kSteps; ++dt) {
                    float *to = mo + (warp * K::kRows + row) * DT + dt * 16;
                    to[k8 ? 2 * (lane / 4) : lane / 4] = o[dt][nt][x];
                    to[k8 ? 2 * (lane / 4) + 1 : lane / 4 + 8] = o[dt][nt][x + 2];
                }
            }
        __syncthreads();
        const int c_first = (int)(((item_begin + 1) * active - 1) / total), c_last = (int)((item_end * active - 1) / total);
        const int parts = c_last - c_first + 1;
        const float v_scale = k8 && p.c.v_scale ? p.c.v_scale[kvh] : 1.f;
        constexpr float kLn2 = 0.6931471805599453f;
        // A joined row: o / l, and its lse.
        auto finish = [&](int row, int d, const Joined &j) {
            const bool any = j.l > 0.f || j.l != j.l;
            const float f = any ? v_scale / j.l : 0.f;
            T *out = static_cast<T *>(p.out) + b * p.o_row + (h0 + row) * p.o_head + d;
            *reinterpret_cast<uint2 *>(out) =
                make_uint2(elem::pair_from_f32<T>(j.o.x * f, j.o.y * f), elem::pair_from_f32<T>(j.o.z * f, j.o.w * f));
            if (p.lse && d == 0)
                p.lse[(long long)b * p.heads + h0 + row] = any ? (j.m + log2f(j.l) - kUp) * kLn2 : -INFINITY;
        };
        // The place of the i-th partial result of this item.
        auto part = [&](int i) { return p.partial + ((long long)(c_first + i) * 2 + (i == 0)) * kMaxPartial; };
        auto leave = [&](float *to, int row, int d, const Joined &j, int joined) {
            __stcg(reinterpret_cast<float4 *>(to + row * DT + d), j.o);
            if (d == 0)
                __stcg(reinterpret_cast<float2 *>(to + K::kRows * (DT + 2 * joined) + 2 * row), make_float2(j.m, j.l));
        };
        for (int i = tid; i < rows * (DT / 4); i += K::kThreads) {
            const int row = i / (DT / 4), d = i % (DT / 4) * 4;
            if (d >= D) continue;
            Joined j;
#pragma unroll
            for (int w = 0; w < K::kWarps; ++w)
                j.take(mm[w * K::kRows + row], ml[w * K::kRows + row],
                       *reinterpret_cast<const float4 *>(mo + (w * K::kRows + row) * DT + d));
            if (parts == 1) finish(row, d, j);
            else leave(part(cta - c_first), row, d, j, 0);
        }
        if (parts > 1) {
            // Joined by the last CTA to arrive: first in groups of consecutive CTAs (when there are many), then
            // over the groups. A CTA is in front of the end of one item only, so counters at its number, one for
            // items that begin in it and one for the item that does not, are not shared.
            int group = 8;
            while (group * group < parts) ++group;
            const int of = (cta - c_first) / group, in_group = min(group, parts - of * group);
            const int groups = (parts + group - 1) / group;
            auto last_of = [&](unsigned int *counter, int n) {
                __threadfence();
                __syncthreads();
                if (tid == 0) {
                    is_last = atomicAdd(counter, 1u) == (unsigned int)n - 1u;
                    if (is_last) *counter = 0u;  // ready for the next call
                }
                __syncthreads();
                const bool yes = is_last;
                if (yes) __threadfence();
                return yes;
            };
            auto join = [&](int from, int step, int n, int joined, bool end) {
                for (int i = tid; i < rows * (DT / 4); i += K::kThreads) {
                    const int row = i / (DT / 4), d = i % (DT / 4) * 4;
                    if (d >= D) continue;
                    Joined j;
                    for (int c = 0; c < n; c += 8) {
                        float2 ml2[8];
                        float4 y[8];
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            const float *x = part(from + min(c + u, n - 1) * step);
                            ml2[u] = __ldcg(reinterpret_cast<const float2 *>(x + K::kRows * (DT + 2 * joined) + 2 * row));
                            y[u] = __ldcg(reinterpret_cast<const float4 *>(x + row * DT + d));
                        }
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            if (c + u < n) j.take(ml2[u].x, ml2[u].y, y[u]);
                    }
                    if (end) finish(row, d, j);
                    else leave(part(from), row, d, j, 1);
                }
            };
            unsigned int *counter = of == 0 ? p.counters + c_first : p.counters + kMaxCtas + c_first + of * group;
            if (last_of(counter, in_group)) {
                join(of * group, 1, in_group, 0, groups == 1);
                if (groups > 1 && last_of(p.counters + 2 * kMaxCtas + c_first, groups)) join(0, group, groups, 1, true);
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
cudaError_t launch(Params p, int sms, cudaStream_t s) {
    using K = Config<T, C, DT, NT>;
    auto kernel = paged_attention_kernel<T, C, DT, NT>;
    cudaError_t e = ensure_max_dyn_smem((const void *)kernel, K::kSmem);
    if (e != cudaSuccess) return e;
    p.head_blocks = (p.group + K::kRows - 1) / K::kRows;
    const long long tiles = ((long long)p.max_pages * p.c.page_size + K::kTile - 1) / K::kTile * p.batch *
                            p.c.kv_heads * p.head_blocks;
    const int ctas = sms * kPerSm < kMaxCtas ? sms * kPerSm : kMaxCtas;
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
cudaError_t launch_dims(const Params &p, int sms, cudaStream_t s) {
    const bool two = p.group > 8;
    if (p.c.head_dim <= 64) return two ? launch<T, C, 64, 2>(p, sms, s) : launch<T, C, 64, 1>(p, sms, s);
    if (p.c.head_dim <= 128) return two ? launch<T, C, 128, 2>(p, sms, s) : launch<T, C, 128, 1>(p, sms, s);
    return launch<T, C, 256, 1>(p, sms, s);
}

// Defined in paged_attention_f16.cu and paged_attention_bf16.cu.
cudaError_t launch_f16(const Params &p, int sms, cudaStream_t s);
cudaError_t launch_bf16(const Params &p, int sms, cudaStream_t s);

}  // namespace attn
}  // namespace w4a16
