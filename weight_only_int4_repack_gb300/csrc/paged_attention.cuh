// Attention of one new token of each request over its pages of the cache.
//     s_j = scale * q . K_j (capped),  out = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m)
// Bound by HBM: each visible key and value is read once for each block of 16 query
// heads (8 where heads are wider than 128) that share it.
//
// Work. A tile is kWarps slices of 16 or 32 tokens of one request, kv head and block
// of 8 * NT query heads. All tiles, request after request and head after head, form
// one line that is cut into equal parts, one for each CTA, so lengths may differ as
// they like and a single long request still fills the GPU. What a CTA has of a head's
// tokens is a segment; a head whose tokens lie in several CTAs leaves one partial
// result (maximum, sum, unnormalised output) for each, and the CTA that finishes
// last joins them in the order of the tokens, so results do not depend on timing.
// Many partial results are joined in two rounds, groups first.
//
// A segment. Warp w takes the w-th slice of each tile and keeps its own running
// maximum, sum and output; the warps meet once, at the segment's end. Each warp
// feeds a ring of its own with 16-byte asynchronous copies (no CTA barrier in the
// loop), and begins to fill it for the next segment before the warps meet. Tokens
// are the rows of the matrix instruction and query heads its columns (m16n8k16:
// S^T = K Q^T, O^T = V^T P^T), so heads are padded to 8, not to 16, and scores and
// outputs of one head stay in the same threads.
//
// Measured (GB300, in a CUDA graph): 64 requests of 0 to 8191 tokens, 40 query and 8
// kv heads of 128 in fp16 (1.16 GB) 173 to 180 us, 6.5 to 6.7 TB/s, the rate of a plain
// copy; 121 requests of up to 16001 tokens, 32 and 2 heads, 8-bit cache (0.59 GB) 105
// to 107 us with fp16 queries, 107 to 108 with bf16 ones, bound by instructions (about
// 560 for each 16 tokens of 16 heads, of which 64 convert e4m3 to fp16). A call that is
// not long, or has few heads, pays about 4 us until the first keys arrive (lengths, then
// the table, then keys) and 3 to 12 us for joins: one request of 1000 tokens 7.8 us, two
// of up to 200003 with 2 kv heads 56 us. 32 query heads on one key head are two blocks,
// so everything is read twice: 128 requests of up to 8000 tokens (0.32 GB) 95 us, 32 of
// them 32 us.
// Rows of a head that are no multiple of 128 bytes, in a cache laid out tokens first,
// share memory lines with other heads' that are read at another time: 52% of the copy
// rate with 64 e4m3 elements, 73% with 96 of fp16; heads first 92% and 100%.
#pragma once

#include <cmath>
#include <type_traits>

#include "decode_ops.h"
#include "elem.cuh"
#include "ptx.cuh"

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
    int one_page;  // page_size is a multiple of 16
    unsigned int k_page, k_token, v_page, v_token;  // strides below 2^31
    float scale, softcap;
    unsigned int *err;
};

constexpr int kMaxCtas = 1024;
constexpr int kMaxPartial = 16 * (128 + 4);  // floats of the largest partial result (8 * (256 + 4) is less)
constexpr int kMostPerSm = 3;                // CTAs on an SM at most

// The reference that scores are taken relative to is moved (and everything summed so
// far rescaled) only when a score passes it by more than kSlack powers of two. The
// reference's own weight is 2^kUp. As fp16 operands weights then reach 2^15, within the
// range, and are held down to 2^-25 of the reference with full precision, smaller ones
// to 2^-36 of it. bf16 has the range of fp32: there they stay below 1, so that values of
// any size can be summed.
constexpr float kSlack = 4.f, kLowest = -3.402823466e38f;
template <typename M>
constexpr float kUpOf = std::is_same<M, __half>::value ? 11.f : -kSlack;

template <typename T, typename C, int DT, int NT>
struct Config {
    using M = typename std::conditional<sizeof(C) == 1, __half, T>::type;  // operand type
    static constexpr float kUp = kUpOf<M>;
    static constexpr int kDim = DT;                        // head_dim, rounded up
    static constexpr int kRows = 8 * NT;                   // query heads of a block
    static constexpr int kBytes = sizeof(C);
    static constexpr int kRowBytes = DT * kBytes;          // a token's keys (or values) in the ring
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kTok = DT == 64 ? 32 : 16;  // tokens of a slice
    static constexpr uint32_t kAll = kTok == 32 ? 0xffffffffu : 0xffffu;
    // CTAs on an SM: one streams while another begins or ends a segment. 8-bit slices cost more instructions for
    // each byte, so a third CTA's warps are needed.
    static constexpr int kPerSm = kBytes == 1 && DT <= 128 ? 3 : 2;
    static constexpr int kSliceBytes = kTok * kRowBytes;   // keys or values of a slice
    static constexpr int kWarps = DT == 256 ? (kBytes == 1 ? 3 : 2) : 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kTile = kWarps * kTok;
    static constexpr int kStagesFit = (kBytes == 1 ? 147456 : 196608) / kPerSm / (kWarps * 2 * kSliceBytes);
    static constexpr int kStages = kStagesFit > 6 ? 6 : kStagesFit;
    static constexpr int kRing = kStages * 2 * kSliceBytes;  // one warp's
    static constexpr int kPitch = DT + 4;                    // of a row in the merge area: no bank conflicts
    static constexpr int kMerge = kWarps * 8 * kPitch * 4;   // 8 heads of every warp
    static_assert(kMerge >= kRows * DT * 2, "the queries lie in the merge area");
    static constexpr int kSmem = kWarps * kRing + kMerge;
    // A partial result: outputs, then maxima and sums, then room for those of a joined group.
    static constexpr int kPartial = kRows * (DT + 4);
    static constexpr int kStaged = kRows * (DT + 2);         // floats of one of them while they are joined
    static constexpr int kJoin = kWarps * kRing / (kStaged * 4) < 24 ? kWarps * kRing / (kStaged * 4) : 24;
    static_assert(kWarps * 8 >= kRows, "a joined row's maximum and sum lie where the warps' were");
    static_assert(kStages >= 3, "one slice is computed on while two are on their way");
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

// Two weights as pairs of 16-bit operands: h, and l for what h's rounding left. h is rounded
// down and l is never 0 where h is not (2^-24 or 2^-126 at least), so that an infinite value
// times either is that infinity.
__device__ __forceinline__ void split(float a, float b, uint32_t &h, uint32_t &l, __half) {
    uint32_t least;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(b), "f"(a));
    const float2 f = elem::pair_to_f32<__half>(h);
    l = elem::pair_from_f32<__half>(a - f.x, b - f.y);
    asm("min.f16x2 %0, %1, %2;" : "=r"(least) : "r"(h), "r"(0x00010001u));
    asm("max.f16x2 %0, %1, %2;" : "=r"(l) : "r"(l), "r"(least));
}
__device__ __forceinline__ void split(float a, float b, uint32_t &h, uint32_t &l, __nv_bfloat16) {
    uint32_t least;
    h = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    const float2 f = elem::pair_to_f32<__nv_bfloat16>(h);
    l = elem::pair_from_f32<__nv_bfloat16>(a - f.x, b - f.y);
    asm("min.bf16x2 %0, %1, %2;" : "=r"(least) : "r"(h), "r"(0x00800080u));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(l) : "r"(l), "r"(least));
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
    int lo, hi;
};
__device__ __forceinline__ Range visible(const Params &p, int b) {
    const long long most = (long long)p.max_pages * p.c.page_size;
    Range r;
    r.hi = (int)min((long long)max(p.lens[b], 0), most);
    r.lo = p.window > 0 && r.hi > p.window ? r.hi - p.window : 0;
    return r;
}
template <int kTile>
__device__ __forceinline__ int tiles_of(const Range &r) {
    return r.hi > r.lo ? (r.hi - 1) / kTile + 1 - r.lo / kTile : 0;
}

// Where a slice's tokens are: lane l knows that of token l (with 16 tokens, so does
// lane l + 16). The page number is loaded a slice ahead of its use, so that its
// latency is not waited for.
struct Places {
    int page;          // -1: not a visible token
    unsigned int at;   // the token's place in its page
};
// The lane's token of the slice that is looked up next: its number, and page and place
// as the division gives them once and every step of a tile moves them on.
struct Cursor {
    int tok;
    unsigned int j, at;
};

// One warp's copies of a slice into ring stage `dst`. Returns the mask of its rows
// that hold visible tokens of valid pages; the others become zeros. k, v: the lane's
// 16 bytes of the kv head in the lane's first row, row lane/kLanes of a page.
template <typename K, typename C>
__device__ __forceinline__ uint32_t load_slice(const Params &p, const Places &x, bool in_range, const C *k, const C *v,
                                               uint32_t dst, int lane) {
    constexpr int kLanes = K::kChunks < 8 ? K::kChunks : 8;  // lanes on a row
    constexpr int kRowsAt = 32 / kLanes;
    const int chunks = p.c.head_dim * K::kBytes / 16;
    const int sub = lane % kLanes, row0 = lane / kLanes;
    const bool good = x.page >= 0 && x.page < p.c.pages;
    if (!good && in_range) atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG);
    const uint32_t mask = __ballot_sync(0xffffffffu, good) & K::kAll;
    // The offset of the lane's token from the pool's first (a slice begins at a multiple of 16 tokens).
    const unsigned int page = good ? x.page : 0, at = good ? x.at : 0;
    const unsigned long long k_token = p.k_token, v_token = p.v_token;  // products below are of 64 bits
    const unsigned long long k_at = (unsigned long long)page * p.k_page + at * k_token;
    const unsigned long long v_at = (unsigned long long)page * p.v_page + at * v_token;
    auto copy_row = [&](int i, const C *kr, const C *vr) {
        const bool ok = (mask >> (i * kRowsAt + row0)) & 1u;
#pragma unroll
        for (int c = 0; c < K::kChunks / kLanes; ++c)
            if (c * kLanes + sub < chunks) {
                const uint32_t o = place<K::kChunks>(i * kRowsAt + row0, c * kLanes + sub);
                copy16(dst + o, kr + c * kLanes * (16 / K::kBytes), ok);
                copy16(dst + K::kSliceBytes + o, vr + c * kLanes * (16 / K::kBytes), ok);
            }
    };
    if (p.one_page) {  // pages of a multiple of 16 tokens: 16 tokens lie in one, that of the first visible one
#pragma unroll
        for (int g = 0; g < K::kTok / 16; ++g) {
            const uint32_t here = (mask >> (16 * g)) & 0xffffu;
            const int from = here ? __ffs(here) - 1 : 0;
            const C *kr = k + (__shfl_sync(0xffffffffu, k_at, 16 * g + from) - from * k_token);
            const C *vr = v + (__shfl_sync(0xffffffffu, v_at, 16 * g + from) - from * v_token);
#pragma unroll
            for (int i = 0; i < 16 / kRowsAt; ++i)
                copy_row(g * (16 / kRowsAt) + i, kr + i * kRowsAt * k_token, vr + i * kRowsAt * v_token);
        }
    } else {
#pragma unroll
        for (int i = 0; i < K::kTok / kRowsAt; ++i) {
            const int row = i * kRowsAt + row0;
            copy_row(i, k + (__shfl_sync(0xffffffffu, k_at, row) - row0 * k_token),
                     v + (__shfl_sync(0xffffffffu, v_at, row) - row0 * v_token));
        }
    }
    return mask;
}

// What a CTA has of one item of the line (a request, kv head and block of heads).
struct Segment {
    int b, kvh, h0, rows, count;  // first query head, heads, tiles
    int begin, end;               // the item's tiles in the line
    int t, base;                  // the line's tile behind the segment, and the request's first
    int c_first, parts;           // the first CTA with tokens of the item, and how many have some (set at its end)
};

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

// Where a segment's results go.
template <typename K, typename T>
struct Ends {
    const Params &p;
    const Segment seg;
    const float v_scale;

    // A joined row: o / l, and its lse.
    __device__ __forceinline__ void finish(int row, int d, const Joined &j) const {
        constexpr float kLn2 = 0.6931471805599453f;
        const bool any = j.l > 0.f || j.l != j.l;
        const float f = any ? v_scale / j.l : 0.f;
        T *out = static_cast<T *>(p.out) + seg.b * p.o_row + (seg.h0 + row) * p.o_head + d;
        *reinterpret_cast<uint2 *>(out) =
            make_uint2(elem::pair_from_f32<T>(j.o.x * f, j.o.y * f), elem::pair_from_f32<T>(j.o.z * f, j.o.w * f));
        if (p.lse && d == 0)
            p.lse[(long long)seg.b * p.heads + seg.h0 + row] = any ? (j.m + log2f(j.l) - K::kUp) * kLn2 : -INFINITY;
    }
    // The place of the i-th partial result of these heads.
    __device__ __forceinline__ float *part(int i) const {
        return p.partial + ((long long)(seg.c_first + i) * 2 + (i == 0)) * kMaxPartial;
    }
    __device__ __forceinline__ void leave(float *to, int row, int d, const Joined &j, int joined) const {
        __stcg(reinterpret_cast<float4 *>(to + row * K::kDim + d), j.o);
        if (d == 0)
            __stcg(reinterpret_cast<float2 *>(to + K::kRows * (K::kDim + 2 * joined) + 2 * row), make_float2(j.m, j.l));
    }
    // Joins n partial results, `step` apart from `from` on, into the output or the first one's place. They come
    // through shared memory (the ring, which is idle by then), so that all their loads are on their way together.
    // rows: room for kRows pairs.
    __device__ __forceinline__ void join(float *area, float2 *rows, int from, int step, int n, int joined, bool end) const {
        constexpr int kCols = K::kRows * K::kDim / 4, kEach = (kCols + K::kThreads - 1) / K::kThreads;
        const int cols = seg.rows * (K::kDim / 4);
        Joined j[kEach];
        for (int c = 0; c < n; c += K::kJoin) {
            const int here = min(K::kJoin, n - c);
            const uint32_t to = ptx::smem_u32(area) + threadIdx.x * 16;
#pragma unroll 4
            for (int u = 0; u < here; ++u) {
                const float *x = part(from + (c + u) * step) + threadIdx.x * 4;
#pragma unroll
                for (int y = 0; y < kEach; ++y)
                    if ((int)threadIdx.x + y * K::kThreads < cols)
                        copy16(to + u * (K::kStaged * 4) + y * (K::kThreads * 16), x + y * (K::kThreads * 4), true);
                if (threadIdx.x < K::kRows / 2)
                    copy16(to + u * (K::kStaged * 4) + kCols * 16, x + K::kRows * (K::kDim + 2 * joined), true);
            }
            copies_commit();
            copies_wait<0>();
            __syncthreads();
            // A warp takes a row: the maximum, each part's factor (in the place of its maximum) and the sum.
            const int lane = threadIdx.x & 31;
            for (int row = threadIdx.x >> 5; row < seg.rows; row += K::kWarps) {
                float2 *at = reinterpret_cast<float2 *>(area + lane * K::kStaged + kCols * 4) + row;
                const float2 ml = lane < here ? *at : make_float2(-INFINITY, 0.f);
                float top = ml.x;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float f = exp2_approx(ml.x - (top == -INFINITY ? 0.f : top));
                float sum = f * ml.y;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (lane < here) at->x = f;
                if (lane == 0) rows[row] = make_float2(top, sum);
            }
            __syncthreads();
            float4 o[kEach];
#pragma unroll
            for (int y = 0; y < kEach; ++y) o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int u = 0; u < here; ++u) {
                const float *x = area + u * K::kStaged;
#pragma unroll
                for (int y = 0; y < kEach; ++y) {
                    const int i = min((int)threadIdx.x + y * K::kThreads, cols - 1);
                    const float f = reinterpret_cast<const float2 *>(x + kCols * 4)[i / (K::kDim / 4)].x;
                    const float4 v = reinterpret_cast<const float4 *>(x)[i];
                    o[y].x += f * v.x, o[y].y += f * v.y, o[y].z += f * v.z, o[y].w += f * v.w;
                }
            }
#pragma unroll
            for (int y = 0; y < kEach; ++y) {
                const float2 r = rows[min((int)threadIdx.x + y * K::kThreads, cols - 1) / (K::kDim / 4)];
                j[y].take(r.x, r.y, o[y]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int y = 0; y < kEach; ++y) {
            const int i = threadIdx.x + y * K::kThreads, row = i / (K::kDim / 4), d = i % (K::kDim / 4) * 4;
            if (i >= cols || d >= p.c.head_dim) continue;
            if (end) finish(row, d, j[y]);
            else leave(part(from), row, d, j[y], 1);
        }
    }
};

// Partial results are joined by the last CTA to arrive: first in groups of consecutive
// CTAs (when there are many), then over the groups. A CTA is in front of the end of one
// item only, so counters at its number, one for items that begin in it and one for the
// item that does not, are not shared.
template <typename K>
struct Groups {
    int group, of, here, all;  // CTAs of a group, this CTA's group, its CTAs, groups
    __device__ __forceinline__ Groups(const Segment &seg) {
        group = seg.parts;  // one round, if shared memory holds them all
        if (group > K::kJoin) {
            group = min(8, K::kJoin);
            while (group * group < seg.parts) ++group;
        }
        of = ((int)blockIdx.x - seg.c_first) / group;
        here = min(group, seg.parts - of * group);
        all = (seg.parts + group - 1) / group;
    }
};
// Whether this is the last of `n` arrivals. What the CTA's other threads have written
// before a barrier in front of this counts as written before it.
__device__ __forceinline__ bool arrive(unsigned int *counter, int n) {
    unsigned int old;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
    const bool last = old == (unsigned int)n - 1u;
    if (last) *counter = 0u;  // ready for the next call
    return last;
}
template <typename K>
__device__ __forceinline__ bool arrive_for(const Params &p, const Segment &seg) {
    const Groups<K> g(seg);
    return arrive(g.of == 0 ? p.counters + seg.c_first : p.counters + kMaxCtas + seg.c_first + g.of * g.group, g.here);
}
// Joins the CTA's segments that are not whole: the one whose item begins before the CTA
// (for which it has arrived where it ended, if others followed: arrived) and the one
// whose item ends behind it. It arrives for what is left before it joins either: a join
// takes as long as others would wait for the second arrival.
template <typename K, typename T>
__device__ __forceinline__ void join_parts(const Params &p, const Segment *open, bool arrived, bool k8, float *area, float2 *rows, int *last) {
    if (threadIdx.x < 2 && !(threadIdx.x == 0 && arrived)) {
        const Segment seg = open[threadIdx.x];
        last[threadIdx.x] = seg.parts > 1 && arrive_for<K>(p, seg);
    }
    __syncthreads();
#pragma unroll 1
    for (int x = 0; x < 2; ++x) {
        if (!last[x]) continue;
        const Segment seg = open[x];
        const Groups<K> g(seg);
        const Ends<K, T> ends{p, seg, k8 && p.c.v_scale ? p.c.v_scale[seg.kvh] : 1.f};
        // Both rounds go through the same instructions: those of a second copy would come from far away.
#pragma unroll 1
        for (int round = 0; round < 2; ++round) {
            const bool end = round || g.all == 1;
            ends.join(area, rows, round ? 0 : g.of * g.group, round ? g.group : 1, round ? g.all : g.here, round, end);
            if (end) break;
            __syncthreads();
            if (threadIdx.x == 0) last[2] = arrive(p.counters + 2 * kMaxCtas + seg.c_first, g.all);
            __syncthreads();
            if (!last[2]) break;
        }
    }
}

template <typename T, typename C, int DT, int NT>
__global__ void __launch_bounds__(Config<T, C, DT, NT>::kThreads, Config<T, C, DT, NT>::kPerSm) paged_attention_kernel(const __grid_constant__ Params p) {
    using K = Config<T, C, DT, NT>;
    constexpr bool k8 = sizeof(C) == 1;
    using M = typename K::M;
    constexpr float kUp = K::kUp;
    // Weights become one operand of 16 bits and, with 16-bit caches, a second one for what the first's rounding
    // left (together 22 bits of fp16, 16 of bf16): alone it would be as coarse as the output's own rounding. With
    // 8-bit values, whose own rounding is 2^-4, that second product is not spent (104 -> 117 us for 121 requests of
    // 32 heads), but the weights are summed as they are rounded too, so that the output is a mean of the values
    // (104 -> 105 us; error against 64 bits 2.1e-4 to 2.4e-4 in place of 2.5e-4 to 2.9e-4, the plain form's 2.1e-4).
    constexpr bool kTwo = !k8;
    constexpr int kSteps = DT / 16, MT = K::kTok / 16;
    constexpr int kAsk = (kSteps + K::kWarps - 1) / K::kWarps;  // steps whose queries a warp brings
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int sums[K::kWarps];
    __shared__ Segment segs[2], open[2];  // this segment and the next; those that begin before the CTA or end behind it
    __shared__ uint32_t masks[K::kWarps][K::kStages];
    __shared__ float2 meet[K::kWarps][8];  // maxima and sums
    __shared__ int last[3];
    __shared__ float ups[K::kRows];  // what a head's products have to be multiplied by, where that is not 1 (kOwnPower)
    // With launch overlap the next kernel's CTAs come when this one's leave, not earlier: beside these, which fill the
    // SMs' shared memory, they only took SMs in an uneven way (a decoding step of four layers of width 5120: 333 us
    // against 339 with an early signal for 8 requests, 295 against 314 for one).
    ptx::grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x, ctas = gridDim.x;
    const int D = p.c.head_dim;
    const int items = p.c.kv_heads * p.head_blocks;  // of a request

    // Where this CTA's part of the line begins.
    const int per = (p.batch + K::kThreads - 1) / K::kThreads;
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    int mine = 0;  // all tiles are below 2^31: the host has seen to that
    for (int b = b0; b < b1; ++b) mine += tiles_of<K::kTile>(visible(p, b));
    int upto = mine;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, x);
        if (lane >= x) upto += y;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int total = 0;
#pragma unroll
    for (int w = 0; w < K::kWarps; ++w) {
        if (w == warp) upto += total;
        total += sums[w];
    }
    total *= items;
    const int active = min(ctas, total);  // CTAs with work: each has a tile at least
    int t_begin = 0, t_end = 0;           // total * cta / active, in 32 bits
    if (cta < active) {
        const int each = total / active, over = total - each * active;
        t_begin = each * cta + over * cta / active;
        t_end = each * (cta + 1) + over * (cta + 1) / active;
    }
    int before = (upto - mine) * items;
    if (t_begin < t_end && before <= t_begin && t_begin < upto * items) {
        for (int b = b0; b < b1; ++b) {
            const int n = tiles_of<K::kTile>(visible(p, b)) * items;
            if (t_begin < before + n) {
                segs[1].b = b, segs[1].base = before, segs[1].t = t_begin;
                break;
            }
            before += n;
        }
    }
    if (tid < 2) open[tid].parts = 0;
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
    float *mo = reinterpret_cast<float *>(smem + K::kWarps * K::kRing);  // [warp][8][kPitch]
    constexpr int kLanes = K::kChunks < 8 ? K::kChunks : 8;

    // Of the segment whose slices are being loaded: the visible range, slices left, the lane's token of the next
    // slice and where it is, its token of the one after.
    int lo = 0, hi = 0, left = 0;
    const int32_t *table = nullptr;
    const C *kp = nullptr, *vp = nullptr;
    Places ahead{-1, 0u};
    Cursor cur{0, 0u, 0u};
    const unsigned int page_size = (unsigned int)p.c.page_size;
    const unsigned int tile_pages = K::kTile / page_size, tile_rest = K::kTile % page_size;
    uint32_t asked[kAsk][NT][2];

    auto visible_token = [&](int tok) { return tok >= lo && tok < hi; };
    auto look_ahead = [&] {
        ahead.page = visible_token(cur.tok) ? __ldg(table + cur.j) : -1;
        ahead.at = cur.at;
        cur.tok = (int)((unsigned int)cur.tok + K::kTile);
        cur.j += tile_pages, cur.at += tile_rest;
        if (cur.at >= page_size) cur.at -= page_size, ++cur.j;
    };
    auto load_next = [&](int stage) {
        if (left > 0) {
            const Places now = ahead;
            const bool in = visible_token((int)((unsigned int)cur.tok - K::kTile));
            look_ahead();
            const uint32_t mask = load_slice<K, C>(p, now, in, kp, vp, ring + stage * 2 * K::kSliceBytes, lane);
            if (lane == 0) masks[warp][stage] = mask;
            --left;
        }
        copies_commit();
    };
    // Finds the segment after segs[turn ^ 1], which every thread notes in segs[turn] (the same values).
    auto find_segment = [&](int turn) {
        Segment s = segs[turn ^ 1];
        Range r = visible(p, s.b);
        int n = tiles_of<K::kTile>(r);
        while (s.t >= s.base + n * items) {
            s.base += n * items;
            r = visible(p, ++s.b);
            n = tiles_of<K::kTile>(r);
        }
        const int item = (s.t - s.base) / n;
        s.begin = s.base + item * n, s.end = s.begin + n;
        const int seg_end = min(t_end, s.end);
        s.kvh = item / p.head_blocks;
        s.h0 = s.kvh * p.group + (item % p.head_blocks) * K::kRows;
        s.rows = min(K::kRows, (s.kvh + 1) * p.group - s.h0);
        s.count = seg_end - s.t;
        lo = r.lo, hi = r.hi;
        left = s.count;
        // The lane's first token. Tokens behind the last one may lie beyond 31 bits: taken modulo 2^32 they turn
        // negative and so are outside [lo, hi).
        const unsigned int tok =
            (unsigned int)(r.lo / K::kTile + (s.t - s.begin)) * K::kTile + warp * K::kTok + lane % K::kTok;
        cur.tok = (int)tok;
        cur.j = tok / page_size;
        cur.at = tok - cur.j * page_size;
        table = p.table + s.b * p.table_stride;
        kp = static_cast<const C *>(p.c.k) + s.kvh * p.c.k_head + lane / kLanes * p.c.k_token + lane % kLanes * (16 / K::kBytes);
        vp = static_cast<const C *>(p.c.v) + s.kvh * p.c.v_head + lane / kLanes * p.c.v_token + lane % kLanes * (16 / K::kBytes);
        s.t = seg_end;
        segs[turn] = s;
        look_ahead();
    };
    // Queries as the B operand (column n = head lane/4, two k of each half), in shared memory in the order of the
    // lanes: [step][lane][NT][2]. With 8-bit keys the k of a step are taken in the order in which four consecutive
    // bytes of a row come out of the ring. Each warp brings some of the steps: ask_queries() loads them, in front
    // of the keys, so that they do not queue behind them; put_queries() writes them when the area is free.
    auto ask_queries = [&](int turn) {
        const int rows = segs[turn].rows;
        const T *qs = static_cast<const T *>(p.q) + segs[turn].b * p.q_row + segs[turn].h0 * p.q_head;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int head = nt * 8 + lane / 4;
            const T *qh = qs + head * p.q_head;
#pragma unroll
            for (int x = 0; x < kAsk; ++x) {
                const int ks = warp * kAsk + x, k0 = ks * 16 + (k8 ? 4 : 2) * (lane % 4);
                const bool in = ks < kSteps && head < rows && ks * 16 < D && p.scale != 0.f;
                const bool in2 = in && (k8 || ks * 16 + 8 < D);
                asked[x][nt][0] = in ? *reinterpret_cast<const uint32_t *>(qh + k0) : 0u;
                asked[x][nt][1] = in2 ? *reinterpret_cast<const uint32_t *>(qh + k0 + (k8 ? 2 : 8)) : 0u;
            }
        }
    };
    uint32_t *q_area = reinterpret_cast<uint32_t *>(mo);
    constexpr bool kOwnPower = k8 && !std::is_same<T, __half>::value;
    auto put_queries = [&] {
        // A scale of 0 or below turns into queries that are 0 (above) or negated, and a positive scale.
        const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
        [[maybe_unused]] float down[NT];
        if constexpr (kOwnPower) {
            // bf16 queries against 8-bit keys: keys become fp16 (exact), queries fp16 after a power of two that
            // brings their head's largest below 2; what that loses is 2^-25 of the largest.
            static_assert(NT <= 2, "a warp's maxima of two heads lie in one pair");
            float big[2] = {0.f, 0.f};  // of heads lane/4 and 8 + lane/4
#pragma unroll
            for (int x = 0; x < kAsk; ++x)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float2 f = elem::pair_to_f32<T>(asked[x][nt][y]);
                        big[nt] = fmaxf(big[nt], fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                big[nt] = fmaxf(big[nt], __shfl_xor_sync(0xffffffffu, big[nt], 1));
                big[nt] = fmaxf(big[nt], __shfl_xor_sync(0xffffffffu, big[nt], 2));
            }
            if (lane % 4 == 0) meet[warp][lane / 4] = make_float2(big[0], big[1]);
            __syncthreads();
            auto power = [&](int nt, int head) {
                float most = 0.f;
#pragma unroll
                for (int w = 0; w < K::kWarps; ++w) most = fmaxf(most, nt ? meet[w][head].y : meet[w][head].x);
                return most > 0.f && most < INFINITY ? max(ilogbf(most), -120) : 0;
            };
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int e = power(nt, lane / 4);
                down[nt] = ldexpf(1.f, -e);
                ups[nt * 8 + lane / 4] = ldexpf(1.f, e);  // every thread of the head writes the same
            }
        }
#pragma unroll
        for (int x = 0; x < kAsk; ++x)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    asked[x][nt][y] ^= flip;
                    if constexpr (kOwnPower) {
                        const float2 f = elem::pair_to_f32<T>(asked[x][nt][y]);
                        asked[x][nt][y] = elem::pair_from_f32<__half>(f.x * down[nt], f.y * down[nt]);
                    }
                }
                if (warp * kAsk + x < kSteps)
                    *reinterpret_cast<uint2 *>(q_area + ((warp * kAsk + x) * 32 + lane) * (2 * NT) + 2 * nt) =
                        make_uint2(asked[x][nt][0], asked[x][nt][1]);
            }
        __syncthreads();
    };
    auto queries = [&](int ks, uint32_t (&q)[NT][2]) {
        const uint32_t *at = q_area + (ks * 32 + lane) * (2 * NT);
        if constexpr (NT == 1) {
            const uint2 x = *reinterpret_cast<const uint2 *>(at);
            q[0][0] = x.x, q[0][1] = x.y;
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; nt += 2) {
                const uint4 x = *reinterpret_cast<const uint4 *>(at + 2 * nt);
                q[nt][0] = x.x, q[nt][1] = x.y, q[nt + 1][0] = x.z, q[nt + 1][1] = x.w;
            }
        }
    };
    auto fill = [&](int stage) {
#pragma unroll 1
        for (int i = 0; i < K::kStages - 1; ++i) {
            load_next(stage);
            stage = stage + 1 == K::kStages ? 0 : stage + 1;
        }
    };

    int stage = 0, turn = 0;
    bool more = t_begin < t_end, arrived = false;
    if (more) {
        find_segment(turn);
        ask_queries(turn);
        fill(0);
    }
    while (more) {
        float o[kSteps][NT][4];
        // Of the thread's two heads: the reference, the score that moves it, the sum of the weights (of the thread's own
        // rows) and, where they are rounded once, that of what they were rounded to.
        float m[NT][2], limit[NT][2], l[NT][2], rounded[kTwo ? 1 : NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int ks = 0; ks < kSteps; ++ks) o[ks][nt][0] = o[ks][nt][1] = o[ks][nt][2] = o[ks][nt][3] = 0.f;
            m[nt][0] = m[nt][1] = limit[nt][0] = limit[nt][1] = kLowest;  // no token so far
            l[nt][0] = l[nt][1] = 0.f;
            if constexpr (!kTwo) rounded[nt][0] = rounded[nt][1] = 0.f;
        }
        put_queries();
        // Scores in units of log2 are the products times unit().
        constexpr float kLog2e = 1.4426950408889634f;
        const float to_score =
            (p.scale != 0.f ? fabsf(p.scale) : 1.f) * (k8 && p.c.k_scale ? p.c.k_scale[segs[turn].kvh] : 1.f);
        // A unit that is no normal number would be 0 times minus infinity where nothing is visible; the smallest one
        // makes the same of finite scores: all alike.
        auto normal = [](float x) { return x < 1.2e-38f ? 1.2e-38f : x; };
        const float unit_all = p.softcap > 0.f ? 1.f : normal(to_score * kLog2e), slack_all = kSlack / unit_all;
        float units[kOwnPower ? NT : 1][2];
        if constexpr (kOwnPower)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    units[nt][x] = p.softcap > 0.f ? 1.f : normal(to_score * kLog2e * ups[nt * 8 + 2 * (lane % 4) + x]);
        auto unit = [&](int nt, int x) { return kOwnPower ? units[kOwnPower ? nt : 0][x] : unit_all; };
        auto slack = [&](int nt, int x) { return kOwnPower ? kSlack / unit(nt, x) : slack_all; };

        const int count = segs[turn].count;
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
                uint32_t q[k8 ? 2 : 1][NT][2];
#pragma unroll
                for (int x = 0; x < (k8 ? 2 : 1); ++x) queries(ks + x, q[x]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t w[4];
                    ldsm4(w, sk + place<K::kChunks>(mt * 16 + (lane & 15), (k8 ? ks : 2 * ks) + (lane >> 4)));
                    if constexpr (!k8) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma<M>(s[mt][nt], w, q[0][nt][0], q[0][nt][1]);
                    } else {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {  // two steps for each four matrices
                            uint32_t a[4];
                            elem::e4m3x4_to_half2(w[2 * x], a[0], a[2]);
                            elem::e4m3x4_to_half2(w[2 * x + 1], a[1], a[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma<M>(s[mt][nt], a, q[x][nt][0], q[x][nt][1]);
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
                        for (int x = 0; x < 4; ++x)
                            s[mt][nt][x] = out * tanhf(s[mt][nt][x] * (kOwnPower ? in * ups[nt * 8 + 2 * (lane % 4) + (x & 1)] : in));
            }
            if (mask != K::kAll) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        if (!((mask >> (mt * 16 + lane / 4 + (x < 2 ? 0 : 8))) & 1u))
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) s[mt][nt][x] = -INFINITY;
            }
            // Where a score has left the reference far behind, the slice's maximum becomes the new one.
            bool move = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float y = fmaxf(s[0][nt][x], s[0][nt][x + 2]);
#pragma unroll
                    for (int mt = 1; mt < MT; ++mt) y = fmaxf(y, fmaxf(s[mt][nt][x], s[mt][nt][x + 2]));
                    move |= y > limit[nt][x];
                }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float keep[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float y = fmaxf(s[0][nt][x], s[0][nt][x + 2]);
#pragma unroll
                        for (int mt = 1; mt < MT; ++mt) y = fmaxf(y, fmaxf(s[mt][nt][x], s[mt][nt][x + 2]));
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
                        y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
                        y = fmaxf(y, m[nt][x]);
                        keep[x] = exp2_approx((m[nt][x] - y) * unit(nt, x));
                        m[nt][x] = y;
                        limit[nt][x] = y + slack(nt, x);
                        l[nt][x] *= keep[x];
                        if constexpr (!kTwo) rounded[nt][x] *= keep[x];
                    }
#pragma unroll
                    for (int dt = 0; dt < kSteps; ++dt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) o[dt][nt][x] *= keep[x & 1];
                }
            }
            uint32_t ph[MT][NT][2], pl[kTwo ? MT : 1][kTwo ? NT : 1][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x)  // differences first: however large both are, the reference's weight is 2^kUp
                        w[x] = exp2_approx(fmaf(s[mt][nt][x] - m[nt][x & 1], unit(nt, x & 1), kUp));
                    l[nt][0] += w[0] + w[2], l[nt][1] += w[1] + w[3];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        if constexpr (kTwo) {
                            uint32_t h, lo;
                            split(w[2 * x], w[2 * x + 1], h, lo, M());
                            ph[mt][nt][x] = transpose8x8(h), pl[mt][nt][x] = transpose8x8(lo);
                        } else {
                            const uint32_t h = elem::pair_from_f32<M>(w[2 * x], w[2 * x + 1]);
                            ph[mt][nt][x] = transpose8x8(h);
                            const float2 f = elem::pair_to_f32<M>(h);
                            rounded[nt][0] += f.x, rounded[nt][1] += f.y;
                        }
                    }
                }
            // Outputs: 16 elements of the head at a time.
#pragma unroll
            for (int dt = 0; dt < kSteps; dt += k8 ? 2 : 1)
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
                            uint32_t a[4];
                            elem::e4m3x4_to_half2(__byte_perm(w[2 * x], 0, 0x3120), a[0], a[1]);
                            elem::e4m3x4_to_half2(__byte_perm(w[2 * x + 1], 0, 0x3120), a[2], a[3]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma<M>(o[dt + x][nt], a, ph[mt][nt][0], ph[mt][nt][1]);
                        }
                    }
                }
            __syncwarp();  // all lanes have read the stage that is filled next time
            load_next(stage == 0 ? K::kStages - 1 : stage - 1);
            stage = stage + 1 == K::kStages ? 0 : stage + 1;
        }
        // Copied before the warps meet: a warp that has met the others may write segs[turn] again.
        Segment seg = segs[turn];
        seg.c_first = cta, seg.parts = 1;
        if (seg.begin < t_begin || seg.end > t_end) {  // tile x lies with CTA ((x + 1) * active - 1) / total
            seg.c_first = (int)((((long long)seg.begin + 1) * active - 1) / total);
            seg.parts = (int)(((long long)seg.end * active - 1) / total) - seg.c_first + 1;
        }
        if (seg.parts > 1 && tid == 0) open[cta == seg.c_first] = seg;
        // What is loaded from here on belongs to the next segment.
        turn ^= 1;
        more = seg.t < t_end;
        if (more) {
            find_segment(turn);
            ask_queries(turn);
            fill(stage);
        }
        __syncthreads();  // all warps are done with the queries

        // The warps' results meet in shared memory, 8 heads at a time.
        const Ends<K, T> ends{p, seg, k8 && p.c.v_scale ? p.c.v_scale[seg.kvh] : 1.f};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int row = 2 * (lane % 4) + x;
                auto over_rows = [](float y) {
                    y += __shfl_xor_sync(0xffffffffu, y, 4);
                    y += __shfl_xor_sync(0xffffffffu, y, 8);
                    return y + __shfl_xor_sync(0xffffffffu, y, 16);
                };
                const float sum = over_rows(l[nt][x]);
                if (lane < 4) meet[warp][row] = make_float2(m[nt][x] * unit(nt, x), sum);
                if constexpr (!kTwo) {  // from here on outputs belong to the sum of the weights as they were
                    const float of = over_rows(rounded[nt][x]), f = of > 0.f ? sum / of : 1.f;
#pragma unroll
                    for (int dt = 0; dt < kSteps; ++dt) o[dt][nt][x] *= f, o[dt][nt][x + 2] *= f;
                }
#pragma unroll
                for (int dt = 0; dt < kSteps; ++dt) {
                    float *to = mo + (warp * 8 + row) * K::kPitch + dt * 16;
                    to[k8 ? 2 * (lane / 4) : lane / 4] = o[dt][nt][x];
                    to[k8 ? 2 * (lane / 4) + 1 : lane / 4 + 8] = o[dt][nt][x + 2];
                }
            }
            __syncthreads();
#pragma unroll
            for (int i0 = 0; i0 < 8 * (DT / 4); i0 += K::kThreads) {
                const int i = i0 + tid, row = i / (DT / 4), d = i % (DT / 4) * 4;
                if (i >= 8 * (DT / 4) || nt * 8 + row >= seg.rows || d >= D) continue;
                Joined j;
#pragma unroll
                for (int w = 0; w < K::kWarps; ++w) j.m = fmaxf(j.m, meet[w][row].x);
#pragma unroll
                for (int w = 0; w < K::kWarps; ++w) {
                    const float f = exp2_approx(meet[w][row].x - (j.m == -INFINITY ? 0.f : j.m));
                    const float4 x = *reinterpret_cast<const float4 *>(mo + (w * 8 + row) * K::kPitch + d);
                    j.l += f * meet[w][row].y;
                    j.o.x += f * x.x, j.o.y += f * x.y, j.o.z += f * x.z, j.o.w += f * x.w;
                }
                if (seg.parts == 1) ends.finish(nt * 8 + row, d, j);
                else ends.leave(ends.part(cta - seg.c_first), nt * 8 + row, d, j, 0);
            }
            __syncthreads();
        }
        // Arriving takes about a microsecond: worth it here where more than that is still to be streamed (8 requests of
        // 1000 tokens, two tiles for a CTA: 12.4 us with it, 11.9 without; 32 of up to 4000: 52.6 and 54.2).
        if (seg.parts > 1 && cta != seg.c_first && t_end - seg.t >= 4) {
            arrived = true;
            if (tid == 0) last[0] = arrive_for<K>(p, seg);
        }
    }
    copies_wait<0>();
    // The parts that are not whole (the first segment and the last at most) are joined behind the loop, where
    // nothing of it holds registers.
    __syncthreads();
    join_parts<K, T>(p, open, arrived, k8, reinterpret_cast<float *>(smem), meet[0], last);
}

template <typename T, typename C, int DT, int NT>
cudaError_t launch(Params p, int sms, cudaStream_t s) {
    using K = Config<T, C, DT, NT>;
    auto kernel = paged_attention_kernel<T, C, DT, NT>;
    cudaError_t e = ensure_max_dyn_smem((const void *)kernel, K::kSmem);
    if (e != cudaSuccess) return e;
    p.k_page = (unsigned int)p.c.k_page, p.k_token = (unsigned int)p.c.k_token;
    p.v_page = (unsigned int)p.c.v_page, p.v_token = (unsigned int)p.c.v_token;
    p.head_blocks = (p.group + K::kRows - 1) / K::kRows;
    const long long tiles = ((long long)p.max_pages * p.c.page_size + K::kTile - 1) / K::kTile * p.batch *
                            p.c.kv_heads * p.head_blocks;
    const int ctas = sms * K::kPerSm < kMaxCtas ? sms * K::kPerSm : kMaxCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles < ctas ? tiles : ctas), 1, 1);
    cfg.blockDim = dim3(K::kThreads, 1, 1);
    cfg.dynamicSmemBytes = K::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = as_dependent(s) ? 1 : 0;
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
