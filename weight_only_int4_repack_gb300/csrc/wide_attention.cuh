// Attention of many query rows over the pages of a cache: several new tokens of each
// request, or one new token of every request behind a shared prefix (entry points of
// both: prompt_attention.cu).
//     s_j = scale * q . K_j (capped),  out = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m)
// in one pass over the keys, with a running reference m and sum for each row (fp32).
//
// Rows. What reads the same keys is a sequence: a request (its new tokens, each of which
// sees the keys up to its own), or a prefix (the requests behind it, which all see all of
// it). The rows of a sequence and kv head are its tokens times the heads of the group;
// they are taken in tiles of kRows rows, whole tokens each, so that a key that has been
// brought serves the heads of the group and up to kRows / group tokens.
//
// Work. A unit is a tile of rows against kKeys keys. The units of all tiles, kv head after
// kv head, form one line that is cut into equal parts, one for each CTA (one on an SM).
// What a CTA has of a tile is a segment; a tile that lies in several CTAs leaves its sums in
// the workspace, and a second kernel joins them in the order of the keys. Results do not
// depend on timing. (Whole tiles dealt out in turn leave half of the SMs without work where
// there are few rows, and a last round where there are many.)
//
// A CTA. Four warps bring queries, keys and values into the layout of the 128-byte swizzle:
// by boxes of a tensor map where 8 keys or more of a box lie in one page and all rows of the
// warp are visible, otherwise by 16-byte copies, row by row (any page size and order; e4m3
// becomes the operands' type in its place, which is exact). Boxes are issued by the four
// warps, each for its rows (by one warp: 228 us against 222 with 4099 rows). One lane issues
// the matrix products (tcgen05, both operands of Q K^T in shared memory, the weights of P V
// in tensor memory). Two groups of four warps have 128 rows each, a row to a thread: maximum,
// weights, sum, and at the end the output. While the tensor cores work for one group the
// other has its softmax. Heads wider than 128 leave tensor memory for one group; its scores
// are two units ahead instead.
//
// What bounds it. Cycles of a unit of 256 rows and 128 keys with heads of 128, measured in
// the kernel: a group waits about 1100 for its scores and takes about 2600 for the softmax (850
// the maximum, 1000 to 1100 each half of the weights), 3700 together, in which the tensor
// cores have 2170 to do (16 of 128 x 128 x 16 for Q K^T and as many for P V, 64 to 72 each). The softmax
// is bound by issue and by exponentials (8 a cycle and SM partition). Beside the units: 8 us
// until the plan is made and the first scores are there, 4000 cycles at a segment's end for
// the output, 1500 more in a unit with masks. Code is kept small (rolled loops, waits out of
// line): the roles together do not fit the first instruction caches, and what is rarely run
// is fetched anew (an output's first time costs 7500 cycles).
// 4099 rows of 40 heads over 8 kv heads of 128, bf16: 200 us, 0.86 PFLOP/s, 45% of a large
// library product; 16 of it join the tiles that were cut (42 MB of sums, written and read).
// 13 packed prompts behind prefixes, e4m3, 16 heads to a kv head: 333 us, 46%. 4 prompts of
// heads of 256 with a window and a cap: 120 us, 22% (the cap takes 2000 of the 3900 cycles of
// a unit of 128 rows and 64 keys). 64 requests behind 16001 tokens: 97 us, of which 43 are the
// requests' own tokens, 8 the join.
#pragma once

#include <cuda.h>

#include <cmath>
#include <type_traits>

#include "decode_ops.h"
#include "elem.cuh"
#include "ptx.cuh"
#include "tc5.cuh"

namespace w4a16 {
namespace wide {

using elem::E4M3;

constexpr int kMaxSeqs = 8192;      // requests of a call
constexpr int kMaxPrefixes = 2048;  // prefixes of a call
constexpr int kMaxCtas = 256;

// What a CTA's last tile leaves for the kernel that joins (prompts): the parts lie with
// the CTAs from this one on.
struct Cut {
    int parts, rows, q0, h0, kvh, heads, seq, first;
};
// Where a request's sums over its prefix are (prefixes): parts from CTA `first` on, in
// row `row` of each; first < 0: whole, in its own row.
struct Found {
    int first, parts, row, pad;
};

struct Params {
    CUtensorMap q_map, k_map, v_map;  // where q_tma, kv_rows say that they are used
    int q_tma;           // queries of a tile come in one box for each 64 elements (requests)
    int kv_rows;         // keys of a box: they lie in one page; 0: none
    const void *q;
    void *out;
    long long q_row, q_head, o_row, o_head;
    w4a16_kv_cache c;
    const int32_t *table, *lens, *starts;  // starts: nullptr where the sequences are prefixes
    const int32_t *ptable, *plens, *pof;   // nullptr without prefixes
    long long table_stride, ptable_stride;
    int max_pages, pmax_pages, prefixes;
    int rows, batch, heads, group, window;
    float scale, softcap;
    float *lse;
    Cut *cuts;          // [CTAs]
    Found *found;       // [kv heads * head blocks][batch]
    float *slots;       // [2 * CTAs][kRows][kPitch]
    float *whole;       // [batch * heads][kPitch]
    const float *raw, *raw_lse;  // prefixes: the requests' own tokens, [batch * heads][head_dim] and log2 of the sums
    int *odd;           // [CTAs]: whether a CTA has written something that is no finite number
    int ctas;
    int wide_out;       // rows of out are 32-byte aligned
    unsigned int *err;
    unsigned long long wait_ns;
};

// The reference that weights are taken relative to is moved when a score passes it by more
// than kSlack powers of two. As fp16 operands weights are 2^11 at the reference, so that
// they keep 11 bits down to 2^-25 of it; bf16 has the range of fp32.
constexpr float kSlack = 4.f, kLowest = -3.402823466e38f, kLog2e = 1.4426950408889634f;

template <typename T, typename C, int DT>
struct Config {
    static constexpr bool k8 = sizeof(C) == 1;
    using M = typename std::conditional<k8, __half, T>::type;  // operands
    static constexpr bool kB16 = std::is_same<M, __nv_bfloat16>::value;
    static constexpr bool kOwnPower = k8 && std::is_same<T, __nv_bfloat16>::value;  // queries brought to fp16
    static constexpr float kUp = kB16 ? -kSlack : 11.f;
    static constexpr int kDim = DT;                       // head_dim, rounded up
    static constexpr int kTiles = DT > 128 ? 1 : 2;       // groups of 128 rows
    static constexpr int kRows = 128 * kTiles;
    static constexpr int kKeys = DT > 128 ? 64 : 128;     // of a unit
    static constexpr int kAhead = DT > 128 ? 2 : 1;       // units whose scores fit beside the outputs
    static constexpr int kStageBytes = kKeys * DT * 2;    // keys or values of a unit
    static constexpr int kStages = DT == 64 ? 8 : 4;
    static constexpr int kQBytes = 128 * DT * 2;          // queries of a group
    static constexpr int kRing = kTiles * kQBytes;        // offset of the ring
    static constexpr int kAfter = kRing + kStages * kStageBytes;
    static constexpr int kPitch = DT + 8;                 // floats of a row of sums: outputs, then m, l
    static constexpr int kSlot = kRows * kPitch;
    // Tensor memory: kAhead units' scores of each group (weights take their place), and its outputs.
    static constexpr int kO = 256, kOStep = 128, kSStep = 128, kSBuffer = 64;
    static constexpr int kWeights = kKeys == 128 ? 64 : 0;  // where weights begin in their scores' place
    static_assert(kAhead * kKeys <= kSStep, "scores lie in front of the outputs");
    static constexpr int kWarps = 4 * kTiles + 8, kThreads = 32 * kWarps;
    static constexpr int kLoader = 4 * kTiles, kMma = kLoader + 4;  // first warps of the roles
};

constexpr int kQueue = 4;  // segments that are described ahead
constexpr int kOver = 2;   // units that a tile's beginning and end cost, about
// A segment, as the scheduling warp describes it to the others.
struct Segment {
    int rows, heads;     // of the tile that are real; heads of a token
    int q0;              // row of q of the tile's first token (requests)
    int first;           // visible keys of the tile's first token; each further token sees one more (requests)
    int total;           // keys of the sequence
    int kvh, h0;         // kv head, first query head
    int key0, count;     // first key, units
    int lo, hi;          // keys that some row sees
    int own0, gap;       // keys of the prefix in front of the request's own; numbers between them that are no keys
    const int32_t *own_pages, *pre_pages;
    int slot;            // where the sums go; -1: the tile is whole
    int last;            // no segment follows
};

template <int kRows>
struct Shared {
    int counts[kMaxPrefixes], least[kMaxPrefixes];  // of each prefix: requests, shortest own length
    int members[kQueue][kRows];                     // requests of a tile (prefixes)
    float powers[kQueue][kRows];                    // what a row's scores have to be multiplied by (kOwnPower)
    uint32_t bad[16][4];                            // keys of a unit whose page is none
    Segment segs[kQueue];
    // Barriers: tiles of the ring there and free; segments; of each group (and place) scores there, weights of the first 64
    // keys and all weights there, a unit's product added, the last one's; queries there and free; the end after an abort.
    uint64_t full[8], empty[8], seg_full[kQueue], seg_empty[kQueue], s_full[2][2], p_half[2], p_full[2][2], o_step[2], o_full[2],
        q_full, q_empty, drain;
    int sums[32];
    int start_s, start_t, start_hd, start_base, tiles, work;
    uint32_t tmem;
    int abort, odd, begun[2];
};

// ------------------------------------------------------------------ sequences and tiles
struct Seq {
    int n;       // tokens (requests: new ones; prefixes: requests behind it)
    int total;   // keys
    int q0;      // first row of q (requests)
    int own0;    // requests: tokens in front of the own ones
    int pre;     // requests: the prefix, -1: none
};
__device__ __forceinline__ int clamp_len(int len, int pages, int page_size) {
    const long long most = (long long)pages * page_size;
    return (int)min((long long)max(len, 0), most);
}
// The prefix of request b, or -1; *none: the number was neither a prefix nor negative.
__device__ __forceinline__ int prefix_of(const Params &p, int b, bool *none) {
    if (!p.pof) return -1;
    const int x = p.pof[b];
    if (x >= p.prefixes) *none = true;
    return x >= 0 && x < p.prefixes ? x : -1;
}
static __device__ __noinline__ Seq request(const Params &p, int b, bool report) {
    Seq s;
    const int from = p.starts[b], to = p.starts[b + 1], len = p.lens[b];
    bool bad = from < 0 || to < from || to > p.rows;
    s.n = bad ? 0 : to - from;
    s.q0 = from;
    const int own = clamp_len(len, p.max_pages, p.c.page_size);
    bad |= own != len || own < s.n;
    s.pre = prefix_of(p, b, &bad);
    s.own0 = 0;
    if (s.pre >= 0) {
        s.own0 = clamp_len(p.plens[s.pre], p.pmax_pages, p.c.page_size);
        bad |= s.own0 != p.plens[s.pre];
    }
    s.total = s.own0 + own;
    if (bad && report) atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG);
    return s;
}
// Whether request b is one of a prefix's (has a prefix and a token of its own).
__device__ __forceinline__ bool behind(const Params &p, int b, int prefix) {
    return p.pof[b] == prefix && p.lens[b] > 0;
}

// Keys are numbered with a gap between a request's prefix and its own, up to the next unit's first one: so that units, and
// the blocks of keys in them, begin where pages do.
template <typename K>
__device__ __forceinline__ int gap_of(int own0) {
    return -own0 & (K::kKeys - 1);
}
__device__ __forceinline__ int placed_from(int j, int own0, int gap) { return j >= own0 ? j + gap : j; }
__device__ __forceinline__ int placed_to(int j, int own0, int gap) { return j > own0 ? j + gap : j; }

// A tile of a sequence: its tokens, the keys that any of them sees (as numbered with the gap), its units.
struct Tile {
    int tok0, toks, first, lo, hi, key0, count;
};
template <typename K>
__device__ __noinline__ Tile tile_of(const Params &p, const Seq &s, int least, int tt, int t) {
    Tile x;
    x.tok0 = t * tt;
    x.toks = min(tt, s.n - x.tok0);
    if (p.starts) {
        x.first = s.total - s.n + x.tok0 + 1;
        x.hi = max(x.first + x.toks - 1, 0);
        x.lo = p.window > 0 ? max(0, max(x.first, 0) - p.window) : 0;  // (rows in front of the first token see none: below 0)
        const int gap = gap_of<K>(s.own0);
        x.hi = placed_to(x.hi, s.own0, gap), x.lo = placed_from(x.lo, s.own0, gap);
    } else {
        x.first = 0;
        x.hi = s.total;
        x.lo = p.window > 0 ? (int)max(0ll, (long long)s.total + least - p.window) : 0;
    }
    x.key0 = 0, x.count = 1;
    if (x.lo < x.hi) {
        x.key0 = x.lo / K::kKeys * K::kKeys;
        x.count = (x.hi - 1) / K::kKeys + 1 - x.lo / K::kKeys;
    }
    return x;
}

// Sum over the threads in front of this one, and over all.
template <int kWarps>
__device__ __forceinline__ int scan(int mine, int *sums, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += sums[w];
        all += sums[w];
    }
    *total = all;
    return before + upto - mine;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool real) {
    const int n = real ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy16_all(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(ptx::smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// ptx::mbar_wait for all lanes of a warp alike. What comes after the first try is kept out of the way of the instruction
// caches, once for all calls.
static __device__ __noinline__ bool wait_longer(uint64_t *bar, uint32_t parity, volatile int *abort_flag, unsigned int *err,
                                                uint64_t limit_ns) {
    const uint64_t since = ptx::globaltimer();
    bool over = limit_ns == 0;
#pragma unroll 1
    for (;;) {
        if (over && err) atomicExch(err, (unsigned int)W4A16_ERR_TIMEOUT);
        if (over) *abort_flag = 1;
        if (__any_sync(0xffffffffu, over || *abort_flag)) return false;
        if (__all_sync(0xffffffffu, ptx::mbar_try_wait_sleep(bar, parity, 20000u))) return true;
        over = ptx::globaltimer() - since >= limit_ns;
    }
}
__device__ __forceinline__ bool wait_on(uint64_t *bar, uint32_t parity, volatile int *abort_flag, unsigned int *err, uint64_t limit_ns) {
    return __all_sync(0xffffffffu, ptx::mbar_try_wait_sleep(bar, parity, 20000u)) || wait_longer(bar, parity, abort_flag, err, limit_ns);
}

// The same value in all lanes, so that the compiler knows it.
__device__ __forceinline__ int uniform(int x) { return (int)__reduce_or_sync(0xffffffffu, (unsigned)x); }

// One lane of the warp, always the same: matrix instructions are issued by it, and the compiler knows that it is one.
__device__ __forceinline__ bool elect() {
    uint32_t x;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(x));
    return x != 0;
}
// A box of a tensor map into shared memory.
__device__ __forceinline__ void load_box(void *dst, const CUtensorMap *map, int x, int y, int z, int w, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
            ptx::smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(ptx::smem_u32(bar))
        : "memory");
}
// 32 bytes, 32-byte aligned.
__device__ __forceinline__ void store8(float *to, const float *x) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                 "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
}

// Two at a time.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}

// A score in units of log2 is a raw product times this. A scale of 0 or below is in the queries (none, or negated); a unit
// that is no normal number would be 0 times minus infinity where nothing is visible.
__device__ __forceinline__ float unit_of(const Params &p, float k_scale) {
    return fmaxf((p.scale != 0.f ? fabsf(p.scale) : 1.f) * k_scale * kLog2e, 1.2e-38f);
}

// How a raw product becomes a score, in units of log2.
struct Scores {
    float unit;            // without a cap: score * log2(e) of a product
    float in, cap;         // with one: 2 * log2(e) / softcap * scale, softcap * log2(e) (no more than 1e30: sums and products of it
                           // stay finite, and what it would take off lower scores is not seen)
    float slack;           // kSlack powers of two, as a difference of products
    bool capped;
    __device__ __forceinline__ Scores(const Params &p, float k_scale) {
        const float to_score = (p.scale != 0.f ? fabsf(p.scale) : 1.f) * k_scale;
        unit = unit_of(p, k_scale);
        capped = p.softcap > 0.f;
        const float most = fminf(p.softcap, 1e30f);
        in = capped ? fminf(2.f * kLog2e * to_score / most, 3e38f) : 0.f;  // (0 times it is 0)
        cap = most * kLog2e;
        slack = kSlack / unit;
    }
    // cap * tanh(x), 2x the exponent of e that `in` gives as one of 2.
    static __device__ __forceinline__ float squeezed(float s, float in, float cap) { return cap * tanhf(s * (in * 0.34657359f)); }
    __device__ __forceinline__ float squeezed(float s) const { return squeezed(s, in, cap); }
    // What a reference m is as a score.
    __device__ __forceinline__ float of(float m) const { return capped ? squeezed(m) : m * unit; }
};

// A cap up to here is taken by 1 - 2 / (1 + e^2x), which is off by 2^-22 of the cap: less than 2^-15 in a score, where an
// operand's weight has 2^-11. Above it that would be seen, and scores that a large cap leaves as they are would be lost in it.
constexpr float kQuickCap = 128.f * kLog2e;
// 32 columns of scores with a larger cap, in their place. (Out of line: caps are smaller, as a rule.)
static __device__ __noinline__ void squeeze_in_place(uint32_t at, float in, float cap) {
    uint32_t v[32];
    tc5::ld32(at, v);
    tc5::wait_ld();
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(Scores::squeezed(__uint_as_float(v[i]), in, cap));
    tc5::st32(at, v);
    tc5::wait_st();
}

// ------------------------------------------------------------------ the kernel
template <typename T, typename C, int DT>
__global__ void __launch_bounds__(Config<T, C, DT>::kThreads, 1) wide_kernel(const __grid_constant__ Params p) {
    using K = Config<T, C, DT>;
    using Sh = Shared<K::kRows>;
    constexpr int kTiles = K::kTiles, kKeys = K::kKeys, kStages = K::kStages;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    Sh &sh = *reinterpret_cast<Sh *>(smem + K::kAfter);
    volatile int *abort_flag = &sh.abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
    const int cta = blockIdx.x;
    const int D = p.c.head_dim;

    if (tid == 0) {
#pragma unroll 1
        for (int i = 0; i < kStages; ++i) ptx::mbar_init(&sh.full[i], 4), ptx::mbar_init(&sh.empty[i], 1);
#pragma unroll 1
        for (int i = 0; i < kQueue; ++i) ptx::mbar_init(&sh.seg_full[i], 1), ptx::mbar_init(&sh.seg_empty[i], 4 * kTiles + 5);
#pragma unroll 1
        for (int i = 0; i < 2; ++i)
            ptx::mbar_init(&sh.p_half[i], 4), ptx::mbar_init(&sh.o_step[i], 1), ptx::mbar_init(&sh.o_full[i], 1);
#pragma unroll 1
        for (int i = 0; i < 4; ++i) ptx::mbar_init(&sh.s_full[i >> 1][i & 1], 1), ptx::mbar_init(&sh.p_full[i >> 1][i & 1], 4);
        ptx::mbar_init(&sh.q_full, 4), ptx::mbar_init(&sh.q_empty, 1), ptx::mbar_init(&sh.drain, 1);
        sh.abort = 0, sh.odd = 0, sh.work = 0, sh.begun[0] = sh.begun[1] = 0;
        ptx::mbar_init_fence();
    }
    if (warp == K::kMma) tc5::alloc(&sh.tmem, 512);
    ptx::grid_dep_wait();

    // ---------------------------------------------------------------- plan
    const int gb = min(p.group, K::kRows), head_blocks = (p.group + gb - 1) / gb, tt = K::kRows / gb;
    const int hds = p.c.kv_heads * head_blocks;
    const int seqs = p.starts ? p.batch : p.prefixes;
    int *plan_off = reinterpret_cast<int *>(smem), *plan_n = plan_off + seqs + 1, *plan_total = plan_n + seqs, *plan_own = plan_total + seqs;
    if (!p.starts) {
#pragma unroll 1
        for (int i = tid; i < seqs; i += K::kThreads) sh.counts[i] = 0, sh.least[i] = 0x7fffffff;
        __syncthreads();
#pragma unroll 1
        for (int b = tid; b < p.batch; b += K::kThreads) {
            bool bad = false;
            const int x = prefix_of(p, b, &bad), len = p.lens[b], own = clamp_len(len, p.max_pages, p.c.page_size);
            if (x >= 0 && len > 0) atomicAdd(&sh.counts[x], 1), atomicMin(&sh.least[x], own);
            if (bad && cta == 0) atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG);
        }
        __syncthreads();
    }
    auto seq_of = [&](int i, bool report) {
        if (p.starts) return request(p, i, report);
        Seq s{sh.counts[i], clamp_len(p.plens[i], p.pmax_pages, p.c.page_size), 0, 0, i};
        if (report && s.total != p.plens[i]) atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG);
        return s;
    };
    {
        const int per = (seqs + K::kThreads - 1) / K::kThreads, s0 = min(tid * per, seqs), s1 = min(s0 + per, seqs);
        int mine = 0, all = 0;
#pragma unroll 1
        for (int i = s0; i < s1; ++i) {
            const Seq s = seq_of(i, cta == 0);
            plan_n[i] = s.n, plan_total[i] = s.total, plan_own[i] = s.own0;
            mine += (s.n + tt - 1) / tt;
        }
        int at = scan<K::kWarps>(mine, sh.sums, &all);
#pragma unroll 1
        for (int i = s0; i < s1; ++i) {
            plan_off[i] = at;
            at += (plan_n[i] + tt - 1) / tt;
        }
        // Requests whose rows overlap (starts that fall) may have more tiles than the host has counted with: nothing is done.
        const bool many = all > p.rows / tt + seqs;
        if (many && cta == 0 && tid == 0) atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG);
        if (tid == 0) plan_off[seqs] = all, sh.tiles = many ? 0 : all;
    }
    __syncthreads();
    int total_units = 0, t_begin = 0, t_end = 0;  // below 2^31: the host has seen to that
    int active, over;
    {
        const int tiles = sh.tiles;
        const int per = (tiles + K::kThreads - 1) / K::kThreads, i0 = min(tid * per, tiles), i1 = min(i0 + per, tiles);
        int s_first = 0;
        if (i0 < i1) {  // the sequence of the thread's first tile: the last one that begins at or in front of it
            int lo = 0, hi = seqs - 1;
#pragma unroll 1
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (plan_off[mid] <= i0) lo = mid;
                else hi = mid - 1;
            }
            s_first = lo;
        }
        auto units_of = [&](int s, int i) {
            const Seq q{plan_n[s], plan_total[s], 0, plan_own[s], 0};
            return tile_of<K>(p, q, p.starts ? 0 : sh.least[s], tt, i - plan_off[s]).count;
        };
        int mine = 0, per_hd = 0;
#pragma unroll 1
        for (int i = i0, s = s_first; i < i1; ++i) {
#pragma unroll 1
            while (i >= plan_off[s + 1]) ++s;
            mine += units_of(s, i);
        }
        int before = scan<K::kWarps>(mine, sh.sums, &per_hd);
        // A tile costs about as much as kOver units besides (queries, a first and a last unit that nothing overlaps,
        // outputs): where CTAs have several tiles the line counts them, in front of the tile's own units.
        over = per_hd * hds >= 8 * (int)gridDim.x ? kOver : 0;
        before += over * i0, mine += over * (i1 - i0), per_hd += over * tiles;
        total_units = per_hd * hds;
        active = min((int)gridDim.x, total_units);
        if (cta < active) {
            const int each = total_units / active, rest = total_units - each * active;
            t_begin = each * cta + rest * cta / active;
            t_end = each * (cta + 1) + rest * (cta + 1) / active;
            const int hd = t_begin / per_hd, rem = t_begin - hd * per_hd;
            if (rem >= before && rem < before + mine) {
                int at = before;
#pragma unroll 1
                for (int i = i0, s = s_first; i < i1; ++i) {
#pragma unroll 1
                    while (i >= plan_off[s + 1]) ++s;
                    const int n = units_of(s, i) + over;
                    if (rem < at + n) {
                        const int base = t_begin - rem + at, end = min(base + n, t_end);
                        sh.start_s = s, sh.start_t = i - plan_off[s], sh.start_hd = hd, sh.start_base = base;
                        sh.work = end > max(t_begin, base + over) || t_end - (base + n) > over;
                        break;
                    }
                    at += n;
                }
            }
        }
    }
    // The plan has been written and read by ordinary accesses where boxes of tensor maps are written next.
    fence_async();
    tc5::fence_before();
    __syncthreads();
    tc5::fence_after();
    const uint32_t tmem = uniform(sh.tmem);
    const int gb_inv = (65535 + gb) / gb;  // x * gb_inv >> 16 is x / gb for all rows of a tile
    const bool has_work = cta < active && sh.work;
    const uint32_t q_base = ptx::smem_u32(smem), ring = q_base + K::kRing;
    const int k_steps = (D + 15) / 16;

    if (warp >= K::kLoader && warp < K::kMma) {
        // ------------------------------------------------------------ loaders
        const int w = warp - K::kLoader;
        bool ok = true, last = !has_work;
        int stage = 0, unit_n = 0, tiles_n = 0, queries_n = 0;  // tiles of the ring and of queries that are on their way or there
        uint32_t ring_phase = 1;  // of the empty barriers
        constexpr int kMine = kKeys / 4;  // rows of a warp
        // e4m3 to fp16, a few rows at a time: what lies in their own place is read before it is overwritten.
        [[maybe_unused]] auto widen = [&](uint32_t at) {
            constexpr int kChunks = DT / 16, kAt = 32 / kChunks, kOnce = kMine / kAt < 4 ? kMine / kAt : 4;
            const int c = lane % kChunks, r0 = lane / kChunks, c0 = (2 * c) & 7;
            const uint32_t row = at + (w * kMine + r0) * 128;
            const uint32_t from = row + (DT / 64 - (kChunks + 7) / 8 + (c >> 3)) * (kKeys * 128) + ((c & 7) << 4);
            const uint32_t to = row + (c >> 2) * (kKeys * 128);
            __syncwarp();
#pragma unroll 1
            for (int i0 = 0; i0 < kMine / kAt; i0 += kOnce) {
                uint4 y[kOnce];
#pragma unroll
                for (int i = 0; i < kOnce; ++i)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(y[i].x), "=r"(y[i].y), "=r"(y[i].z), "=r"(y[i].w)
                                 : "r"(from + (i0 + i) * kAt * 128) : "memory");
                __syncwarp();
#pragma unroll
                for (int i = 0; i < kOnce; ++i) {
                    const int turn = ((i0 + i) * kAt + r0) & 7;
                    uint32_t h[8];
                    elem::e4m3x4_to_half2(y[i].x, h[0], h[1]);
                    elem::e4m3x4_to_half2(y[i].y, h[2], h[3]);
                    elem::e4m3x4_to_half2(y[i].z, h[4], h[5]);
                    elem::e4m3x4_to_half2(y[i].w, h[6], h[7]);
                    const uint32_t row_to = to + (i0 + i) * kAt * 128;
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row_to + ((c0 ^ turn) << 4)), "r"(h[0]), "r"(h[1]),
                                 "r"(h[2]), "r"(h[3])
                                 : "memory");
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row_to + (((c0 + 1) ^ turn) << 4)), "r"(h[4]), "r"(h[5]),
                                 "r"(h[6]), "r"(h[7])
                                 : "memory");
                }
            }
        };
        // Copies on their way, oldest first: the barriers that wait for them.
        constexpr int kLag = 2;
        uint64_t *pend[kLag + 1];
        int pending = 0;
        auto signal = [&](uint64_t *bar) {
            if constexpr (K::k8)
                if (bar != &sh.q_full) widen(ring + (uint32_t)(bar - sh.full) * K::kStageBytes);
            fence_async();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar);
        };
        auto drain = [&] {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
            for (int i = 0; i < kLag + 1; ++i)
                if (i < pending) signal(pend[i]);
            pending = 0;
        };
        auto queue = [&](uint64_t *bar) {
            asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
            for (int i = 0; i < kLag + 1; ++i)
                if (i == pending) pend[i] = bar;
            if (++pending == kLag + 1) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kLag) : "memory");
                signal(pend[0]);
#pragma unroll
                for (int i = 0; i < kLag; ++i) pend[i] = pend[i + 1];
                pending = kLag;
            }
        };
        // Waits; what is on its way is signalled first, as others may need it to come to an end.
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (!__all_sync(0xffffffffu, mbar_test(bar, parity))) {
                drain();
                ok = wait_on(bar, parity, abort_flag, p.err, p.wait_ns);
            }
            return ok;
        };
#pragma unroll 1
        for (int n = 0; ok && !last; ++n) {
            const int qi = n % kQueue;
            if (!wait(&sh.seg_full[qi], (uint32_t)(n / kQueue) & 1u)) break;
            const Segment &g = sh.segs[qi];  // stays as it is until this warp has been counted at the segment's end
            last = g.last;
            // Queries, in the order of the rows.
            if (!wait(&sh.q_empty, (uint32_t)(n + 1) & 1u)) break;
            if (!K::kOwnPower && p.q_tma) {
                // A box holds the tile's rows in their order: heads of a token, token after token. Rows behind the request's last
                // one are others' or zero, or what lay there before: they have no part in what the tile's own rows get.
                if (w == 0 && elect()) {
                    ptx::mbar_arrive_expect_tx(&sh.q_full, (uint32_t)(tt * gb * DT * 2));
                    for (int i = 0; i < DT / 64; ++i)
                        load_box(smem + i * (K::kRows * 128), &p.q_map, i * 64, g.h0, g.q0, 0, &sh.q_full);
                } else if (w > 0 && lane == 0) {
                    ptx::mbar_arrive(&sh.q_full);
                }
                __syncwarp();
            } else {
                constexpr int kChunks = DT / 8, kLanes = kChunks < 32 ? kChunks : 32, kAt = 32 / kLanes;
                const int c = lane % kLanes, rows = g.rows;
#pragma unroll 1
                for (int r0 = w * (K::kRows / 4); r0 < (w + 1) * (K::kRows / 4) && r0 < (rows + 127) / 128 * 128; r0 += 32) {
                    const int r = r0 + lane, tk = r * gb_inv >> 16, hh = r - tk * gb;
                    const bool in = r < rows && hh < g.heads && p.scale != 0.f;
                    const long long row = !in ? 0 : p.starts ? g.q0 + tk : sh.members[qi][tk];
                    const long long at = in ? row * p.q_row + (g.h0 + hh) * p.q_head : -1;
                    // Several rows at a time: their places and, where they pass through registers, all their loads come first.
                    constexpr int kOnce = K::kOwnPower && 8 * kAt <= 32 ? 8 : 4;
#pragma unroll 1
                    for (int i0 = 0; i0 < 32; i0 += kOnce * kAt) {
                        long long srcs[kOnce];
                        [[maybe_unused]] uint4 ys[kOnce];
#pragma unroll
                        for (int z = 0; z < kOnce; ++z) srcs[z] = __shfl_sync(0xffffffffu, at, i0 + z * kAt + lane / kLanes);
                        if constexpr (K::kOwnPower)
#pragma unroll
                            for (int z = 0; z < kOnce; ++z)
                                ys[z] = srcs[z] >= 0 && c * 8 < D ? __ldcg(reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q) + srcs[z] + c * 8))
                                                                  : make_uint4(0, 0, 0, 0);
#pragma unroll
                        for (int z = 0; z < kOnce; ++z) {
                            const int rr = r0 + i0 + z * kAt + lane / kLanes;
                            const uint32_t to = q_base + (c >> 3) * (K::kRows * 128) + rr * 128 + (((c & 7) ^ (rr & 7)) << 4);
                            if constexpr (!K::kOwnPower) {
                                const bool real = srcs[z] >= 0 && c * 8 < D;
                                if (c * 8 < 16 * k_steps) copy16(to, static_cast<const T *>(p.q) + (real ? srcs[z] + c * 8 : 0), real);
                            } else {
                                // To fp16, after a power of two that brings the row's largest below 2 (of the largest numbers:
                                // below 4): what that loses is 2^-25 of the largest.
                                const uint32_t w4[4] = {ys[z].x, ys[z].y, ys[z].z, ys[z].w};
                                float big = 0.f;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float2 f = elem::pair_to_f32<T>(w4[e]);
                                    big = fmaxf(big, fmaxf(fabsf(f.x), fabsf(f.y)));
                                }
#pragma unroll
                                for (int o = 1; o < kLanes; o <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
                                const int e2 = big > 0.f && big < INFINITY ? min(max((int)(__float_as_uint(big) >> 23) - 127, -120), 126) : 0;
                                const float down = __uint_as_float((uint32_t)(127 - e2) << 23);
                                uint32_t h[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float2 f = elem::pair_to_f32<T>(w4[e]);
                                    h[e] = elem::pair_from_f32<__half>(f.x * down, f.y * down);
                                }
                                if (c == 0) sh.powers[qi][rr] = __uint_as_float((uint32_t)(127 + e2) << 23);
                                if (c * 8 < 16 * k_steps)
                                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3])
                                                 : "memory");
                            }
                        }
                    }
                }
                if constexpr (K::kOwnPower) signal(&sh.q_full);
                else queue(&sh.q_full);
            }
            ++queries_n;
            // Keys and values, unit after unit.
            const int take = g.count, kvh = g.kvh;
            const bool boxes = p.kv_rows > 0;  // a box's keys lie in one page
            const bool blocks = p.c.page_size % 16 == 0 && D == DT;  // 16 keys lie in one page
            auto look_up = [&](int u, int &page, int &at, bool &in, bool &none) {
                const int j = g.key0 + u * kKeys + w * kMine + lane % kMine, own0 = g.own0;
                in = j >= g.lo && j < g.hi;
                none = j >= own0 && j < own0 + g.gap;
                in = in && !none;
                page = -1, at = 0;
                if (in) {
                    const bool pre = j < own0;
                    const unsigned int y = pre ? j : j - own0 - g.gap, n = y / (unsigned int)p.c.page_size;
                    at = (int)(y - n * (unsigned int)p.c.page_size);
                    page = __ldcg((pre ? g.pre_pages : g.own_pages) + n);  // (written by the kernel in front, as a rule: not through the read-only path)
                }
            };
            // Keys run kAhead units ahead of the values, as the products that need them do. A unit's places are looked up when its
            // keys are brought, and kept for its values.
            int page, at;
            bool in, none;
            look_up(0, page, at, in, none);
            int v_page[K::kAhead + 1] = {}, v_at[K::kAhead + 1] = {};
            uint32_t v_rows[K::kAhead + 1] = {};
#pragma unroll 1
            for (int u = 0; ok && u < take + K::kAhead; ++u) {
                uint32_t bad = 0;
                if (u < take) {
                    const bool good = in && page >= 0 && page < p.c.pages;
                    bad = __ballot_sync(0xffffffffu, none || (in && !good));
                    if (in && !good) atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG);
                    v_rows[K::kAhead] = __ballot_sync(0xffffffffu, good);
                    v_page[K::kAhead] = good ? page : 0, v_at[K::kAhead] = good ? at : 0;
                    if (u + 1 < take) look_up(u + 1, page, at, in, none);
                }
#pragma unroll 1
                for (int side = 0; side < 2; ++side) {  // keys of unit u, values of unit u - kAhead
                    if (side ? u < K::kAhead : u >= take) continue;
                    if (!wait(&sh.empty[stage], ring_phase)) break;
                    if (side == 0) {
                        if (lane == 0) sh.bad[unit_n & 15][w] = kMine == 32 ? bad : bad & 0xffffu;
                        ++unit_n;
                    }
                    const uint32_t good_rows = side ? v_rows[0] : v_rows[K::kAhead];
                    const int my_page = side ? v_page[0] : v_page[K::kAhead], my_at = side ? v_at[0] : v_at[K::kAhead];
                    const uint32_t all = kMine == 32 ? 0xffffffffu : 0xffffu;
                    const uint32_t dst = ring + stage * K::kStageBytes;
                    if (!K::k8 && boxes && (good_rows & all) == all) {  // as a rule
                        if (lane == 0) ptx::mbar_arrive_expect_tx(&sh.full[stage], (uint32_t)(kMine * DT * 2));
                        __syncwarp();
#pragma unroll 1
                        for (int i = 0; i < kMine; i += p.kv_rows) {
                            const int box_page = __shfl_sync(0xffffffffu, my_page, i), box_at = __shfl_sync(0xffffffffu, my_at, i);
                            if (elect()) {
                                unsigned char *to = smem + K::kRing + stage * K::kStageBytes + (w * kMine + i) * 128;
#pragma unroll
                                for (int z = 0; z < DT / 64; ++z)
                                    load_box(to + z * (kKeys * 128), side ? &p.v_map : &p.k_map, z * 64, box_at, kvh, box_page, &sh.full[stage]);
                            }
                        }
                        __syncwarp();
                    } else {
                        const C *pool = static_cast<const C *>(side ? p.c.v : p.c.k) + kvh * (side ? p.c.v_head : p.c.k_head);
                        const unsigned long long off = my_page * (unsigned long long)(side ? p.c.v_page : p.c.k_page) +
                                                       my_at * (unsigned long long)(side ? p.c.v_token : p.c.k_token);
                        // A chunk is 16 bytes of a row. 8-bit rows wait in the last blocks of their own place until they are widened.
                        constexpr int kChunks = DT * (int)sizeof(C) / 16, kLanes = kChunks < 32 ? kChunks : 32, kAt = 32 / kLanes;
                        const int c = lane % kLanes, r0 = lane / kLanes;
                        const C *from = pool + c * (16 / (int)sizeof(C));
                        const uint32_t to = dst + ((c >> 3) + (K::k8 ? DT / 64 - (kChunks + 7) / 8 : 0)) * (kKeys * 128) + (w * kMine + r0) * 128;
                        auto turned = [&](int i) { return (uint32_t)((c & 7) ^ (K::k8 ? 0 : (i + r0) & 7)) << 4; };
                        if ((good_rows & all) == all && blocks) {  // as a rule
                            const unsigned long long token = side ? p.c.v_token : p.c.k_token;
                            const C *row = from + r0 * token;
    #pragma unroll 1
                            for (int i0 = 0; i0 < kMine; i0 += 16) {
                                const C *at_row = row + __shfl_sync(0xffffffffu, off, i0);
    #pragma unroll
                                for (int i = 0; i < 16; i += kAt) {
                                    copy16_all(to + (i0 + i) * 128 + turned(i), at_row);
                                    at_row += kAt * token;
                                }
                            }
                        } else {
    #pragma unroll 1
                            for (int i = 0; i < kMine; i += kAt) {
                                const unsigned long long src = __shfl_sync(0xffffffffu, off, i + r0);
                                const bool there = ((good_rows >> (i + r0)) & 1u) && c * (16 / (int)sizeof(C)) < D;
                                if (c * (16 / (int)sizeof(C)) < 16 * k_steps) copy16(to + i * 128 + turned(i), there ? from + src : pool, there);
                            }
                        }
                        queue(&sh.full[stage]);
                    }
                    ++tiles_n;
                    if (++stage == kStages) stage = 0, ring_phase ^= 1u;
                }
#pragma unroll
                for (int i = 0; i < K::kAhead; ++i) v_page[i] = v_page[i + 1], v_at[i] = v_at[i + 1], v_rows[i] = v_rows[i + 1];
            }
            if (!ok) break;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sh.seg_empty[qi]);
        }
        drain();
        asm volatile("cp.async.wait_all;" ::: "memory");
        // Nothing may be on its way when the CTA ends. After a wait that ran out the warps may have stopped at different
        // tiles: each one arrives for those that others have begun, so that what is on its way for them can be waited for.
        if (lane == 0) atomicMax(&sh.begun[0], tiles_n), atomicMax(&sh.begun[1], queries_n);
        ptx::named_bar_sync(1, 128);
        const int tiles_all = *(volatile int *)&sh.begun[0], queries_all = *(volatile int *)&sh.begun[1];
        if (lane == 0) {
            volatile int no_abort = 0;
#pragma unroll 1
            for (int i = tiles_n; i < tiles_all; ++i) ptx::mbar_arrive(&sh.full[i % kStages]);
            if (queries_n < queries_all) ptx::mbar_arrive(&sh.q_full);
#pragma unroll 1
            for (int i = max(tiles_all - kStages, 0); i < tiles_all; ++i)
                ptx::mbar_wait(&sh.full[i % kStages], (uint32_t)(i / kStages) & 1u, &no_abort, nullptr, 200000000ull);
            if (queries_all > 0) ptx::mbar_wait(&sh.q_full, (uint32_t)(queries_all - 1) & 1u, &no_abort, nullptr, 200000000ull);
        }
        __syncwarp();
    } else if (warp >= K::kMma) {
        // ------------------------------------------------------------ segments and matrix products
        if (warp == K::kMma + 1) {
            // -------------------------------------------------------- segments
            if (lane == 0 && p.cuts) p.cuts[cta].parts = 0;
            int s = sh.start_s, t = sh.start_t, hd = sh.start_hd, x = t_begin, base = sh.start_base;
#pragma unroll 1
            for (int n = 0; has_work && x < t_end;) {
                const Seq seq = seq_of(s, false);
                const Tile tile = tile_of<K>(p, seq, p.starts ? 0 : sh.least[s], tt, t);
                const int end = base + over + tile.count;  // of the tile in the line
                const int from = max(x - base - over, 0), take = min(end, t_end) - (base + over) - from;
                const int kvh = hd / head_blocks, h0 = kvh * p.group + hd % head_blocks * gb;
                const bool begins = from == 0, ends = from + take == tile.count;
                x = min(end, t_end);
                base = x;
                const int s_now = s, hd_now = hd;
                if (x < t_end && ++t >= (seq.n + tt - 1) / tt) {
                    t = 0;
#pragma unroll 1
                    for (;;) {  // the next sequence with a row
                        if (++s >= seqs) s = 0, ++hd;
                        const int y = s + lane;
                        const bool some = y < seqs && (p.starts ? request(p, y, false).n > 0 : sh.counts[y] > 0);
                        const uint32_t mask = __ballot_sync(0xffffffffu, some);
                        if (mask) {
                            s += __ffs(mask) - 1;
                            break;
                        }
                        s += 31;
                    }
                }
                if (take <= 0) continue;  // only what the line counts besides
                const int qi = n % kQueue;
                if (!wait_on(&sh.seg_empty[qi], (uint32_t)(n / kQueue + 1) & 1u, abort_flag, p.err, p.wait_ns)) break;
                ++n;
                int *members = sh.members[qi];
                if (!p.starts) {  // the requests of these ranks
                    int rank = 0;
#pragma unroll 1
                    for (int b0 = 0; b0 < p.batch && rank < tile.tok0 + tile.toks; b0 += 32) {
                        const int b = b0 + lane;
                        const bool in = b < p.batch && behind(p, b, s_now);
                        const uint32_t mask = __ballot_sync(0xffffffffu, in);
                        const int r = rank + __popc(mask & ((1u << lane) - 1u)) - tile.tok0;
                        if (in && r >= 0 && r < tile.toks) members[r] = b;
                        rank += __popc(mask);
                    }
                    __syncwarp();
                }
                int parts = 1;
                if (begins && !ends) parts = (int)(((long long)end * active - 1) / total_units) - cta + 1;
                if (!p.starts && begins)
#pragma unroll 1
                    for (int i = lane; i < tile.toks; i += 32)
                        p.found[(long long)hd_now * p.batch + members[i]] = Found{ends ? -1 : cta, parts, i * gb, 0};
                if (lane == 0) {
                    Segment &g = sh.segs[qi];
                    g.rows = tile.toks * gb, g.heads = min(gb, (kvh + 1) * p.group - h0);
                    g.q0 = seq.q0 + tile.tok0, g.first = tile.first, g.total = seq.total;
                    g.kvh = kvh, g.h0 = h0, g.key0 = tile.key0 + from * kKeys, g.count = take;
                    g.lo = tile.lo, g.hi = tile.hi, g.own0 = p.starts ? seq.own0 : seq.total, g.gap = p.starts ? gap_of<K>(seq.own0) : 0;
                    g.own_pages = p.table + (p.starts ? s_now * p.table_stride : 0);
                    g.pre_pages = p.ptable + (seq.pre >= 0 ? seq.pre * p.ptable_stride : 0);
                    g.slot = begins && ends ? -1 : begins ? 2 * cta + 1 : 2 * cta;
                    g.last = end > t_end || t_end - end <= over;
                    if (p.cuts && begins && !ends) p.cuts[cta] = Cut{parts, g.rows, g.q0, h0, kvh, g.heads, s_now, tile.first};
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sh.seg_full[qi]);
            }
        }
        if (warp == K::kMma && has_work) {
            // -------------------------------------------------------- matrix products
            const uint32_t id_qk = tc5::idesc(K::kB16, kKeys, p.scale < 0.f, false);
            const uint32_t id_pv = tc5::idesc(K::kB16, 16 * k_steps, false, true);
            const uint64_t q_desc = tc5::desc_sw128(q_base, 16, 1024), k_desc = tc5::desc_sw128(ring, 16, 1024),
                           v_desc = tc5::desc_sw128(ring, kKeys * 128, 1024);
            int stage = 0;
            uint32_t phase = 0, step_a = 0, step_b = 0;
            bool ok = true, last = false;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                ok = wait_on(bar, parity, abort_flag, p.err, p.wait_ns);
                return ok;
            };
#pragma unroll 1
            for (int n = 0; ok && !last; ++n) {
                const int qi = n % kQueue;
                if (!wait(&sh.seg_full[qi], (uint32_t)(n / kQueue) & 1u)) break;
                const int groups = kTiles == 1 || uniform(sh.segs[qi].rows) <= 128 ? 1 : 2, count = uniform(sh.segs[qi].count);
                last = uniform(sh.segs[qi].last);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sh.seg_empty[qi]);
                if (!wait(&sh.q_full, (uint32_t)n & 1u)) break;
                // Step j: the values of unit j, then the keys of unit j + kAhead, group after group.
#pragma unroll 1
                for (int j = -K::kAhead; ok && j < count; ++j) {
                    const bool values = j >= 0, keys = j + K::kAhead < count;
                    int v_at = 0, k_at = 0;
                    if (keys) {
                        k_at = stage;
                        if (!wait(&sh.full[stage], phase)) break;
                        if (++stage == kStages) stage = 0, phase ^= 1u;
                    }
                    if (values) {
                        v_at = stage;
                        if (!wait(&sh.full[stage], phase)) break;
                        if (++stage == kStages) stage = 0, phase ^= 1u;
                    }
#pragma unroll 1
                    for (int x = 0; x < groups; ++x) {
                        const bool final = x == groups - 1;
                        const uint32_t step = x ? step_b : step_a;  // of the group, over all segments
                        const uint32_t at = step % K::kAhead, turn = step / K::kAhead & 1u;  // the scores' place, and its phase
                        const uint32_t s = tmem + x * K::kSStep + at * K::kSBuffer;
                        if (values) {
                            const uint32_t d = tmem + K::kO + x * K::kOStep;
                            const uint64_t b = v_desc + (uint32_t)(v_at * (K::kStageBytes >> 4));
                            // With 128 keys a unit, the first 64 weights' products do not wait for the others.
                            constexpr int kFirst = kKeys == 128 ? 4 : 0, kTurn = kKeys == 128 ? 4 : 0;  // keys 64 to 127 come first
                            if constexpr (kFirst > 0) {
                                if (!wait(&sh.p_half[x], step & 1u)) break;
                                tc5::fence_after();
                                if (elect())
#pragma unroll
                                    for (int ks = 0; ks < kFirst; ++ks)
                                        tc5::mma_ts(d, s + K::kWeights + ks * 8, b + (uint32_t)((ks ^ kTurn) * (2048 >> 4)), id_pv, j > 0 || ks > 0);
                            }
                            if (!wait(&sh.p_full[x][at], turn)) break;
                            tc5::fence_after();
                            if (elect()) {
#pragma unroll
                                for (int ks = kFirst; ks < kKeys / 16; ++ks)
                                    tc5::mma_ts(d, s + K::kWeights + ks * 8, b + (uint32_t)((ks ^ kTurn) * (2048 >> 4)), id_pv, j > 0 || ks > 0);
                                tc5::commit(j == count - 1 ? &sh.o_full[x] : &sh.o_step[x]);
                                if (final) tc5::commit(&sh.empty[v_at]);
                            }
                            __syncwarp();
                        }
                        if (keys) {
                            // These scores go where this step's weights have been or, at the beginning, to the first places.
                            const uint32_t to = (values ? step : step + (uint32_t)(j + K::kAhead)) % K::kAhead;
                            const uint32_t d = tmem + x * K::kSStep + to * K::kSBuffer;
                            const uint64_t a = q_desc + (uint32_t)(x * (16384 >> 4)), b = k_desc + (uint32_t)(k_at * (K::kStageBytes >> 4));
                            tc5::fence_after();
                            if (elect()) {
#pragma unroll
                                for (int ks = 0; ks < DT / 16; ++ks)
                                    if (ks < k_steps)
                                        tc5::mma_ss(d, a + (uint32_t)((ks >> 2) * (K::kRows * 128 >> 4) + (ks & 3) * 2),
                                                    b + (uint32_t)((ks >> 2) * (kKeys * 128 >> 4) + (ks & 3) * 2), id_qk, ks > 0);
                                tc5::commit(&sh.s_full[x][to]);
                                if (final) {
                                    tc5::commit(&sh.empty[k_at]);
                                    if (j + K::kAhead + 1 == count) tc5::commit(&sh.q_empty);
                                }
                            }
                            __syncwarp();
                        }
                        if (values) {
                            if (x) ++step_b;
                            else ++step_a;
                        }
                    }
                }
            }
            if (!ok) {  // what has been issued comes to an end before tensor memory is given back
                if (elect()) tc5::commit(&sh.drain);
                volatile int no_abort = 0;
                ptx::mbar_wait(&sh.drain, 0u, &no_abort, nullptr, 200000000ull);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax and output
        const int x = warp >> 2;                                   // group
        const int row = x * 128 + (warp & 3) * 32 + lane;          // of the tile
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;  // tensor memory lanes of this warp
        const uint32_t t_s0 = tmem + lanes + x * K::kSStep, t_o = tmem + lanes + K::kO + x * K::kOStep;
        uint32_t step = 0, segs_had = 0;  // units and segments that the group has had
        int unit_n = 0;
        bool last = !has_work, ok = true, odd = false;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok = wait_on(bar, parity, abort_flag, p.err, p.wait_ns);
            return ok;
        };
#pragma unroll 1
        for (int n = 0; ok && !last; ++n) {
            const int qi = n % kQueue;
            if (!wait(&sh.seg_full[qi], (uint32_t)(n / kQueue) & 1u)) break;
            const Segment &g = sh.segs[qi];
            last = g.last;
            const int count = g.count, key_first = g.key0, slot = g.slot, kvh = g.kvh;
            const int tk = row * gb_inv >> 16, hh = row - tk * gb, head = g.h0 + hh;
            const bool in = row < g.rows && hh < g.heads;
            const bool some = x * 128 + (warp & 3) * 32 < g.rows;  // the warp has a row
            const bool idle = x * 128 >= g.rows;                     // so has none of the group
            int b = 0, lo = 0, hi = 0x7fffffff;  // rows that are none see everything, so that nothing has to be hidden for them
            if (in) {
                if (p.starts) {
                    b = g.q0 + tk;
                    hi = max(g.first + tk, 0);
                    lo = placed_from(p.window > 0 ? max(0, hi - p.window) : 0, g.own0, g.gap);
                    hi = placed_to(hi, g.own0, g.gap);
                } else {
                    b = sh.members[qi][tk];
                    hi = g.total;
                    if (p.window > 0)
                        lo = (int)max(0ll, (long long)hi + clamp_len(p.lens[b], p.max_pages, p.c.page_size) - p.window);
                }
            }
            auto done = [&] {
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sh.seg_empty[qi]);
            };
            if (idle) {
                done();
                unit_n += count;
                continue;
            }
            float k_scale = K::k8 && p.c.k_scale ? p.c.k_scale[kvh] : 1.f, unit = 1.f, slack = 0.f, in2 = 0.f, cap = 0.f;
            float m = kLowest, limit = kLowest, shift = 0.f;
            bool far = false;
            float2 l = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int j = 0; j < count; ++j, ++unit_n, ++step) {
                const uint32_t at = step % K::kAhead, t_s = t_s0 + at * K::kSBuffer;
                if (!wait(&sh.s_full[x][at], step / K::kAhead & 1u)) break;
                tc5::fence_after();
                if (j == 0) {
                    if constexpr (K::kOwnPower) k_scale *= sh.powers[qi][row];
                    unit = unit_of(p, k_scale);
                    if (p.softcap > 0.f) {
                        const Scores sc(p, k_scale);
                        unit = 1.f, in2 = sc.in, cap = sc.cap;
                    }
                    slack = kSlack / unit;
                    done();
                }
                if (some) {
                    const int key0 = key_first + j * kKeys;
                    const uint32_t *bad = sh.bad[unit_n & 15];
                    const bool masked = __any_sync(0xffffffffu, lo > key0 || hi - kKeys < key0) || (bad[0] | bad[1] | bad[2] | bad[3]);
                    if (masked || cap != 0.f) {  // what is not a plain product goes back to where the products were
#pragma unroll 1
                        for (int c = 0; c < kKeys / 32; ++c) {
                            // Which of these 32 the row sees, as bits; where all rows see all of them the products stay.
                            const int from = lo - (key0 + c * 32), to = hi - (key0 + c * 32);
                            uint32_t seen = ~(kKeys == 128 ? bad[c] : bad[2 * c] | (bad[2 * c + 1] << 16));
                            seen &= from <= 0 ? ~0u : from < 32 ? ~0u << from : 0u;
                            seen &= to >= 32 ? ~0u : to > 0 ? ~(~0u << to) : 0u;
                            const bool whole = __all_sync(0xffffffffu, seen == ~0u);
                            const bool quick = cap != 0.f && cap <= kQuickCap;
                            if (cap > kQuickCap) squeeze_in_place(t_s + c * 32, in2, cap);
                            if (whole && !quick) continue;
                            uint32_t v[32];
                            tc5::ld32(t_s + c * 32, v);
                            tc5::wait_ld();
                            if (quick) {  // cap * (1 - 2 / (1 + e^2x)), step by step for all 32
                                auto all = [&](auto f) {
#pragma unroll
                                    for (int i = 0; i < 32; i += 2) {
                                        const float2 y = f(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])));
                                        v[i] = __float_as_uint(y.x), v[i + 1] = __float_as_uint(y.y);
                                    }
                                };
                                const float2 by = make_float2(in2, in2), two = make_float2(-2.f * cap, -2.f * cap), one = make_float2(cap, cap);
                                all([&](float2 x) { x = fma2(x, by, make_float2(0.f, 0.f)); return make_float2(ex2(x.x), ex2(x.y)); });
                                all([&](float2 x) { x = add2(x, make_float2(1.f, 1.f)); return make_float2(rcp(x.x), rcp(x.y)); });
                                all([&](float2 x) { return fma2(x, two, one); });
                            }
                            if (!whole)
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (!(seen & 1u << i)) v[i] = 0xff800000u;
                            tc5::st32(t_s + c * 32, v);
                        }
                        tc5::wait_st();
                    }
                    // The maximum, 32 scores at a time, the next ones on their way. The code is kept small: all roles' together has
                    // to fit the instruction caches (a loop over 128 scores in registers, 14 KB, was slower).
                    uint32_t v[2][32];
                    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    auto tops = [&](const uint32_t (&z)[32]) {
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            top[i / 2 & 3] = fmaxf(top[i / 2 & 3], fmaxf(__uint_as_float(z[i]), __uint_as_float(z[i + 1])));
                    };
                    tc5::ld32(t_s, v[0]);
#pragma unroll 1
                    for (int c = 0; c < kKeys / 32; c += 2) {
                        tc5::wait_ld();
                        tc5::ld32(t_s + c * 32 + 32, v[1]);
                        tops(v[0]);
                        tc5::wait_ld();
                        if (c + 2 < kKeys / 32) tc5::ld32(t_s + c * 32 + 64, v[0]);
                        tops(v[1]);
                    }
                    const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    // Rows that are none have no vote here: what is in them is other requests' or an earlier kernel's.
                    if (__any_sync(0xffffffffu, in && mx > limit)) {
                        const float y = fmaxf(m, mx), far_y = y * unit, at_y = y > kLowest ? fmaf(-y, unit, K::kUp) : 0.f;
                        far = __any_sync(0xffffffffu, in && fabsf(far_y) >= 1024.f && y > kLowest);
                        const float keep = m == kLowest ? 0.f : far ? ex2((m - y) * unit) : ex2(at_y - shift);  // nothing so far: nothing is kept
                        if (j > 0) {  // once the last product has been added to the outputs
                            if (!wait(&sh.o_step[x], (step - segs_had - 1) & 1u)) break;
                            tc5::fence_after();
                            constexpr int kBoth = DT > 128 ? 2 : 1;  // (with 128 registers a thread two spill)
#pragma unroll 1
                            for (int c = 0; c < (D + 16 * kBoth - 1) / (16 * kBoth); ++c) {
                                uint32_t o[kBoth][16];
#pragma unroll
                                for (int z = 0; z < kBoth; ++z) tc5::ld16(t_o + (c * kBoth + z) * 16, o[z]);
                                tc5::wait_ld();
#pragma unroll
                                for (int z = 0; z < kBoth; ++z) {
#pragma unroll
                                    for (int i = 0; i < 16; ++i) o[z][i] = __float_as_uint(__uint_as_float(o[z][i]) * keep);
                                    tc5::st16(t_o + (c * kBoth + z) * 16, o[z]);
                                }
                            }
                        }
                        l.x *= keep, l.y *= keep;
                        m = y, limit = y + slack, shift = at_y;
                    }
                    // Weights are 2^(s unit + shift), 2^kUp at the reference; the shift's rounding is in all of them alike and in
                    // the shift that is kept. Where scores are so large that it could be seen, differences to the reference are
                    // taken first. Weights are rounded to the operands' type, half a step at most each; the sum that outputs are
                    // divided by is that of the unrounded ones (that of the rounded ones, as costly as all other sums and maxima
                    // together, would leave the errors' bound as it is).
                    const float2 by2 = far ? make_float2(1.f, 1.f) : make_float2(unit, unit);
                    const float2 up2 = far ? make_float2(K::kUp, K::kUp) : make_float2(shift, shift);
                    auto weights = [&](uint32_t (&z)[32], uint32_t to) {
                        if (far)
#pragma unroll
                            for (int i = 0; i < 32; ++i) z[i] = __float_as_uint((__uint_as_float(z[i]) - m) * unit);
                        uint32_t h[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float2 s = make_float2(__uint_as_float(z[2 * i]), __uint_as_float(z[2 * i + 1]));
                            s = fma2(s, by2, up2);
                            s.x = ex2(s.x), s.y = ex2(s.y);
                            l = add2(l, s);
                            h[i] = elem::pair_from_f32<typename K::M>(s.x, s.y);
                        }
                        tc5::st16(to, h);
                    };
                    // The last 64 scores are still there. Of 128, their weights go where they have been, those of the first 64
                    // behind them, and the product with the values begins with them.
                    uint32_t to = t_s + K::kWeights;
#pragma unroll 1
                    for (int c = kKeys / 64 - 1; c >= 0; --c, to += 32) {
                        weights(v[0], to);
                        if (c > 0) tc5::ld32(t_s, v[0]);
                        weights(v[1], to + 16);
                        if (c > 0) {
                            tc5::ld32(t_s + 32, v[1]);
                            tc5::wait_ld();
                            tc5::wait_st();
                            tc5::fence_before();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(&sh.p_half[x]);
                        }
                    }
                    tc5::wait_st();
                } else if (lane == 0 && kKeys == 128) {
                    ptx::mbar_arrive(&sh.p_half[x]);
                }
                tc5::fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&sh.p_full[x][at]);
            }
            if (!ok) break;
            if (!wait(&sh.o_full[x], segs_had & 1u)) break;
            ++segs_had;
            tc5::fence_after();
            if (!some) continue;
            const float v_scale = K::k8 && p.c.v_scale ? p.c.v_scale[kvh] : 1.f;
            const float sum = l.x + l.y;
            const bool any = sum > 0.f || sum != sum;
            const bool direct = slot < 0 && p.starts;
            const float f = !direct ? 1.f : any ? v_scale / sum : 0.f;
            float *sums = nullptr;
            if (!direct)
                sums = slot >= 0 ? p.slots + (long long)slot * K::kSlot + row * K::kPitch
                                   : p.whole + ((long long)b * p.heads + head) * K::kPitch;
            T *out = static_cast<T *>(p.out) + (long long)b * p.o_row + head * p.o_head;
            float check[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int c = 0; c < (D + 31) / 32; ++c) {
                uint32_t v[32];
                float o[32];
                tc5::ld32(t_o + c * 32, v);
                tc5::wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __uint_as_float(v[i]) * f;  // (0 of weights of 0)
                if (direct) {
                    uint32_t h[16];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c * 32 + (i & ~7) < D) check[i & 3] = fmaf(o[i], 0.f, check[i & 3]);
#pragma unroll
                    for (int i = 0; i < 16; ++i) h[i] = elem::pair_from_f32<T>(o[2 * i], o[2 * i + 1]);
                    if (in)
#pragma unroll
                        for (int i = 0; i < 16; i += 8) {
                            T *to = out + c * 32 + 2 * i;
                            if (p.wide_out && c * 32 + 2 * i + 16 <= D) {
                                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(h[i]), "r"(h[i + 1]),
                                             "r"(h[i + 2]), "r"(h[i + 3]), "r"(h[i + 4]), "r"(h[i + 5]), "r"(h[i + 6]), "r"(h[i + 7])
                                             : "memory");
                            } else {
                                if (c * 32 + 2 * i < D) *reinterpret_cast<uint4 *>(to) = make_uint4(h[i], h[i + 1], h[i + 2], h[i + 3]);
                                if (c * 32 + 2 * i + 8 < D)
                                    *reinterpret_cast<uint4 *>(to + 8) = make_uint4(h[i + 4], h[i + 5], h[i + 6], h[i + 7]);
                            }
                        }
                } else if (in) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        if (c * 32 + i < D) store8(sums + c * 32 + i, o + i);
                }
            }
            if (in) {
                if (direct) {
                    const float all = (check[0] + check[1]) + (check[2] + check[3]);
                    odd |= all != all;
                    if (p.lse)
                        p.lse[(long long)b * p.heads + head] = any ? (log2f(sum) - shift) / kLog2e : -INFINITY;
                } else {
                    *reinterpret_cast<float4 *>(sums + DT) = make_float4(any ? -shift : -INFINITY, sum, 0.f, 0.f);
                }
            }
        }
        if (odd) sh.odd = 1;  // every thread writes the same
    }
    tc5::fence_before();
    __syncthreads();
    tc5::fence_after();
    if (warp == K::kMma) tc5::dealloc(tmem, 512);
    if (tid == 0) p.odd[cta] = sh.odd;
}

// ------------------------------------------------------------------ joins
// Sums over some keys of a row: a lane holds the elements 4 * (lane + 32 i).
template <int DT>
struct Sums {
    static constexpr int kEach = DT > 128 ? 2 : 1;
    float m = -INFINITY, l = 0.f;
    float4 o[kEach];
};
// Joins a row's parts, which lie with the CTAs from `first` on.
template <typename K>
__device__ __forceinline__ Sums<K::kDim> join_parts(const Params &p, int first, int parts, int row, int D) {
    constexpr int DT = K::kDim, kOnce = 4;
    Sums<DT> r;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < r.kEach; ++e) r.o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i0 = 0; i0 < parts; i0 += kOnce) {  // all that some parts have is asked for at once
        float4 s[kOnce], y[kOnce][r.kEach];
#pragma unroll
        for (int i = 0; i < kOnce; ++i) {
            const int part = i0 + i;
            const bool there = part < parts;
            const float *from = p.slots + (long long)(2 * (first + part) + (part == 0)) * K::kSlot + row * K::kPitch;
            s[i] = there ? __ldcg(reinterpret_cast<const float4 *>(from + DT)) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
#pragma unroll
            for (int e = 0; e < r.kEach; ++e) {
                const int d = 4 * (lane + 32 * e);
                y[i][e] = there && d < D ? __ldcg(reinterpret_cast<const float4 *>(from + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        float top = r.m;
#pragma unroll
        for (int i = 0; i < kOnce; ++i) top = fmaxf(top, s[i].x);
        const float base = top == -INFINITY ? 0.f : top, keep = ex2(r.m - base);
        r.m = top, r.l *= keep;
#pragma unroll
        for (int e = 0; e < r.kEach; ++e) r.o[e].x *= keep, r.o[e].y *= keep, r.o[e].z *= keep, r.o[e].w *= keep;
#pragma unroll
        for (int i = 0; i < kOnce; ++i) {
            const float f = ex2(s[i].x - base);
            if (f == 0.f) continue;  // nothing there, or nothing that would count
            r.l = fmaf(f, s[i].y, r.l);
#pragma unroll
            for (int e = 0; e < r.kEach; ++e) {
                r.o[e].x = fmaf(f, y[i][e].x, r.o[e].x), r.o[e].y = fmaf(f, y[i][e].y, r.o[e].y);
                r.o[e].z = fmaf(f, y[i][e].z, r.o[e].z), r.o[e].w = fmaf(f, y[i][e].w, r.o[e].w);
            }
        }
    }
    return r;
}

// One row (a warp) from its definition: what a weight of 0 times an infinity, or a value that
// this row does not see but others of its tile do, has spoilt. Keys [lo, hi) of a prefix of
// `own0` keys and the request's own; only the tokens with a weight are looked at.
template <typename T, typename C, int DT>
__device__ __noinline__ void one_row(const Params &p, const T *q, T *out, float *lse, int kvh, const int32_t *pre_pages,
                                     const int32_t *own_pages, int own0, int lo, int hi) {
    constexpr int kEach = (DT + 31) / 32;
    const int lane = threadIdx.x & 31, D = p.c.head_dim;
    const float k_scale = sizeof(C) == 1 && p.c.k_scale ? p.c.k_scale[kvh] : 1.f;
    const float v_scale = sizeof(C) == 1 && p.c.v_scale ? p.c.v_scale[kvh] : 1.f;
    const Scores sc(p, k_scale);
    float qv[kEach], o[kEach], m = kLowest, m_score = 0.f, l = 0.f;
    auto number = [](C x) {
        if constexpr (sizeof(C) == 1) {
            uint32_t a, b;
            elem::e4m3x4_to_half2(x.bits, a, b);
            return elem::pair_to_f32<__half>(a).x;
        } else {
            return (float)x;
        }
    };
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int d = lane + 32 * e;
        qv[e] = d < D && p.scale != 0.f ? (float)q[d] : 0.f;
        if (p.scale < 0.f) qv[e] = -qv[e];
        o[e] = 0.f;
    }
#pragma unroll 1
    for (int j = lo; j < hi; ++j) {
        const bool pre = j < own0;
        const unsigned int y = pre ? j : j - own0, n = y / (unsigned int)p.c.page_size;
        const int page = (pre ? pre_pages : own_pages)[n];
        if (page < 0 || page >= p.c.pages) continue;
        const unsigned long long at = y - n * (unsigned int)p.c.page_size, pg = page;
        const C *k = static_cast<const C *>(p.c.k) + pg * p.c.k_page + at * p.c.k_token + kvh * p.c.k_head;
        const C *v = static_cast<const C *>(p.c.v) + pg * p.c.v_page + at * p.c.v_token + kvh * p.c.v_head;
        float s = 0.f;
        if (p.scale != 0.f)
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int d = lane + 32 * e;
                if (d < D) s = fmaf(qv[e], number(k[d]), s);
            }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float top = fmaxf(m, s);
        if (top > m) {
            const float top_score = sc.of(top);
            const float keep = sc.capped ? ex2(m_score - top_score) : ex2((m - top) * sc.unit);
            const bool none = l == 0.f;
            l = none ? 0.f : l * keep;
#pragma unroll
            for (int e = 0; e < kEach; ++e) o[e] = none || keep == 0.f ? 0.f : o[e] * keep;
            m = top, m_score = top_score;
        }
        const float w = sc.capped ? ex2(sc.of(s) - m_score) : ex2((s - m) * sc.unit);
        l += w;
        if (w != 0.f)
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int d = lane + 32 * e;
                if (d < D) o[e] = fmaf(w, number(v[d]), o[e]);
            }
    }
    const bool any = l > 0.f || l != l;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const int d = lane + 32 * e;
        if (d < D) out[d] = any ? (T)(o[e] / l * v_scale) : (T)0.f;
    }
    if (lse && lane == 0) *lse = any ? (sc.of(m) + log2f(l)) / kLog2e : -INFINITY;
}

// The largest magnitude of what a lane holds is no finite number in some lane.
__device__ __forceinline__ bool spoilt(float check) { return __any_sync(0xffffffffu, check != check); }

// Four elements of a row; *check becomes NaN where one is no finite number.
template <typename T>
__device__ __forceinline__ void store4(T *to, const float4 &y, float *check) {
    *check = fmaf(y.x, 0.f, fmaf(y.y, 0.f, fmaf(y.z, 0.f, fmaf(y.w, 0.f, *check))));
    *reinterpret_cast<uint2 *>(to) = make_uint2(elem::pair_from_f32<T>(y.x, y.y), elem::pair_from_f32<T>(y.z, y.w));
}

// Of a block. (8 rows to a block: 17 us to join 4099 rows' tiles and 6 for drafts, 32: 15.6 and 6, 16: 16 and 4.7.)
constexpr int kJoinWarps = 8, kJoinRows = 16;

// Requests: the tiles that were cut are joined, and rows that are no finite numbers looked at again.
template <typename T, typename C, int DT>
__global__ void __launch_bounds__(32 * kJoinWarps) finish_kernel(const __grid_constant__ Params p) {
    using K = Config<T, C, DT>;
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = p.c.head_dim;
    constexpr int kBlocks = K::kRows / kJoinRows;  // of a tile
    const int gb = min(p.group, K::kRows), cta = blockIdx.x / kBlocks, r0 = blockIdx.x % kBlocks * kJoinRows;
    auto again = [&](int b, int row, int head, int hi) {
        const Seq s = request(p, b, false);
        const int lo = p.window > 0 ? max(0, hi - p.window) : 0, kvh = head / p.group;
        one_row<T, C, DT>(p, static_cast<const T *>(p.q) + (long long)row * p.q_row + head * p.q_head,
                          static_cast<T *>(p.out) + (long long)row * p.o_row + head * p.o_head,
                          p.lse ? p.lse + (long long)row * p.heads + head : nullptr, kvh,
                          s.pre >= 0 ? p.ptable + s.pre * p.ptable_stride : nullptr, p.table + b * p.table_stride, s.own0, lo, hi);
    };
    const Cut c = p.cuts[cta];
    if (c.parts > 1 && cta + c.parts <= p.ctas)
#pragma unroll 1
        for (int i = 0; i < kJoinRows / kJoinWarps; ++i) {
            const int r = r0 + i * kJoinWarps + warp, tk = r / gb, hh = r - tk * gb;
            if (r >= c.rows || hh >= c.heads) continue;
            const Sums<DT> x = join_parts<K>(p, cta, c.parts, r, D);
            const bool any = x.l > 0.f || x.l != x.l;
            const float f = any ? (K::k8 && p.c.v_scale ? p.c.v_scale[c.kvh] : 1.f) / x.l : 0.f;
            const int row = c.q0 + tk, head = c.h0 + hh;
            T *out = static_cast<T *>(p.out) + (long long)row * p.o_row + head * p.o_head;
            float check = 0.f;
#pragma unroll
            for (int e = 0; e < x.kEach; ++e) {
                const int d = 4 * (lane + 32 * e);
                if (d < D) store4(out + d, make_float4(x.o[e].x * f, x.o[e].y * f, x.o[e].z * f, x.o[e].w * f), &check);
            }
            if (p.lse && lane == 0)
                p.lse[(long long)row * p.heads + head] = any ? (x.m + log2f(x.l)) / kLog2e : -INFINITY;
            if (spoilt(check)) again(c.seq, row, head, max(c.first + tk, 0));
        }
    if (!__syncthreads_or((int)threadIdx.x < p.ctas && p.odd[threadIdx.x])) return;
#pragma unroll 1
    for (long long i = (long long)blockIdx.x * kJoinWarps + warp; i < (long long)p.rows * p.heads; i += (long long)gridDim.x * kJoinWarps) {
        const int row = (int)(i / p.heads), head = (int)(i % p.heads);
        const T *out = static_cast<const T *>(p.out) + (long long)row * p.o_row + head * p.o_head;
        float check = 0.f;
#pragma unroll 1
        for (int d = lane; d < D; d += 32) check = fmaf((float)out[d], 0.f, check);
        if (!spoilt(check)) continue;
        bool cut = false;  // joined above, or being joined
#pragma unroll 1
        for (int x = lane; x < p.ctas; x += 32) {
            const Cut y = p.cuts[x];
            cut |= y.parts > 1 && row >= y.q0 && row < y.q0 + y.rows / gb && head >= y.h0 && head < y.h0 + y.heads;
        }
        if (__any_sync(0xffffffffu, cut)) continue;
#pragma unroll 1
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
            Seq s{0, 0, 0, 0, 0};
            if (b0 + lane < p.batch) s = request(p, b0 + lane, false);
            const uint32_t mask = __ballot_sync(0xffffffffu, row >= s.q0 && row - s.q0 < s.n);
            if (!mask) continue;
            const int from = __ffs(mask) - 1;
            const int hi = __shfl_sync(0xffffffffu, max(s.total - s.n + (row - s.q0) + 1, 0), from);
            again(b0 + from, row, head, hi);
            break;
        }
    }
}

// Prefixes: what a request sees of its prefix is joined with its own tokens.
template <typename T, typename C, int DT>
__global__ void __launch_bounds__(32 * kJoinWarps) prefix_join_kernel(const __grid_constant__ Params p) {
    using K = Config<T, C, DT>;
    ptx::grid_dep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = p.c.head_dim;
    const long long i = (long long)blockIdx.x * kJoinWarps + warp;
    if (i >= (long long)p.batch * p.heads) return;
    const int b = (int)(i / p.heads), head = (int)(i % p.heads), kvh = head / p.group, in_group = head % p.group;
    const int gb = min(p.group, K::kRows), head_blocks = (p.group + gb - 1) / gb;
    const int own = clamp_len(p.lens[b], p.max_pages, p.c.page_size);
    T *out = static_cast<T *>(p.out) + b * p.o_row + head * p.o_head;
    bool none = false;
    const int pre = own > 0 ? prefix_of(p, b, &none) : -1;
    Sums<DT> x;
#pragma unroll
    for (int e = 0; e < x.kEach; ++e) x.o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (pre >= 0) {
        const Found f = p.found[(long long)(kvh * head_blocks + in_group / gb) * p.batch + b];
        const int row = f.row + in_group % gb;
        if (f.first < 0) {
            const float *from = p.whole + i * K::kPitch;
            const float4 s = __ldcg(reinterpret_cast<const float4 *>(from + DT));
            x.m = s.x, x.l = s.y;
#pragma unroll
            for (int e = 0; e < x.kEach; ++e) {
                const int d = 4 * (lane + 32 * e);
                if (d < D) x.o[e] = __ldcg(reinterpret_cast<const float4 *>(from + d));
            }
        } else if (f.parts > 0 && f.first + f.parts <= p.ctas && row >= 0 && row < K::kRows) {
            x = join_parts<K>(p, f.first, f.parts, row, D);
        }
    }
    const float own_lse = own > 0 ? p.raw_lse[i] : -INFINITY;
    const bool any = x.l > 0.f || x.l != x.l, any_own = !(own_lse == -INFINITY);
    const float a = any ? x.m + log2f(x.l) : -INFINITY;
    const float top = fmaxf(a, own_lse), from = top == -INFINITY ? 0.f : top;
    const float wa = any ? ex2(a - from) : 0.f, wo = any_own ? ex2(own_lse - from) : 0.f;
    const float sum = wa + wo, f = any ? wa / sum * (K::k8 && p.c.v_scale ? p.c.v_scale[kvh] : 1.f) / x.l : 0.f;
    const float fo = any_own ? wo / sum : 0.f;
    float check = 0.f;
#pragma unroll
    for (int e = 0; e < x.kEach; ++e) {
        const int d = 4 * (lane + 32 * e);
        if (d >= D) continue;
        float4 y = make_float4(x.o[e].x * f, x.o[e].y * f, x.o[e].z * f, x.o[e].w * f);
        if (any_own) {
            const float4 z = __ldcg(reinterpret_cast<const float4 *>(p.raw + i * D + d));
            y.x = fmaf(z.x, fo, y.x), y.y = fmaf(z.y, fo, y.y), y.z = fmaf(z.z, fo, y.z), y.w = fmaf(z.w, fo, y.w);
        }
        store4(out + d, y, &check);
    }
    if (p.lse && lane == 0) p.lse[i] = any || any_own ? (from + log2f(sum)) / kLog2e : -INFINITY;
    if (spoilt(check)) {
        const int shared = pre >= 0 ? clamp_len(p.plens[pre], p.pmax_pages, p.c.page_size) : 0;
        const long long hi = (long long)shared + own;
        one_row<T, C, DT>(p, static_cast<const T *>(p.q) + b * p.q_row + head * p.q_head, out, p.lse ? p.lse + i : nullptr, kvh,
                          pre >= 0 ? p.ptable + pre * p.ptable_stride : nullptr, p.table + b * p.table_stride, shared,
                          p.window > 0 ? (int)max(0ll, hi - p.window) : 0, (int)hi);
    }
}

// ------------------------------------------------------------------ launches
// Grid and block of a launch on `s`, as a programmatic dependent where that is wanted.
struct Launch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    Launch(unsigned blocks, int threads, int smem, cudaStream_t s) {
        cfg.gridDim = dim3(blocks, 1, 1);
        cfg.blockDim = dim3((unsigned)threads, 1, 1);
        cfg.dynamicSmemBytes = (size_t)smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = as_dependent(s) ? 1 : 0;
    }
};

// The kernels of a call, chosen by the types and the head's width.
enum Which { kWide, kFinish, kPrefixJoin };
template <typename T, typename C, int DT>
cudaError_t launch(Which which, const Params &p, cudaStream_t s) {
    using K = Config<T, C, DT>;
    constexpr int kSmem = K::kAfter + (int)sizeof(Shared<K::kRows>) + 1024;
    static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
    static_assert((4 * kMaxSeqs + 1) * 4 <= K::kAfter, "the plan lies where queries, keys and values come later");
    static_assert(K::kAfter % 1024 == 0, "alignment");
    if (which == kWide) {
        auto kernel = wide_kernel<T, C, DT>;
        const cudaError_t e = ensure_max_dyn_smem((const void *)kernel, kSmem);
        if (e != cudaSuccess) return e;
        Launch l((unsigned)p.ctas, K::kThreads, kSmem, s);
        return cudaLaunchKernelEx(&l.cfg, kernel, p);
    }
    if (which == kFinish) {
        Launch l((unsigned)(p.ctas * (K::kRows / kJoinRows)), 32 * kJoinWarps, 0, s);
        return cudaLaunchKernelEx(&l.cfg, finish_kernel<T, C, DT>, p);
    }
    Launch l((unsigned)(((long long)p.batch * p.heads + kJoinWarps - 1) / kJoinWarps), 32 * kJoinWarps, 0, s);
    return cudaLaunchKernelEx(&l.cfg, prefix_join_kernel<T, C, DT>, p);
}
template <typename T, typename C>
cudaError_t launch_dims(Which which, const Params &p, cudaStream_t s) {
    if (p.c.head_dim <= 64) return launch<T, C, 64>(which, p, s);
    if (p.c.head_dim <= 128) return launch<T, C, 128>(which, p, s);
    return launch<T, C, 256>(which, p, s);
}

// A head's width as the kernels have it, the rows of a tile, the keys of a unit.
inline int dim_of(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : 256; }
inline int rows_of(int head_dim) { return head_dim > 128 ? 128 : 256; }
inline int keys_of(int head_dim) { return head_dim > 128 ? 64 : 128; }

// Defined in wide_attention_f16.cu and wide_attention_bf16.cu.
cudaError_t launch_f16(Which which, const Params &p, cudaStream_t s);
cudaError_t launch_bf16(Which which, const Params &p, cudaStream_t s);

}  // namespace wide
}  // namespace w4a16
