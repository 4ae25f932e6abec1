// The next token of each row of logits: temperature, top-k, top-p, min-p, with a given random number.
//     w_i = 2^(-(max - x_i) log2(e) / T); of the tokens in the order of falling x (equal ones by number) the first k, of
//     these the fewest whose weights reach p of theirs, of these the ones with w_i >= min_p; the token drawn is the first, by
//     number, at which the kept weights' running sum exceeds u times their sum
//
// Weights are fixed-point numbers of 44 binary places in 64-bit integers, off by less than 2^-30 of themselves (2^-32 each
// from the table, the rest's whole number and the product, as much from the rest's roundings) and, below 2^-12 of the largest,
// by what is cut off below 2^-44 of it. Sums are exact and so do not depend on any order. A border between two tokens, a
// quotient of two sums, moves by less than 2^-31, about what it would take for a 32-bit random number to show it, and by less
// than 2^-44 for each token (where 2^18 tokens are all that far below the largest, 2^-26: a few of them). A weight below 2^-44
// of the largest is 0.
//
// A row is one cluster of CTAs, which keeps its logits in shared memory, so that each is read from memory once. The border of
// top-k and top-p is found by a histogram of counts over 32 bins for each factor of two of the weight. It
// names the bin of the k-th token, and a few bins that hold the border of top-p (a bin's weights are alike to 2%); a second
// pass adds up exactly what lies in front of these, and in each of them. Where few tokens lie above the border (as a rule)
// they are gathered, and one CTA sorts them and draws; otherwise the border's bin is resolved (by sorting its tokens or, when
// it holds many, by halving the range of its values) and one more pass sums and draws.
//
// What bounds it: instructions and barriers, not HBM. Mean cycles of a CTA of 37500 bf16 logits, two CTAs to an SM (256 rows of
// 150001, top-p alone, 315 us, 11 of them the bytes): logits and maximum 11000, counts 17000, bounds and searches 19000, exact
// sums 47000, the search in them 7000, the border's bin 30000, the last sums and the draw 33000. 61% of all issue slots are
// used, the rest is barriers' above all. A single row of 32001 takes 18 us: launch 3, and a dozen steps of a barrier of the
// cluster and some dependent reads each. Sums of weights in the histogram in place of counts (two shared atomics a logit) made
// 64 rows of 131072 128 us; with counts they are 82.
#include <climits>
#include <cmath>

#include "decode_ops.h"
#include "elem.cuh"
#include "ptx.cuh"

namespace w4a16 {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048, kPerOctave = 32;
constexpr int kMost = 1024;            // gathered tokens
constexpr int kMaxVocab = 1 << 18, kMaxCluster = 8;

struct SampleParams {
    const void *x;
    long long row;
    const float *u, *temperature, *top_p, *min_p;
    const int32_t *top_k;
    int64_t *out;
    int vocab, chunk;  // tokens of a CTA
    unsigned int *err;
};

// 2^(-(i + 1)/256) with 32 binary places, from the series of exp.
struct Table {
    uint32_t v[256];
};
constexpr Table make_table() {
    Table t{};
    for (int i = 0; i < 256; ++i) {
        const double y = -0.69314718055994530942 * (i + 1) / 256;
        double term = 1, sum = 1;
        for (int k = 1; k < 30; ++k) term *= y / k, sum += term;
        t.v[i] = (uint32_t)(sum * 4294967296.0 + 0.5);
    }
    return t;
}
__constant__ Table kPowers = make_table();

// A row's weights.
struct Heat {
    float top, c, c_low;  // largest logit (finite); log2(e) / temperature in two parts
    // 32 bins for each factor of two below the largest, to the nearest; kBins: NaN, and what is 64 factors below or more.
    __device__ __forceinline__ int bin(float x) const {
        const float t = fminf((top - x) * (c * kPerOctave), (float)kBins);
        return (int)(__float_as_uint(t + 12582912.f) - 0x4b400000u);
    }
    // As a product of two 32-bit numbers, which sums take up in one instruction. (Of what is far below the largest, infinities
    // and NaN the second is 0.)
    struct Weight {
        uint32_t part, up;
        __device__ __forceinline__ uint64_t whole() const { return (uint64_t)part * up; }
    };
    __device__ __forceinline__ Weight weight(float x, const uint32_t *powers, const uint2 *octaves) const {
        const float d = top - x, t = fminf(d * c, 64.f);
        // In 256th factors of two: the nearest whole number (the bits of a sum with 1.5 * 2^15), and the rest, with the
        // roundings of the difference and the product and the factor's second part.
        // (What the difference's rounding took is taken back by the sum of two numbers of any magnitudes: `x` may be the larger.)
        const float z = t + 49152.f, over = d - top, back = (top - (d - over)) - (x + over);
        const float low = fmaf(d, c, -t) + fmaf(d, c_low, back * c);
        const float y = ((t - (z - 49152.f)) + low) * 0.693147180559945f;
        const int k = (int)(__float_as_uint(z) - 0x47400001u);  // one less: an entry of the table, from 2^-(1/256) on, times 2^-y is below 1
        // 1 - 2^-y in three terms (|y| < 2^-9.4: the next is below 2^-42), as a whole number of 2^-31.
        const float e = y * fmaf(y, fmaf(y, 1.f / 6, -0.5f), 1.f);
        const int32_t cut = (int32_t)(2 * __float_as_uint(fmaf(e, 2147483648.f, 12582912.f)) - 0x967fffffu);  // twice, and 1: to the nearest, about
        // p - (p cut >> 32), p taken as the signed number that is 2^32 less.
        const uint32_t p = powers[k & 255], w = p - (uint32_t)__mulhi((int)p, cut) - (uint32_t)cut;
        const uint2 places = octaves[k >> 8];  // (-1 beside the largest)
        return Weight{w >> places.x, places.y};
    }
};

// Logits as numbers in their order: larger logits larger, -0 as 0.
template <typename T>
struct Logit;
template <>
struct Logit<float> {
    using Raw = uint32_t;
    static __device__ __forceinline__ float value(Raw r) { return __uint_as_float(r); }
    static __device__ __forceinline__ Raw half(Raw r) { return __float_as_uint(value(r) * 0.5f); }
    static __device__ __forceinline__ uint32_t key(Raw r) {
        if (r == 0x80000000u) r = 0;
        return r & 0x80000000u ? ~r : r | 0x80000000u;
    }
};
template <typename H>
struct Logit16 {
    using Raw = uint16_t;
    static __device__ __forceinline__ float value(Raw r) { return elem::pair_to_f32<H>(r).x; }
    static __device__ __forceinline__ Raw half(Raw r) { return (Raw)elem::pair_from_f32<H>(value(r) * 0.5f, 0.f); }
    static __device__ __forceinline__ uint32_t key(Raw r) {
        if (r == 0x8000u) r = 0;
        return r & 0x8000u ? (uint32_t)(uint16_t)~r : r | 0x8000u;
    }
};
template <>
struct Logit<__half> : Logit16<__half> {};
template <>
struct Logit<__nv_bfloat16> : Logit16<__nv_bfloat16> {};

__device__ __forceinline__ uint32_t remote(const void *local, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(ptx::smem_u32(local)), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t ld32(const uint32_t *local, int rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote(local, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t ld64(const uint64_t *local, int rank) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote(local, rank)) : "memory");
    return v;
}

// floor and ceil of w times a float in [0, 1), exactly.
__device__ __forceinline__ uint64_t part_of(uint64_t w, float f, bool up) {
    const uint32_t bits = __float_as_uint(f), e = bits >> 23;
    const uint64_t m = e ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu;
    const int shift = 150 - (int)(e ? e : 1);  // f = m * 2^-shift, shift >= 24
    const uint64_t lo = w * m, hi = __umul64hi(w, m);
    uint64_t q, rest;
    if (shift < 64) q = hi << (64 - shift) | lo >> shift, rest = lo << (64 - shift);
    else if (shift == 64) q = hi, rest = lo;
    else if (shift < 128) q = hi >> (shift - 64), rest = hi << (128 - shift) | lo;
    else q = 0, rest = hi | lo;
    return q + (up && rest);
}

// What is added up over the cluster.
struct Sums {
    uint64_t mass, front;
    uint32_t count;
};
// A bin: tokens in front of it and in it, and bounds of their weights.
struct Found {
    uint32_t bin, before, in;
    uint64_t most_before, least_before, most_in, least_in;
};

template <typename T>
struct alignas(16) Shared {
    union {
        uint32_t counts[kBins];   // the CTA's histogram
        uint64_t list[kMost];     // its gathered tokens
    };
    union {
        uint32_t parts[2][kBins]; // sums of weights of some bins, in two halves
        struct {
            uint64_t all[kMost], weights[kMost];  // gathered tokens of the whole cluster: key, then number counted down
        };
        uint32_t slice[kBins];    // counts of this CTA's share of the bins, over the cluster
    };
    uint32_t bins[kBins];         // all of them
    uint32_t listed, key_low, key_high;
    uint32_t powers[256];
    uint2 octaves[66];            // of octave o - 1: 44 binary places, 12 more than an entry of powers has, less o - 1
    uint64_t mass_slot[4][2];     // what a step adds up over the cluster
    uint32_t count_slot[4];
    float max_slot;
    uint32_t number_slot;
    uint64_t sums[2][kWarps];
    uint32_t sums32[kWarps];
    int owner;                    // a thread, and what lies in front of its tokens
    uint64_t owner_before;
    uint64_t found_mass, found_border;
    Found found;
    long long token[4];           // what a step has found, read by the whole cluster after its last barrier: a place for each of four steps
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
    using L = Logit<T>;
    using Raw = typename L::Raw;
    extern __shared__ __align__(16) unsigned char raw_smem[];
    Shared<T> &sh = *reinterpret_cast<Shared<T> *>(raw_smem);
    ptx::grid_dep_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t ranks;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(ranks));
    const int cluster = (int)ranks, rank = (int)ptx::cluster_rank(), row = blockIdx.x / cluster;
    const int c0 = min(rank * p.chunk, p.vocab), n = min(p.chunk, p.vocab - c0);  // this CTA's tokens
    const Raw *x = static_cast<const Raw *>(p.x) + row * p.row + c0;
    constexpr int kVec = 16 / sizeof(Raw);
    // Shared memory is skewed as the row is, so that both are read 16 bytes at a time: token c0 + i at mine[i], its vectors from
    // mine[-skew] on. What the first and the last vector have besides is NaN, which is nothing to all that follows.
    const int skew = (int)((uintptr_t)x % 16 / sizeof(Raw)), vectors = n > 0 ? (skew + n + kVec - 1) / kVec : 0;
    Raw *mine = reinterpret_cast<Raw *>(raw_smem + sizeof(Shared<T>)) + skew;
    uint4 *const packed = reinterpret_cast<uint4 *>(raw_smem + sizeof(Shared<T>));
    constexpr Raw kNone = sizeof(Raw) == 4 ? (Raw)0x7fffffffu : (Raw)0x7fffu;
    auto unpacked = [&](const uint4 &v, int z) -> Raw {
        const uint32_t w = z * sizeof(Raw) / 4 == 0 ? v.x : z * sizeof(Raw) / 4 == 1 ? v.y : z * sizeof(Raw) / 4 == 2 ? v.z : v.w;
        return sizeof(Raw) == 4 ? (Raw)w : (Raw)(z & 1 ? w >> 16 : w);
    };
    // f(i, raw) for this CTA's tokens.
    auto each_token = [&](auto f) {
#pragma unroll 1
        for (int v = tid; v < vectors; v += kThreads) {
            const uint4 q = packed[v];
#pragma unroll
            for (int z = 0; z < kVec; ++z) f(v * kVec - skew + z, unpacked(q, z));
        }
    };

    // What the row asks for.
    float heat = p.temperature ? p.temperature[row] : 1.f, top_p = p.top_p ? p.top_p[row] : 1.f, min_p = p.min_p ? p.min_p[row] : 0.f;
    float u = p.u[row];
    int top_k = p.top_k ? p.top_k[row] : 0;
    const bool wrong = !(heat >= 0.f) || top_p != top_p || min_p != min_p || !(u >= 0.f && u <= 1.f);
    if (wrong && rank == 0 && tid == 0) atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG);
    if (!(heat >= 0.f)) heat = 0.f;
    if (top_p != top_p) top_p = 1.f;
    if (min_p != min_p) min_p = 0.f;
    if (!(u >= 0.f)) u = 0.f;
    if (top_k <= 0 || top_k > p.vocab) top_k = p.vocab;

    // ---------------------------------------------------------------- logits into shared memory, and their maximum
    if (tid < 256) sh.powers[tid] = kPowers.v[tid];
    else if (tid < 256 + 66) {
        const int o = tid - 257;
        sh.octaves[o + 1] = make_uint2((unsigned)min(max(o - 12, 0), 31), o < 44 ? 1u << max(12 - o, 0) : 0u);
    }
    float top = -INFINITY;
    {
#pragma unroll 4
        for (int v = tid; v < vectors; v += kThreads) {
            const int i = v * kVec - skew;
            uint4 q;
            if (i >= 0 && i + kVec <= n) {
                q = *reinterpret_cast<const uint4 *>(x + i);
                packed[v] = q;
            } else {
                for (int j = i; j < i + kVec; ++j) mine[j] = j >= 0 && j < n ? x[j] : kNone;
                q = packed[v];
            }
#pragma unroll
            for (int z = 0; z < kVec; ++z) top = fmaxf(top, L::value(unpacked(q, z)));
        }
    }
    auto warp_max = [](float v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        return v;
    };
    auto warp_sum = [](uint64_t v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    top = warp_max(top);
    if (lane == 0) sh.sums32[warp] = __float_as_uint(top);
    __syncthreads();
    if (warp == 0) {
        top = warp_max(lane < kWarps ? __uint_as_float(sh.sums32[lane]) : -INFINITY);
        if (lane == 0) sh.max_slot = top;
    }
    ptx::cluster_sync();
    top = -INFINITY;
    for (int r = 0; r < cluster; ++r) top = fmaxf(top, __uint_as_float(ld32(reinterpret_cast<const uint32_t *>(&sh.max_slot), r)));

    // A step's sums over the cluster: every thread's part in, all of it out, the same everywhere.
    int step = 0;
    auto add_up = [&](uint64_t mass, uint64_t front, uint32_t count) {
        mass = warp_sum(mass), front = warp_sum(front);
        count = __reduce_add_sync(0xffffffffu, count);
        __syncthreads();
        if (lane == 0) sh.sums[0][warp] = mass, sh.sums[1][warp] = front, sh.sums32[warp] = count;
        __syncthreads();
        const int slot = step++ & 3;
        if (warp == 0) {
            mass = warp_sum(lane < kWarps ? sh.sums[0][lane] : 0), front = warp_sum(lane < kWarps ? sh.sums[1][lane] : 0);
            count = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.sums32[lane] : 0u);
            if (lane == 0) sh.mass_slot[slot][0] = mass, sh.mass_slot[slot][1] = front, sh.count_slot[slot] = count;
        }
        ptx::cluster_sync();
        Sums all{0, 0, 0};
        for (int r = 0; r < cluster; ++r)
            all.mass += ld64(&sh.mass_slot[slot][0], r), all.front += ld64(&sh.mass_slot[slot][1], r), all.count += ld32(&sh.count_slot[slot], r);
        return all;
    };
    // The first token, by number, at which the running sum of what(i, raw) over the row exceeds target(the whole sum), which is
    // below it. A thread has consecutive tokens (an odd number of vectors: no bank conflicts).
    const int per = ((vectors + kThreads - 1) / kThreads) | 1, v0 = min(tid * per, vectors), v1 = min(v0 + per, vectors);
    auto locate = [&](auto what, auto target_of) -> long long {
        uint64_t sum = 0;
#pragma unroll 1
        for (int v = v0; v < v1; ++v) {
            const uint4 q = packed[v];
#pragma unroll
            for (int z = 0; z < kVec; ++z) sum += what(v * kVec - skew + z, unpacked(q, z));
        }
        uint64_t upto = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        __syncthreads();
        if (lane == 31) sh.sums[0][warp] = upto;
        const int slot = step++ & 3;
        if (tid == 0) sh.token[slot] = -1, sh.owner = -1;  // (others may still read the last step's)
        __syncthreads();
        uint64_t mine_all = 0, before = upto - sum;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const uint64_t y = sh.sums[0][w];
            before += w < warp ? y : 0, mine_all += y;
        }
        if (tid == 0) sh.mass_slot[slot][0] = mine_all;
        ptx::cluster_sync();
        uint64_t whole = 0;
        for (int r = 0; r < cluster; ++r) {
            const uint64_t y = ld64(&sh.mass_slot[slot][0], r);
            before += r < rank ? y : 0, whole += y;
        }
        const uint64_t target = target_of(whole);
        if (before <= target && target < before + sum) sh.owner = tid, sh.owner_before = before;
        __syncthreads();
        if (warp == 0 && sh.owner >= 0) {  // a strip of 32 tokens at a time
            uint64_t front = sh.owner_before;
            const int first = sh.owner * per * kVec - skew, last = min(first + per * kVec, n);
            for (int i0 = first; i0 < last; i0 += 32) {
                const int i = i0 + lane;
                const uint64_t w = i >= 0 && i < last ? what(i, mine[i]) : 0;
                uint64_t run = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t y = __shfl_up_sync(0xffffffffu, run, o);
                    if (lane >= o) run += y;
                }
                const uint32_t mask = __ballot_sync(0xffffffffu, front + run > target);
                if (mask) {
                    if (lane == 0) sh.token[slot] = c0 + i0 + __ffs(mask) - 1;
                    break;
                }
                front += __shfl_sync(0xffffffffu, run, 31);
            }
        }
        ptx::cluster_sync();
        long long token = -1;
        for (int r = 0; r < cluster; ++r) token = max(token, (long long)ld64(reinterpret_cast<const uint64_t *>(&sh.token[slot]), r));
        return token;
    };
    const bool nothing = top == -INFINITY;                                     // no token may be drawn
    const bool greedy = heat == 0.f || top_k == 1 || top_p <= 0.f || min_p > 1.f;  // the largest logit, the first of equal ones
    if (nothing || greedy) {
        uint32_t first = 0xffffffffu;
        if (!nothing)
            each_token([&](int i, Raw r) {
                if (L::value(r) == top) first = min(first, (uint32_t)(c0 + i));
            });
        first = __reduce_min_sync(0xffffffffu, first);
        __syncthreads();
        if (lane == 0) sh.sums32[warp] = first;
        __syncthreads();
        if (warp == 0) {
            first = __reduce_min_sync(0xffffffffu, lane < kWarps ? sh.sums32[lane] : 0xffffffffu);
            if (lane == 0) sh.number_slot = first;
        }
        ptx::cluster_sync();
        if (rank == 0 && tid == 0) {
            for (int r = 0; r < cluster; ++r) first = min(first, ld32(&sh.number_slot, r));
            p.out[row] = nothing ? -1 : (int64_t)first;
        }
        ptx::cluster_sync();  // no CTA leaves while others read its memory
        return;
    }

    if (top == INFINITY) {  // these alone, all alike
        for (int i = tid; i < n; i += kThreads) mine[i] = L::value(mine[i]) == INFINITY ? (Raw)0 : kNone;
        top = 0.f;
        __syncthreads();
    }
    // Differences to a largest logit beyond 2^100 may be no floats: such a row is halved, and its temperature. (Nothing that this
    // rounds, below 2^-125, is told apart by a weight; fp16 has none of it.)
    if (top > 0x1p100f) {
        for (int i = tid; i < n; i += kThreads) mine[i] = L::half(mine[i]);
        top *= 0.5f, heat *= 0.5f;
        __syncthreads();
    }
    Heat h;
    {
        const double c = 1.4426950408889634 / (double)heat;
        h.top = top;
        h.c = c < 1e37 ? (float)c : 1e37f;  // (32 times that is still a number)
        h.c_low = c < 1e37 ? (float)(c - (double)h.c) : 0.f;
    }
    // The smallest logit that min-p leaves, rounded up.
    float floor_x = -INFINITY;
    if (min_p > 0.f) {
        const double cut = (double)top + (double)heat * log((double)min_p);
        if (cut == cut) floor_x = __double2float_ru(cut);
    }
    // ---------------------------------------------------------------- the border of top-k and top-p
    // Kept is what lies in front of the border in the order of falling keys, equal ones by number, the border included:
    // a 64-bit number, larger for what comes first.
    auto place = [&](uint32_t key, int number) { return (uint64_t)key << 32 | (uint32_t)~number; };
    uint64_t border = 0;  // everything
    const bool need_k = top_k < p.vocab, need_p = top_p < 1.f;
    auto value_of = [&](uint64_t at) {  // the logit at a place
        const uint32_t key = (uint32_t)(at >> 32);
        if constexpr (sizeof(Raw) == 4) return L::value(key & 0x80000000u ? key & 0x7fffffffu : ~key);
        else return L::value((Raw)(key & 0x8000u ? key & 0x7fffu : ~key));
    };
    // The same as a logit and the last of this CTA's tokens that is kept with that logit.
    float border_x = -INFINITY;
    int border_i = INT_MAX;
    auto set_border = [&](uint64_t at) {
        border = at, border_x = value_of(at), border_i = (int)~(uint32_t)at - c0;
    };
    auto in_front_of_border = [&](int i, float v) { return v > border_x || (v == border_x && i <= border_i); };
    uint32_t key_least = 0, key_most = 0;  // of the tokens that this thread has gathered
    // Tokens of the bins from `from` to `to`, gathered by each CTA and then brought together in the first: sh.all, by their
    // places. Returns how many (above kMost: not all are there).
    auto gather = [&](int from, int to) {
        ptx::cluster_sync();  // the last gathering's lists, and what lies where they come together, have been read
        if (tid == 0) sh.listed = 0;
        __syncthreads();
        key_least = 0xffffffffu, key_most = 0;
        each_token([&](int i, Raw r) {
            const int b = h.bin(L::value(r));
            if (b < from || b > to) return;
            const uint32_t key = L::key(r), at = atomicAdd(&sh.listed, 1u);
            key_least = min(key_least, key), key_most = max(key_most, key);
            if (at < kMost) sh.list[at] = place(key, c0 + i);
        });
        ptx::cluster_sync();
        int at = 0;
        for (int r = 0; r < cluster; ++r) {
            const int m = (int)ld32(&sh.listed, r);
            if (rank == 0)
                for (int i = tid; i < m && at + i < kMost; i += kThreads) sh.all[at + i] = ld64(&sh.list[i], r);
            at += m;
        }
        __syncthreads();
        return at;
    };
    // sh.all[0 .. m) in falling order (by pairs of elements, a pair to a thread).
    auto sort = [&](int m) {
        int padded = 2;
        while (padded < m) padded *= 2;
        for (int i = m + tid; i < padded; i += kThreads) sh.all[i] = 0;
        __syncthreads();
        for (int run = 2; run <= padded; run *= 2)
            for (int apart = run / 2; apart > 0; apart /= 2) {
                if (tid < padded / 2) {
                    const int i = 2 * tid - (tid & (apart - 1)), j = i + apart;
                    const uint64_t x = sh.all[i], y = sh.all[j];
                    if ((x < y) == ((i & run) == 0)) sh.all[i] = y, sh.all[j] = x;
                }
                __syncthreads();
            }
    };
    auto weight_at = [&](int i, int m) { return i < m ? h.weight(value_of(sh.all[i]), sh.powers, sh.octaves + 1).whole() : 0; };
    // Running sums of two elements of each thread, over the CTA. Returns the whole sum.
    auto scan = [&](const uint64_t (&w)[2], uint64_t (&upto)[2]) {
        uint64_t x = w[0] + w[1];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) sh.sums[0][warp] = x;
        __syncthreads();
        uint64_t all = 0;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
            x += v < warp ? sh.sums[0][v] : 0;
            all += sh.sums[0][v];
        }
        upto[1] = x, upto[0] = x - w[1];
        return all;
    };
    // The last place that is kept of bin `b`: the one with `k` of the bin's tokens up to it, or the first at which the weights
    // up to it reach `target`.
    auto resolve = [&](int b, bool by_mass, uint32_t k, uint64_t target) -> uint64_t {
        const int m = gather(b, b);
        if (m <= kMost) {
            if (rank == 0) {
                sort(m);
                uint64_t w[2] = {weight_at(2 * tid, m), weight_at(2 * tid + 1, m)}, upto[2];
                if (by_mass) scan(w, upto);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (by_mass ? upto[e] - w[e] < target && upto[e] >= target : 2 * tid + e == (int)k - 1) sh.found_border = sh.all[2 * tid + e];
            }
            ptx::cluster_sync();
            return ld64(&sh.found_border, 0);
        }
        // Many tokens: the largest key at which what has a larger or equal one is enough, by halving the range of keys.
        if (tid == 0) sh.key_low = 0xffffffffu, sh.key_high = 0;
        __syncthreads();
        uint32_t least = __reduce_min_sync(0xffffffffu, key_least), most = __reduce_max_sync(0xffffffffu, key_most);
        if (lane == 0) atomicMin(&sh.key_low, least), atomicMax(&sh.key_high, most);
        ptx::cluster_sync();
        for (int r = 0; r < cluster; ++r) least = min(least, ld32(&sh.key_low, r)), most = max(most, ld32(&sh.key_high, r));
        uint64_t low = least, high = (uint64_t)most + 1;  // enough at low, not at high
        uint64_t above_mass = 0;
        uint32_t above_count = 0;
        while (high - low > 1) {
            const uint64_t mid = low + (high - low) / 2;
            uint64_t sum = 0;
            uint32_t count = 0;
            each_token([&](int, Raw r) {
                if (L::key(r) >= mid && h.bin(L::value(r)) == b) sum += by_mass ? h.weight(L::value(r), sh.powers, sh.octaves + 1).whole() : 0, ++count;
            });
            const Sums s = add_up(sum, 0, count);
            if (by_mass ? s.mass >= target : s.count >= k) low = mid;
            else high = mid, above_mass = s.mass, above_count = s.count;
        }
        // Of the tokens with this key, all of one weight, the first ones.
        const uint32_t key = (uint32_t)low;
        const uint64_t each = h.weight(value_of((uint64_t)key << 32), sh.powers, sh.octaves + 1).whole();
        const uint64_t wanted = by_mass ? (target - above_mass + each - 1) / each : k - above_count;
        const long long number = locate([&](int, Raw r) { return (uint64_t)(L::key(r) == key); }, [&](uint64_t) { return wanted - 1; });
        return place(key, (int)number);
    };
    // Draws from the tokens of the bins up to `last`, which hold all that is kept, ranked against each other in one CTA.
    // whole: what top-p is a part of; 0: the sum of the first k, which are all among them.
    auto draw_from_few = [&](int last, uint64_t whole) {
        const int m = gather(0, last);
        if (rank == 0) {
            static_assert(kMost == 2 * kThreads, "two tokens to a thread");
            sort(m);
            uint64_t w[2], upto[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) w[e] = 2 * tid + e < top_k ? weight_at(2 * tid + e, m) : 0;
            const uint64_t sum_k = scan(w, upto), target = need_p ? part_of(whole ? whole : sum_k, top_p, true) : ~0ull;
            // What is kept is a run from the first one on.
            bool kept[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * tid + e;
                kept[e] = w[e] > 0 && (i == 0 || upto[e] - w[e] < target) && value_of(sh.all[i]) >= floor_x;
            }
            const int count = __syncthreads_count(kept[0]) + __syncthreads_count(kept[1]);
            // The same by their numbers, first ones first.
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int i = 2 * tid + e;
                if (!kept[e]) continue;
                sh.weights[i] = w[e];
                sh.all[i] = sh.all[i] << 32 | (uint32_t)i;
            }
            __syncthreads();
            sort(count);
#pragma unroll
            for (int e = 0; e < 2; ++e) w[e] = 2 * tid + e < count ? sh.weights[(uint32_t)sh.all[2 * tid + e]] : 0;
            const uint64_t sum = scan(w, upto), drawn = u < 1.f ? part_of(sum, u, false) : sum - 1;
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (upto[e] > drawn && upto[e] - w[e] <= drawn) p.out[row] = (uint32_t)~(sh.all[2 * tid + e] >> 32);
        }
        ptx::cluster_sync();
    };

    if (need_k || need_p) {
        const int share = kBins / cluster;  // bins that this CTA adds up
        for (int i = tid; i < kBins; i += kThreads) sh.counts[i] = 0;
        __syncthreads();
        each_token([&](int, Raw r) {
            const int b = h.bin(L::value(r));
            if (b < kBins) atomicAdd(&sh.counts[b], 1u);
        });
        ptx::cluster_sync();
        for (int i = tid; i < share; i += kThreads) {
            uint32_t count = 0;
            for (int r = 0; r < cluster; ++r) count += ld32(&sh.counts[rank * share + i], r);
            sh.slice[i] = count;
        }
        ptx::cluster_sync();
        // All bins, in every CTA: a thread has kEach of them, in their order. With bounds of their weights, wide enough for
        // the bins' own rounding. (Counts stay in shared memory, so that no registers are taken through the pass below.)
        constexpr int kEach = kBins / kThreads;
        auto edge = [&](int b) -> uint64_t {  // the largest weight of bin b, the smallest of b - 1: half a bin above its middle
            const int x = max(8 * b - 4, 0) - 1;
            return x >> 8 < 44 ? ((uint64_t)sh.powers[x & 255] << 13) >> ((x >> 8) + 1) : 0;
        };
        auto count_of = [&](int e) -> uint64_t { return sh.bins[tid * kEach + e]; };
        auto most_of = [&](int e) -> uint64_t {
            const uint64_t up = edge(tid * kEach + e);
            return count_of(e) * (up + (up >> 16) + 1);
        };
        auto least_of = [&](int e) -> uint64_t {
            const uint64_t down = edge(tid * kEach + e + 1);
            return count_of(e) * (down - (down >> 16) - (down > 0));
        };
        uint64_t my_most = 0, my_least = 0, my_count = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int b = tid * kEach + e;
            sh.bins[b] = ld32(&sh.slice[b % share], b / share);
            my_count += count_of(e), my_most += most_of(e), my_least += least_of(e);
        }
        // Sums of two such sets over the bins in front of the thread's, and over all.
        auto in_front = [&](uint64_t a, uint64_t b, uint64_t *a_all, uint64_t *b_all, uint64_t *b_front) {
            uint64_t x = a, y = b;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t v = __shfl_up_sync(0xffffffffu, x, o), w = __shfl_up_sync(0xffffffffu, y, o);
                if (lane >= o) x += v, y += w;
            }
            __syncthreads();
            if (lane == 31) sh.sums[0][warp] = x, sh.sums[1][warp] = y;
            __syncthreads();
            x -= a, y -= b, *a_all = 0, *b_all = 0;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) x += sh.sums[0][w], y += sh.sums[1][w];
                *a_all += sh.sums[0][w], *b_all += sh.sums[1][w];
            }
            *b_front = y;
            return x;
        };
        uint64_t all_most, all_least, all_count, none, before_least, none2;
        const uint64_t before_most = in_front(my_most, my_least, &all_most, &all_least, &before_least);
        const uint64_t before_count = in_front(my_count, 0, &all_count, &none, &none2);
        // The first bin at which the running sum of `each` (from `before` at the thread's first bin) reaches `target`; kBins: none.
        auto find = [&](uint64_t before, auto each, uint64_t target) {
            __syncthreads();
            if (tid == 0) sh.found.bin = kBins;
            __syncthreads();
            uint64_t x = before, c = before_count, m = before_most, l = before_least;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const uint64_t y = each(e);
                if (x < target && x + y >= target)
                    sh.found = Found{(uint32_t)(tid * kEach + e), (uint32_t)c, (uint32_t)count_of(e), m, l, most_of(e), least_of(e)}, sh.found_mass = x;
                x += y, c += count_of(e), m += most_of(e), l += least_of(e);
            }
            __syncthreads();
            return sh.found;
        };
        int bin_k = kBins;
        uint64_t whole_least = all_least, whole_most = all_most;
        if (need_k && (uint64_t)top_k < all_count) {
            const Found f = find(before_count, count_of, (uint64_t)top_k);
            bin_k = (int)f.bin;
            if (f.before + f.in <= kMost) {
                draw_from_few(bin_k, 0);
                return;
            }
            whole_least = f.least_before, whole_most = f.most_before + f.most_in;
            set_border(resolve(bin_k, false, (uint32_t)top_k - f.before, 0));
        } else if (all_count <= kMost) {
            draw_from_few(kBins - 1, 0);
            return;
        }
        if (need_p) {
            // The border lies in one of these bins.
            const Found first = find(before_most, most_of, max(part_of(whole_least, top_p, true), (uint64_t)1));
            const Found last = find(before_least, least_of, part_of(whole_most, top_p, true));
            const int from = min((int)first.bin, kBins - 1), to = max(from, min((int)last.bin, min(bin_k, kBins - 1)));
            ptx::cluster_sync();  // nobody looks at gathered tokens any more
            for (int b = from + tid; b <= to; b += kThreads) sh.parts[0][b] = sh.parts[1][b] = 0;
            __syncthreads();
            uint64_t behind = 0, front = 0;
            each_token([&](int i, Raw r) {
                const float v = L::value(r);
                if (border != 0 && !in_front_of_border(i, v)) return;
                const typename Heat::Weight y = h.weight(v, sh.powers, sh.octaves + 1);
                const int b = h.bin(v);
                (b < from ? front : behind) += y.whole();
                if (b >= from && b <= to) {
                    const uint64_t w = y.whole();
                    const uint32_t old = atomicAdd(&sh.parts[0][b], (uint32_t)w), up = (uint32_t)(w >> 32) + (old + (uint32_t)w < old);
                    if (up) atomicAdd(&sh.parts[1][b], up);
                }
            });
            const Sums s = add_up(front + behind, front, 0);
            uint64_t mass[kEach], my_mass = 0, all_mass;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int b = tid * kEach + e;
                mass[e] = 0;
                if (b >= from && b <= to)
                    for (int r = 0; r < cluster; ++r) mass[e] += ((uint64_t)ld32(&sh.parts[1][b], r) << 32) + ld32(&sh.parts[0][b], r);
                my_mass += mass[e];
            }
            const uint64_t before_mass = s.front + in_front(my_mass, 0, &all_mass, &none, &none2);
            const uint64_t target = part_of(s.mass, top_p, true);
            // (The bins in front of these have no mass here: what is in them is in s.front.)
            const Found f = find(before_mass, [&](int e) { return mass[e]; }, target);
            const uint64_t reached = sh.found_mass;
            if (f.bin < kBins) {
                if (border == 0 && f.before + f.in <= kMost) {
                    draw_from_few((int)f.bin, s.mass);
                    return;
                }
                const uint64_t at = resolve((int)f.bin, true, 0, target - reached);
                if (at > border) set_border(at);
            }
        }
    }

    // ---------------------------------------------------------------- the sum of what is kept, and the token
    if (floor_x > border_x) border_x = floor_x, border_i = INT_MAX;
    auto kept = [&](int i, Raw r) -> uint64_t {
        const float v = L::value(r);
        const typename Heat::Weight w = h.weight(v, sh.powers, sh.octaves + 1);
        return (uint64_t)w.part * (in_front_of_border(i, v) ? w.up : 0u);
    };
    const long long token = locate(kept, [&](uint64_t whole) { return u < 1.f ? part_of(whole, u, false) : whole - 1; });
    if (rank == 0 && tid == 0) p.out[row] = token;
    ptx::cluster_sync();
}

template <typename T>
cudaError_t launch(SampleParams p, int rows, int sms, cudaStream_t s) {
    // CTAs of a row: as many as its tokens need room, and as many as there are SMs for (what a CTA does whatever it has costs
    // as much as a pass over 10000 logits: 256 rows of 150001 took 342 us with 4 CTAs to a row, 463 with 8, in an earlier form).
    // (Two CTAs share an SM's 228 KB, of which each leaves 1 KB to the system.)
    const int room = (int)((113 * 1024 - sizeof(Shared<T>) - 64) / sizeof(T));
    int cluster = 1;
    while (cluster < kMaxCluster && ((p.vocab + cluster - 1) / cluster > room || (rows * cluster <= 2 * sms && p.vocab > 4096 * cluster)))
        cluster *= 2;
    p.chunk = (p.vocab + cluster - 1) / cluster;
    const int smem = (int)sizeof(Shared<T>) + (p.chunk + 16) * (int)sizeof(T) + 16;
    auto kernel = sample_kernel<T>;
    cudaError_t e = ensure_max_dyn_smem((const void *)kernel, 227 * 1024);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * cluster), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = as_dependent(s) ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

w4a16_status w4a16_sample(const void *logits, w4a16_type type, long long row, int rows, int vocab, const float *uniform,
                          const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p, int64_t *out,
                          void *stream) {
    if (type != W4A16_TYPE_F16 && type != W4A16_TYPE_BF16 && type != W4A16_TYPE_F32) return W4A16_ERR_INVALID_ARG;
    if (rows < 0 || vocab <= 0 || row < 0 || (rows > 1 && row < vocab)) return W4A16_ERR_INVALID_ARG;
    if (vocab > kMaxVocab || rows > (1 << 20)) return W4A16_ERR_UNSUPPORTED;
    if (rows == 0) return W4A16_OK;
    if (!logits || !uniform || !out) return W4A16_ERR_INVALID_ARG;
    if (!aligned(logits, type == W4A16_TYPE_F32 ? 4 : 2) || !aligned(out, 8)) return W4A16_ERR_INVALID_ARG;
    for (const void *x : {(const void *)uniform, (const void *)temperature, (const void *)top_k, (const void *)top_p, (const void *)min_p})
        if (!aligned(x, 4)) return W4A16_ERR_INVALID_ARG;
    SampleParams p{logits, row, uniform, temperature, top_p, min_p, top_k, out, vocab, 0, device_error_ptr()};
    if (!p.err) return W4A16_ERR_CUDA;
    cudaStream_t s = (cudaStream_t)stream;
    if (type == W4A16_TYPE_F16) return from_cuda(launch<__half>(p, rows, sm_count(), s));
    if (type == W4A16_TYPE_BF16) return from_cuda(launch<__nv_bfloat16>(p, rows, sm_count(), s));
    return from_cuda(launch<float>(p, rows, sm_count(), s));
}

w4a16_status w4a16_sample_block(const w4a16_sample_args *args) {
    if (!args) return W4A16_ERR_INVALID_ARG;
    const w4a16_sample_args &a = *args;
    return w4a16_sample(a.logits, (w4a16_type)a.type, a.row, a.rows, a.vocab, a.uniform, a.temperature, a.top_k, a.top_p, a.min_p,
                        a.out, a.stream);
}

}  // extern "C"
