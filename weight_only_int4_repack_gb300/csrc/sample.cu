// The next token of each row of logits: temperature, top-k, top-p, min-p, with a given random number.
//     w_i = 2^(-(max - x_i) log2(e) / T); of the tokens in the order of falling x (equal ones by number) the first k, of
//     these the fewest whose weights reach p of theirs, of these the ones with w_i >= min_p; the token drawn is the first, by
//     number, at which the kept weights' running sum exceeds u times their sum
// Bound by HBM at best (each logit is read once), in practice by the steps' latencies: a row is one cluster of CTAs, which
// keeps its logits in shared memory, and every step that all of them have to agree on is a cluster barrier.
//
// Weights are fixed-point numbers of 44 binary places in 64-bit integers, off by less than 2^-31 of themselves: sums are
// exact and so do not depend on any order, and a border between two tokens moves by less than 2^-31 of the sum, about what
// it would take for a 32-bit random number to show it. A weight below 2^-44 of the largest is 0.
//
// The border of top-k and top-p is found by a histogram over 32 bins for each factor of two of the weight (counts, and for
// top-p sums): the bin that holds it, then in that bin. Where few tokens lie above the border (as a rule) they are gathered,
// and one CTA ranks them against each other and draws; otherwise the border's bin is resolved (by ranking its tokens, or, when
// it holds many, by halving the range of its values) and a second pass over shared memory sums and draws.
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
    int vocab, chunk;  // tokens of a CTA, a multiple of kThreads
    unsigned int *err;
};

// 2^(-i/256) with 32 binary places: from the series of exp, the first entry one unit short of 1.
struct Table {
    uint32_t v[256];
};
constexpr Table make_table() {
    Table t{};
    for (int i = 0; i < 256; ++i) {
        const double y = -0.69314718055994530942 * i / 256;
        double term = 1, sum = 1;
        for (int k = 1; k < 30; ++k) term *= y / k, sum += term;
        const double scaled = sum * 4294967296.0 + 0.5;
        t.v[i] = scaled >= 4294967295.0 ? 0xffffffffu : (uint32_t)scaled;
    }
    return t;
}
__constant__ Table kPowers = make_table();

// A row's weights.
struct Heat {
    float top, c, c_low;  // largest logit; log2(e) / temperature in two parts
    __device__ __forceinline__ float down(float x) const { return x == top ? 0.f : top - x; }
    // How far below the largest, in factors of two; NaN and what is far below: 64 and more.
    __device__ __forceinline__ float octaves(float x) const {
        const float t = down(x) * c;
        return t < 64.f ? t : 64.f;
    }
    __device__ __forceinline__ uint64_t weight(float x, const uint32_t *powers) const {
        const float d = down(x), t = d * c;
        if (!(t < 64.f)) return 0;
        // The difference's rounding and the product's, and the factor's second part.
        const float rest = x == top ? 0.f : (top - d) - x;
        const float low = fmaf(d, c, -t) + fmaf(d, c_low, rest * c);
        const float whole = floorf(t);
        const uint64_t fixed = ((uint64_t)(uint32_t)whole << 32) + (uint64_t)((t - whole) * 4294967296.f) + (uint64_t)(int64_t)(low * 4294967296.f);
        if ((int64_t)fixed <= 0) return (uint64_t)powers[0] << 12;
        const uint32_t n = (uint32_t)(fixed >> 32), f = (uint32_t)fixed;
        // 2^-f: a table for the first 8 bits, three terms of 1 - 2^-y for the others (y < 2^-8, the next term is below 2^-37).
        const float y = (float)(f & 0xffffffu) * (0.693147180559945f / 4294967296.f);
        const float e = y * fmaf(y, fmaf(y, 1.f / 6, -0.5f), 1.f);
        const uint32_t p = powers[f >> 24];
        const uint32_t w = p - __umulhi(p, (uint32_t)(e * 4294967296.f));
        return n < 44 ? ((uint64_t)w << 12) >> n : 0;
    }
};

// Logits as numbers in their order: larger logits larger, -0 as 0.
template <typename T>
struct Logit;
template <>
struct Logit<float> {
    static constexpr int kBits = 32;
    using Raw = uint32_t;
    static __device__ __forceinline__ float value(Raw r) { return __uint_as_float(r); }
    static __device__ __forceinline__ uint32_t key(Raw r) {
        if (r == 0x80000000u) r = 0;
        return r & 0x80000000u ? ~r : r | 0x80000000u;
    }
};
template <typename H>
struct Logit16 {
    static constexpr int kBits = 16;
    using Raw = uint16_t;
    static __device__ __forceinline__ float value(Raw r) { return elem::pair_to_f32<H>(r).x; }
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

struct Pair {
    uint64_t mass;
    uint32_t count;
};

template <typename T>
struct alignas(16) Shared {
    uint32_t counts[kBins], low[kBins], high[kBins];  // the CTA's histogram: tokens, and sums of weights in two halves
    uint64_t slice_mass[kBins];   // of this CTA's share of the bins, over the cluster
    uint32_t slice_count[kBins];
    uint64_t list[kMost];         // this CTA's gathered tokens: key, then number counted down
    uint32_t listed;
    uint64_t all[kMost], weights[kMost];  // the cluster's
    uint32_t powers[256];
    uint64_t mass_slot[4];        // what a step adds up over the cluster
    uint32_t count_slot[4];
    float max_slot;
    uint32_t number_slot;
    uint64_t sums[kWarps];
    uint32_t sums32[kWarps];
    uint64_t scan_mass[kWarps];
    uint64_t found_mass, found_border;
    uint32_t found_bin, found_count, found_rank;
    long long token;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleParams p) {
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
    const int skew = (int)((uintptr_t)x % 16 / sizeof(Raw));
    Raw *mine = reinterpret_cast<Raw *>(raw_smem + sizeof(Shared<T>)) + skew;  // token c0 + i at mine[i]

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
    float top = -INFINITY;
    {
        const int blocks = (skew + n + kVec - 1) / kVec;
#pragma unroll 4
        for (int b = tid; b < blocks; b += kThreads) {
            const int i = b * kVec - skew;
            if (i >= 0 && i + kVec <= n) {
                const uint4 v = *reinterpret_cast<const uint4 *>(x + i);
                *reinterpret_cast<uint4 *>(mine + i) = v;
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    if constexpr (sizeof(Raw) == 4) {
                        top = fmaxf(top, __uint_as_float(w[z]));
                    } else {
                        const float2 f = elem::pair_to_f32<T>(w[z]);
                        top = fmaxf(top, fmaxf(f.x, f.y));
                    }
                }
            } else {
                for (int j = max(i, 0); j < min(i + kVec, n); ++j) {
                    const Raw r = x[j];
                    mine[j] = r;
                    top = fmaxf(top, L::value(r));
                }
            }
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
    auto add_up = [&](uint64_t mass, uint32_t count) {
        mass = warp_sum(mass);
        count = __reduce_add_sync(0xffffffffu, count);
        __syncthreads();
        if (lane == 0) sh.sums[warp] = mass, sh.sums32[warp] = count;
        __syncthreads();
        const int slot = step++ & 3;
        if (warp == 0) {
            mass = warp_sum(lane < kWarps ? sh.sums[lane] : 0);
            count = __reduce_add_sync(0xffffffffu, lane < kWarps ? sh.sums32[lane] : 0u);
            if (lane == 0) sh.mass_slot[slot] = mass, sh.count_slot[slot] = count;
        }
        ptx::cluster_sync();
        Pair all{0, 0};
        for (int r = 0; r < cluster; ++r) all.mass += ld64(&sh.mass_slot[slot], r), all.count += ld32(&sh.count_slot[slot], r);
        return all;
    };
    // The first token, by number, at which the running sum of `what` over the row exceeds `target` (which is below the
    // whole sum). A warp has consecutive tokens.
    const int seg = p.chunk / kWarps, s0 = min(warp * seg, n), s1 = min(s0 + seg, n);
    auto locate = [&](auto what, uint64_t target) -> long long {
        uint64_t sum = 0;
        for (int i = s0 + lane; i < s1; i += 32) sum += what(i);
        sum = warp_sum(sum);
        __syncthreads();
        if (lane == 0) sh.scan_mass[warp] = sum;
        if (tid == 0) sh.token = -1;
        __syncthreads();
        const int slot = step++ & 3;
        if (tid == 0) {
            uint64_t all = 0;
            for (int w = 0; w < kWarps; ++w) all += sh.scan_mass[w];
            sh.mass_slot[slot] = all;
        }
        ptx::cluster_sync();
        uint64_t before = 0;
        for (int r = 0; r < rank; ++r) before += ld64(&sh.mass_slot[slot], r);
        for (int w = 0; w < warp; ++w) before += sh.scan_mass[w];
        if (before <= target && target < before + sum) {  // in this warp's tokens
            for (int i0 = s0; i0 < s1; i0 += 32) {
                const uint64_t w = i0 + lane < s1 ? what(i0 + lane) : 0;
                uint64_t upto = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t y = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= o) upto += y;
                }
                const uint32_t mask = __ballot_sync(0xffffffffu, before + upto > target);
                if (mask) {
                    if (lane == 0) sh.token = c0 + i0 + __ffs(mask) - 1;
                    break;
                }
                before += __shfl_sync(0xffffffffu, upto, 31);
            }
        }
        ptx::cluster_sync();
        long long token = -1;
        for (int r = 0; r < cluster; ++r) token = max(token, (long long)ld64(reinterpret_cast<const uint64_t *>(&sh.token), r));
        return token;
    };

    const bool nothing = top == -INFINITY;                                     // no token may be drawn
    const bool greedy = heat == 0.f || top_k == 1 || top_p <= 0.f || min_p > 1.f;  // the largest logit, the first of equal ones
    if (nothing || greedy) {
        uint32_t first = 0xffffffffu;
        if (!nothing)
            for (int i = tid; i < n; i += kThreads)
                if (L::value(mine[i]) == top) {
                    first = c0 + i;
                    break;
                }
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

    Heat h;
    {
        const double c = 1.4426950408889634 / (double)heat;
        h.top = top;
        h.c = c < 3e38 ? (float)c : 3e38f;
        h.c_low = c < 3e38 ? (float)(c - (double)h.c) : 0.f;
    }
    // The smallest logit that min-p leaves, rounded up.
    float floor_x = -INFINITY;
    if (min_p > 0.f && top < INFINITY) {
        const double cut = (double)top + (double)heat * log((double)min_p);
        if (cut == cut) floor_x = __double2float_ru(cut);
    }
    auto key_of = [&](int i) { return L::key(mine[i]); };
    auto bin_of = [&](int i) {
        const float t = h.octaves(L::value(mine[i]));
        return t < 64.f ? (int)(t * kPerOctave) : kBins;
    };

    // ---------------------------------------------------------------- the border of top-k and top-p
    // Kept is what lies in front of the border in the order of falling keys, equal ones by number, the border included:
    // a 64-bit number, larger for what comes first.
    auto place = [&](uint32_t key, int number) { return (uint64_t)key << 32 | (uint32_t)~number; };
    uint64_t border = 0;  // everything
    const bool need_k = top_k < p.vocab, need_p = top_p < 1.f;
    if (need_k || need_p) {
        const int share = kBins / cluster;  // bins that this CTA adds up
        bool with_mass = !need_k;
        for (;;) {
            for (int i = tid; i < kBins; i += kThreads) sh.counts[i] = sh.low[i] = sh.high[i] = 0;
            if (tid == 0) sh.listed = 0;
            __syncthreads();
            for (int i = tid; i < n; i += kThreads) {
                const int b = bin_of(i);
                if (b >= kBins) continue;
                atomicAdd(&sh.counts[b], 1u);
                if (with_mass) {
                    const uint64_t w = h.weight(L::value(mine[i]), sh.powers);
                    const uint32_t old = atomicAdd(&sh.low[b], (uint32_t)w);
                    const uint32_t up = (uint32_t)(w >> 32) + (old + (uint32_t)w < old);
                    if (up) atomicAdd(&sh.high[b], up);
                }
            }
            ptx::cluster_sync();
            for (int i = tid; i < share; i += kThreads) {
                uint64_t mass = 0;
                uint32_t count = 0;
                for (int r = 0; r < cluster; ++r) {
                    count += ld32(&sh.counts[rank * share + i], r);
                    if (with_mass) mass += (uint64_t)ld32(&sh.high[rank * share + i], r) << 32 | 0, mass += ld32(&sh.low[rank * share + i], r);
                }
                sh.slice_mass[i] = mass, sh.slice_count[i] = count;
            }
            ptx::cluster_sync();
            // All bins' sums, in every CTA: a thread has kBins / kThreads of them, in their order.
            constexpr int kEach = kBins / kThreads;
            uint64_t mass[kEach];
            uint32_t count[kEach];
            uint64_t my_mass = 0;
            uint32_t my_count = 0;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int b = tid * kEach + e;
                count[e] = ld32(&sh.slice_count[b % share], b / share);
                mass[e] = with_mass ? ld64(&sh.slice_mass[b % share], b / share) : 0;
                my_mass += mass[e], my_count += count[e];
            }
            uint64_t upto_mass = my_mass;
            uint32_t upto_count = my_count;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t a = __shfl_up_sync(0xffffffffu, upto_mass, o);
                const uint32_t b = __shfl_up_sync(0xffffffffu, upto_count, o);
                if (lane >= o) upto_mass += a, upto_count += b;
            }
            if (lane == 31) sh.sums[warp] = upto_mass, sh.sums32[warp] = upto_count;
            __syncthreads();
            uint64_t all_mass = 0, before_mass = upto_mass - my_mass;
            uint32_t all_count = 0, before_count = upto_count - my_count;
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) before_mass += sh.sums[w], before_count += sh.sums32[w];
                all_mass += sh.sums[w], all_count += sh.sums32[w];
            }
            // The bin in which the count reaches `k`, or the mass `target`: found_bin, and what lies in front of it.
            auto find = [&](bool by_mass, uint32_t k, uint64_t target) {
                __syncthreads();
                if (tid == 0) sh.found_bin = kBins;
                __syncthreads();
                uint64_t m = before_mass;
                uint32_t c = before_count;
#pragma unroll
                for (int e = 0; e < kEach; ++e) {
                    const bool in_front = by_mass ? m < target : c < k;
                    const bool reached = by_mass ? m + mass[e] >= target : c + count[e] >= k;
                    if (in_front && reached) sh.found_bin = tid * kEach + e, sh.found_mass = m, sh.found_count = c, sh.found_rank = count[e];
                    m += mass[e], c += count[e];
                }
                __syncthreads();
            };
            // Tokens of the bins from `from` to `to`, gathered by each CTA and then brought together in every one: sh.all,
            // by their places. Returns how many (above kMost: none gathered).
            auto gather = [&](int from, int to) {
                ptx::cluster_sync();  // the last gathering's lists have been read
                if (tid == 0) sh.listed = 0;
                __syncthreads();
                for (int i = tid; i < n; i += kThreads) {
                    const int b = bin_of(i);
                    if (b < from || b > to) continue;
                    const uint32_t at = atomicAdd(&sh.listed, 1u);
                    if (at < kMost) sh.list[at] = place(key_of(i), c0 + i);
                }
                ptx::cluster_sync();
                int at = 0;
                for (int r = 0; r < cluster; ++r) {
                    const int m = (int)ld32(&sh.listed, r);
                    for (int i = tid; i < m && at + i < kMost; i += kThreads) sh.all[at + i] = ld64(&sh.list[i], r);
                    at += m;
                }
                __syncthreads();
                return at;
            };
            auto value_of = [&](uint64_t at) {  // the logit at a place
                const uint32_t key = (uint32_t)(at >> 32);
                if constexpr (sizeof(Raw) == 4) return L::value(key & 0x80000000u ? key & 0x7fffffffu : ~key);
                else return L::value((Raw)(key & 0x8000u ? key & 0x7fffu : ~key));
            };

            uint32_t before_k = 0, in_k = 0;
            int bin_k = kBins;
            if (need_k && (uint32_t)top_k < all_count) {
                find(false, (uint32_t)top_k, 0);
                bin_k = (int)sh.found_bin, before_k = sh.found_count, in_k = sh.found_rank;
            }
            // The last bin of interest and the tokens up to it.
            int bin_last = bin_k;
            uint32_t tokens = bin_k < kBins ? before_k + in_k : all_count;
            if (!need_k) {  // all_mass is the whole
                find(true, 0, part_of(all_mass, top_p, true));
                if (sh.found_bin < kBins) bin_last = (int)sh.found_bin, tokens = sh.found_count + sh.found_rank;
            }
            if (tokens <= kMost) {
                // ------------------------------------------------ few: ranked against each other
                const int m = gather(0, min(bin_last, kBins - 1));
                if (rank == 0) {
                    for (int i = tid; i < m; i += kThreads) sh.weights[i] = h.weight(value_of(sh.all[i]), sh.powers);
                    __syncthreads();
                    constexpr int kMine = kMost / kThreads;
                    uint64_t in_front[kMine];
                    uint32_t ranked[kMine];
                    uint64_t sum = 0;
#pragma unroll
                    for (int e = 0; e < kMine; ++e) {
                        const int i = tid + e * kThreads;
                        in_front[e] = 0, ranked[e] = 0;
                        if (i >= m) continue;
                        const uint64_t at = sh.all[i];
#pragma unroll 4
                        for (int j = 0; j < m; ++j)
                            if (sh.all[j] > at) in_front[e] += sh.weights[j], ++ranked[e];
                        if (ranked[e] < (uint32_t)top_k) sum += sh.weights[i];
                    }
                    auto block_sum = [&](uint64_t v) {
                        v = warp_sum(v);
                        __syncthreads();
                        if (lane == 0) sh.sums[warp] = v;
                        __syncthreads();
                        v = 0;
                        for (int w = 0; w < kWarps; ++w) v += sh.sums[w];
                        return v;
                    };
                    // Of the first k the whole is their sum; without top-k it is that of all tokens.
                    const uint64_t whole = need_k ? block_sum(sum) : all_mass;
                    const uint64_t target = need_p ? part_of(whole, top_p, true) : ~0ull;
                    sum = 0;
                    bool kept[kMine];
#pragma unroll
                    for (int e = 0; e < kMine; ++e) {
                        const int i = tid + e * kThreads;
                        kept[e] = i < m && ranked[e] < (uint32_t)top_k && (ranked[e] == 0 || in_front[e] < target) &&
                                  value_of(sh.all[i]) >= floor_x;
                        if (kept[e]) sum += sh.weights[i];
                    }
                    sum = block_sum(sum);
#pragma unroll
                    for (int e = 0; e < kMine; ++e) {
                        const int i = tid + e * kThreads;
                        if (i < m && !kept[e]) sh.weights[i] = 0;
                    }
                    __syncthreads();
                    const uint64_t drawn = u < 1.f ? part_of(sum, u, false) : sum - 1;
#pragma unroll
                    for (int e = 0; e < kMine; ++e) {
                        const int i = tid + e * kThreads;
                        if (i >= m || sh.weights[i] == 0) continue;
                        const uint32_t number = ~(uint32_t)sh.all[i];
                        uint64_t before = 0;
#pragma unroll 4
                        for (int j = 0; j < m; ++j)
                            if (~(uint32_t)sh.all[j] < number) before += sh.weights[j];
                        if (before <= drawn && drawn < before + sh.weights[i]) p.out[row] = number;
                    }
                }
                ptx::cluster_sync();
                return;
            }
            if (need_p && !with_mass) {  // again, with sums of weights
                with_mass = true;
                ptx::cluster_sync();
                continue;
            }
            // ---------------------------------------------------- many: the border in its bin
            // Finds in bin `b` the last place that is kept: the one with `k` tokens of the bin in front of and including it, or
            // the first at which the mass in the bin reaches `target`. Returns its place and the bin's mass up to it.
            auto resolve = [&](int b, bool by_mass, uint32_t k, uint64_t target, uint64_t *upto) -> uint64_t {
                const int m = gather(b, b);
                if (m <= kMost) {
                    for (int i = tid; i < m; i += kThreads) sh.weights[i] = h.weight(value_of(sh.all[i]), sh.powers);
                    __syncthreads();
                    for (int i = tid; i < m; i += kThreads) {
                        const uint64_t at = sh.all[i];
                        uint64_t in_front = 0;
                        uint32_t ranked = 0;
                        for (int j = 0; j < m; ++j)
                            if (sh.all[j] > at) in_front += sh.weights[j], ++ranked;
                        const bool last = by_mass ? in_front < target && in_front + sh.weights[i] >= target : ranked + 1 == k;
                        if (last) sh.found_border = at, sh.found_mass = in_front + sh.weights[i];
                    }
                    __syncthreads();
                    *upto = sh.found_mass;
                    const uint64_t at = sh.found_border;
                    __syncthreads();
                    return at;
                }
                // Many tokens in the bin: the largest key at which what has a larger or equal one is enough, by halving.
                uint64_t low = 0, high = 1ull << L::kBits;  // enough at low, not at high
                uint64_t above_mass = 0;
                uint32_t above_count = 0;
                while (high - low > 1) {
                    const uint64_t mid = low + (high - low) / 2;
                    uint64_t sum = 0;
                    uint32_t count_here = 0;
                    for (int i = tid; i < n; i += kThreads)
                        if (bin_of(i) == b && key_of(i) >= mid) sum += by_mass ? h.weight(L::value(mine[i]), sh.powers) : 0, ++count_here;
                    const Pair s = add_up(sum, count_here);
                    if (by_mass ? s.mass >= target : s.count >= k) low = mid;
                    else high = mid, above_mass = s.mass, above_count = s.count;
                }
                // Of the tokens with this key, all of one weight, the first ones.
                const uint32_t key = (uint32_t)low;
                const uint64_t each = h.weight(value_of((uint64_t)key << 32), sh.powers);
                const uint64_t wanted = by_mass ? (target - above_mass + each - 1) / each : k - above_count;
                const long long number = locate([&](int i) { return (uint64_t)(key_of(i) == key); }, wanted - 1);
                if (!by_mass) {  // the sum of what lies above was not asked for
                    uint64_t sum = 0;
                    for (int i = tid; i < n; i += kThreads)
                        if (bin_of(i) == b && key_of(i) > key) sum += h.weight(L::value(mine[i]), sh.powers);
                    above_mass = add_up(sum, 0).mass;
                }
                *upto = above_mass + wanted * each;
                return place(key, (int)number);
            };
            uint64_t whole = all_mass, in_bin = 0;
            if (bin_k < kBins) {
                find(false, (uint32_t)top_k, 0);
                const uint64_t in_front = sh.found_mass;
                const uint32_t first = sh.found_count;
                border = resolve(bin_k, false, (uint32_t)top_k - first, 0, &in_bin);
                whole = in_front + in_bin;  // with need_p the histogram has sums
            }
            if (need_p) {
                const uint64_t target = part_of(whole, top_p, true);
                find(true, 0, target);
                if (sh.found_bin < kBins) {
                    const int b = (int)sh.found_bin;
                    const uint64_t in_front = sh.found_mass;
                    const uint64_t at = resolve(b, true, 0, target - in_front, &in_bin);
                    border = border > at ? border : at;
                }
            }
            break;
        }
    }

    // ---------------------------------------------------------------- the sum of what is kept, and the token
    const uint32_t border_key = (uint32_t)(border >> 32);
    auto kept = [&](int i) -> uint64_t {
        const float v = L::value(mine[i]);
        if (!(v >= floor_x)) return 0;
        const uint32_t key = key_of(i);
        if (key < border_key || (key == border_key && (uint32_t)~(c0 + i) < (uint32_t)border)) return 0;
        return h.weight(v, sh.powers);
    };
    uint64_t sum = 0;
    for (int i = tid; i < n; i += kThreads) sum += kept(i);
    sum = add_up(sum, 0).mass;
    const long long token = locate(kept, u < 1.f ? part_of(sum, u, false) : sum - 1);
    if (rank == 0 && tid == 0) p.out[row] = token;
    ptx::cluster_sync();
}

template <typename T>
cudaError_t launch(SampleParams p, int rows, int sms, cudaStream_t s) {
    // CTAs of a row: as many as its tokens need room, and as many as there are SMs for.
    const int room = (int)((size_t)96 * 1024 / sizeof(T));
    int cluster = 1;
    while (cluster < kMaxCluster && ((p.vocab + cluster - 1) / cluster > room || (rows * cluster * 2 <= 2 * sms && p.vocab > 4096 * cluster)))
        cluster *= 2;
    p.chunk = ((p.vocab + cluster - 1) / cluster + kThreads - 1) / kThreads * kThreads;
    const int smem = (int)sizeof(Shared<T>) + (p.chunk + 16) * (int)sizeof(T);
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
