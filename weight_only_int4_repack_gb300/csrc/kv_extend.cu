// Block tables, slots and positions of a step's new tokens, from the requests'
// lengths, in one launch. Whole-number work of a few hundred kilobytes at most,
// bound by latency: two prefix sums over the requests, then every page handed out
// and every token finds its place by itself.
//
// One cluster of CTAs does it all. Each CTA runs the prefix sums over all requests
// for itself (a few values per thread; sharing them would cost a wait), and keeps
// each request's figures in shared memory. Pages given back are written to the free
// list, a cluster barrier makes them visible, and after it, when every CTA has read
// its inputs, everything is written, so that lengths and count may be updated in
// place.
//
// Measured (GB300, in a CUDA graph): 48 requests with a token each 4.4 us; 1501 requests
// with 40 thousand tokens, prompts and ended ones among them, 14.4 us (1.4 of it until
// the inputs are there, 3.4 the sums and needs, 1.3 the cluster's barrier, the rest pages
// and slots); 300 requests with pages of a single token 20 us.
#include <climits>

#include "decode_ops.h"
#include "ptx.cuh"

namespace w4a16 {
namespace {

struct ExtendParams {
    const int32_t *lens, *new_tokens, *free_count;
    int32_t *table, *free_pages, *lens_out, *free_count_out, *positions, *refused;
    int64_t *slots;
    long long table_stride;
    int batch, max_pages, page_size, pool, n_slots;
    unsigned int magic, shift;  // n / page_size = n * magic >> shift for 0 <= n < 2^31
    int spacing;  // slots from one request's first token to the next one's; 0: they follow each other
    unsigned int *err;
    bool overlap;
};

constexpr int kMostThreads = 1024;
constexpr int kMaxBatch = 8192;

// A request's figures, kept in shared memory. What it has of the step's tokens, of the
// pages handed out and of those given back begins where three more arrays say (never
// less than for the request before it, so they can be searched).
struct Request {
    int len;   // tokens before the step; negative: it gets none (kRefused..., kEnded)
    int held;  // pages before the step
};
constexpr int kRequestBytes = sizeof(Request) + 3 * sizeof(int);
constexpr int kRefusedPages = -1, kRefusedRoom = -2, kEnded = -3;

// Inclusive prefix sums of N values over the CTA's threads; totals are the sums of all.
template <int N>
__device__ __forceinline__ void scan(long long (&x)[N], long long (*sums)[32], long long (&totals)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x / 32;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const long long y = __shfl_up_sync(0xffffffffu, x[n], o);
            if (lane >= o) x[n] += y;
        }
    if (lane == 31)
#pragma unroll
        for (int n = 0; n < N; ++n) sums[n][warp] = x[n];
    __syncthreads();
    long long s[N];  // every warp sums the warps' sums for itself
#pragma unroll
    for (int n = 0; n < N; ++n) s[n] = lane < warps ? sums[n][lane] : 0;
    for (int o = 1; o < warps; o <<= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const long long y = __shfl_up_sync(0xffffffffu, s[n], o);
            if (lane >= o) s[n] += y;
        }
#pragma unroll
    for (int n = 0; n < N; ++n) {
        totals[n] = __shfl_sync(0xffffffffu, s[n], warps - 1);
        const long long in_front = __shfl_sync(0xffffffffu, s[n], max(warp - 1, 0));
        if (warp) x[n] += in_front;
    }
}

__global__ void __launch_bounds__(kMostThreads) kv_extend_kernel(const ExtendParams p) {
    extern __shared__ Request req[];  // [batch], then first token, page handed out and page given back of each
    int *starts = reinterpret_cast<int *>(req + p.batch), *first_page = starts + p.batch, *first_given = first_page + p.batch;
    __shared__ long long warp_sums[3][32];
    __shared__ long long taken;
    if (p.overlap) ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int ctas = gridDim.x, cta = blockIdx.x, tid = threadIdx.x, threads = blockDim.x;
    if (tid == 0) taken = 0;
    const int per = (p.batch + threads - 1) / threads;  // consecutive requests of a thread
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    const unsigned int ps = (unsigned int)p.page_size;
    const long long room = min((long long)p.max_pages * ps, (long long)INT_MAX);
    const long long count0 = min(max(p.free_count[0], 0), p.pool);
    auto by_page = [&](int n) { return (int)(((unsigned long long)(unsigned int)n * p.magic) >> p.shift); };  // n / ps
    auto pages = [&](int n) {  // n / ps, rounded up
        const int whole = by_page(n);
        return whole + (n > whole * p.page_size);
    };

    auto first_slot = [&](int b, long long at) { return p.spacing ? (long long)b * p.spacing : at; };
    auto fits = [&](int b, int len, int add, long long at) {
        return add >= 0 && len >= 0 && (long long)len + add <= room &&
               (add == 0 || (first_slot(b, at) + add <= p.n_slots && (!p.spacing || add <= p.spacing)));
    };

    auto wrong = [&] { atomicExch(p.err, (unsigned int)W4A16_ERR_INVALID_ARG); };

    // Tokens and pages given back, in front of each request.
    long long tokens = 0, given = 0;
    for (int b = b0; b < b1; ++b) {
        const int len = p.lens[b], add = p.new_tokens[b];
        if (add > 0) tokens += add;
        if (add < 0) {
            given += min(pages(max(len, 0)), p.max_pages);
            if (cta == 0 && (len < 0 || len > room)) wrong();
        }
    }
    long long upto2[2] = {tokens, given}, all2[2];
    scan<2>(upto2, warp_sums, all2);
    const long long start = upto2[0] - tokens, all_tokens = all2[0], all_given = all2[1];
    long long give = upto2[1] - given;
    const long long count = min(count0 + all_given, (long long)p.pool);

    // What each request needs.
    long long need = 0, at = start;
    for (int b = b0; b < b1; ++b) {
        const int len = p.lens[b], add = p.new_tokens[b];
        // Kept for the next loop: whether it fits, its pages and how many it needs.
        const bool fit = fits(b, len, add, at);
        const int held = min(pages(max(len, 0)), p.max_pages), more = fit ? pages(len + add) - held : 0;
        req[b].len = fit ? len : add < 0 ? kEnded : kRefusedRoom;
        req[b].held = held;
        first_page[b] = more;
        starts[b] = (int)min(first_slot(b, at), (long long)p.n_slots);
        need += more;
        if (add > 0) at += add;
    }
    long long upto1[1] = {need}, all1[1];
    scan<1>(upto1, warp_sums + 2, all1);
    long long upto = upto1[0] - need, last = 0;
    for (int b = b0; b < b1; ++b) {
        const int n = first_page[b];
        const bool there = n == 0 || upto + n <= count;
        if (n > 0 && there) last = upto + n;
        first_page[b] = (int)min(upto, (long long)INT_MAX);
        first_given[b] = (int)min(give, (long long)p.pool);
        if (req[b].len >= 0 && !there) req[b].len = kRefusedPages;
        if (req[b].len == kEnded) give += req[b].held;
        upto += n;
    }
    // Pages handed out in all: what all need, if that is there.
    if (all1[0] <= count) {
        if (tid == 0) taken = all1[0];
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
        if ((tid & 31) == 0 && last) atomicMax(&taken, last);
    }
    __syncthreads();

    // Goes through `total` things (tokens, pages) that belong to the requests as `first` says: asks for a value for
    // each of them, then does something with it. A warp takes consecutive groups of 32; it searches for the first
    // one's request, and from there on a group's requests are among the next 32, one to a lane. What is asked for
    // kAt groups is on its way together.
    const int lane = tid & 31, gwarp = (tid >> 5) * ctas + cta, gwarps = ctas * (threads / 32);
    auto go_through = [&](int by, const int *first, int total, auto &&ask, auto &&take) {  // by: the warp's number
        constexpr int kAt = 4;
        const int all = (int)(((long long)total + 31) / 32), groups = (all + gwarps - 1) / gwarps;
        const int g_begin = (int)min((long long)by * groups, (long long)all), g_end = min(g_begin + groups, all);
        auto search = [&](int t) {  // the last request that begins at or before t
            int lo = 0, hi = p.batch - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (first[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            return lo;
        };
        int at = g_begin > 0 && g_begin < g_end ? search(g_begin * 32) : 0;
        for (int g = g_begin; g < g_end; g += kAt) {
            int lo[kAt], got[kAt];
#pragma unroll
            for (int x = 0; x < kAt; ++x) {
                lo[x] = got[x] = 0;
                if (g + x >= g_end) continue;
                const int t = (g + x) * 32 + lane;
                const int next = at + 1 + lane < p.batch ? first[at + 1 + lane] : INT_MAX;
                int c = 0;  // how many of the 32 begin at or before t
#pragma unroll
                for (int step = 16; step; step >>= 1)
                    if (__shfl_sync(0xffffffffu, next, c + step - 1) <= t) c += step;
                if (__shfl_sync(0xffffffffu, next, c) <= t) ++c;
                lo[x] = c < 32 ? at + c : search(t);  // 32: many requests without any
                at = __shfl_sync(0xffffffffu, lo[x], 31);
                if (t < total) got[x] = ask(t, lo[x]);
            }
#pragma unroll
            for (int x = 0; x < kAt; ++x) {
                const int t = (g + x) * 32 + lane;
                if (g + x < g_end && t < total) take(t, lo[x], got[x]);
            }
        }
    };

    // Pages given back, behind those that are free.
    go_through(gwarp, first_given, (int)min(all_given, (long long)p.pool - count0),
               [&](int n, int b) { return p.table[(long long)b * p.table_stride + (n - first_given[b])]; },
               [&](int n, int, int page) {
                   p.free_pages[count0 + n] = page;
                   if (page < 0) wrong();
               });
    __syncwarp();
    ptx::cluster_sync();

    // Lengths and refusals, in place perhaps: from here on nobody reads the old ones.
    for (int b = cta * threads + (threads - 1 - tid); b < p.batch; b += ctas * threads) {
        const int len = req[b].len;
        p.lens_out[b] = len == kEnded ? 0 : len >= 0 ? len + p.new_tokens[b] : p.lens[b];
        p.refused[b] = len == kRefusedPages ? 1 : len == kRefusedRoom ? 2 : 0;
    }

    // Pages handed out: the n-th from the top of the list. Few are the last warps', few tokens the first ones'.
    const long long top = count - 1;
    go_through(gwarps - 1 - gwarp, first_page, (int)taken, [&](int n, int) { return __ldcg(p.free_pages + (top - n)); },
               [&](int n, int b, int page) {
                   p.table[(long long)b * p.table_stride + req[b].held + (n - first_page[b])] = page;
                   if (page < 0) wrong();
               });

    // Every token's place.
    auto position = [&](int t, int b) {  // -1: no slot
        const int nth = t - starts[b], len = req[b].len;
        return len >= 0 && (p.spacing ? nth < p.new_tokens[b] : t < all_tokens) ? len + nth : -1;
    };
    go_through(gwarp, starts, p.n_slots,
               [&](int t, int b) {
                   const int pos = position(t, b), j = by_page(max(pos, 0)), held = req[b].held;
                   return pos < 0    ? 0
                          : j < held ? p.table[(long long)b * p.table_stride + j]
                                     : __ldcg(p.free_pages + (top - (first_page[b] + j - held)));
               },
               [&](int t, int b, int page) {
                   const int pos = position(t, b);
                   p.slots[t] = pos < 0 || page < 0 ? -1ll : (long long)page * ps + (pos - by_page(pos) * p.page_size);
                   if (page < 0) wrong();
                   p.positions[t] = max(pos, 0);
               });

    if (cta == 0 && tid == 0) p.free_count_out[0] = (int)(count - taken);
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" w4a16_status w4a16_kv_extend(const int32_t *lens, const int32_t *new_tokens, int32_t *table,
                                        long long table_stride, int batch, int max_pages, int page_size,
                                        int32_t *free_pages, int pool, const int32_t *free_count, int32_t *lens_out,
                                        int32_t *free_count_out, int64_t *slots, int32_t *positions, int n_slots,
                                        int32_t *refused, int spacing, void *stream) {
    if (batch < 0 || spacing < 0 || max_pages <= 0 || page_size <= 0 || pool <= 0 || n_slots < 0 || table_stride < max_pages)
        return W4A16_ERR_INVALID_ARG;
    if (batch > kMaxBatch || n_slots > INT_MAX - 63) return W4A16_ERR_UNSUPPORTED;
    if (batch == 0) return W4A16_OK;
    if (!lens || !new_tokens || !table || !free_pages || !free_count || !lens_out || !free_count_out || !refused ||
        (n_slots && (!slots || !positions)))
        return W4A16_ERR_INVALID_ARG;
    for (const void *q : {(const void *)lens, (const void *)new_tokens, (const void *)table, (const void *)free_pages,
                          (const void *)free_count, (const void *)lens_out, (const void *)free_count_out,
                          (const void *)positions, (const void *)refused})
        if (!aligned(q, 4)) return W4A16_ERR_INVALID_ARG;
    if (!aligned(slots, 8)) return W4A16_ERR_INVALID_ARG;
    // Division by page_size as a product: with 2^l the first power of two not below it, 2^(31 + l) / page_size rounded
    // up is below 2^32, and what the rounding adds stays below one for every n below 2^31.
    unsigned int l = 0;
    while ((1ull << l) < (unsigned int)page_size) ++l;
    const unsigned long long whole = ((1ull << (31 + l)) + page_size - 1) / page_size;
    const unsigned int magic = (unsigned int)whole, shift = 31 + l;
    const ExtendParams p{lens,      new_tokens, free_count, table,        free_pages, lens_out,  free_count_out,
                         positions, refused,    slots,      table_stride, batch,      max_pages, page_size,
                         pool,      n_slots,    magic,        shift,      spacing,   device_error_ptr(), launch_overlap()};
    if (!p.err) return W4A16_ERR_CUDA;
    cudaError_t e = ensure_max_dyn_smem((const void *)kv_extend_kernel, kMaxBatch * kRequestBytes);
    if (e != cudaSuccess) return from_cuda(e);
    // A step of running requests fits one CTA, and a small one is done sooner with fewer warps to wait for.
    const int ctas = batch <= 1024 && n_slots <= 4096 ? 1 : 8;
    const int threads = batch <= 128 && n_slots <= 1024 ? 256 : batch <= 512 && n_slots <= 4096 ? 512 : kMostThreads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)batch * kRequestBytes;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = as_dependent(cfg.stream) ? 2 : 1;
    return from_cuda(cudaLaunchKernelEx(&cfg, kv_extend_kernel, p));
}

extern "C" w4a16_status w4a16_kv_extend_block(const w4a16_kv_extend_args *args) {
    if (!args) return W4A16_ERR_INVALID_ARG;
    const w4a16_kv_extend_args &a = *args;
    return w4a16_kv_extend(a.lens, a.new_tokens, a.table, a.table_stride, a.batch, a.max_pages, a.page_size, a.free_pages,
                           a.pool, a.free_count, a.lens_out, a.free_count_out, a.slots, a.positions, a.n_slots,
                           a.refused, a.spacing, a.stream);
}
