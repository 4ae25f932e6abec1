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
#include <climits>

#include "ptx.cuh"
#include "w4a16_internal.h"

namespace w4a16 {
namespace {

struct ExtendParams {
    const int32_t *lens, *new_tokens, *free_count;
    int32_t *table, *free_pages, *lens_out, *free_count_out, *positions, *refused;
    int64_t *slots;
    long long table_stride;
    int batch, max_pages, page_size, pool, n_slots;
};

constexpr int kThreads = 1024;
constexpr int kMaxBatch = 8192;

// A request's figures, kept in shared memory.
struct Request {
    int start;   // its first token in the step, at most n_slots
    int len;     // tokens before the step; negative: it gets none (kRefused..., kEnded)
    int held;    // pages before the step
    int page0;   // pages handed out before its first; ended: pages given back before its first
};
constexpr int kRefusedPages = -1, kRefusedRoom = -2, kEnded = -3;

// Inclusive prefix sum over the CTA's threads; *total is the sum of all.
__device__ __forceinline__ long long scan(long long x, long long *warp_sums, long long *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();  // the last scan's sums have been read
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        long long s = lane < kThreads / 32 ? warp_sums[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        warp_sums[lane] = s;
    }
    __syncthreads();
    *total = warp_sums[kThreads / 32 - 1];
    return x + (warp ? warp_sums[warp - 1] : 0);
}

__global__ void __launch_bounds__(kThreads) kv_extend_kernel(const ExtendParams p) {
    extern __shared__ Request req[];
    __shared__ long long warp_sums[32];
    __shared__ long long taken;
    ptx::grid_dep_launch();
    ptx::grid_dep_wait();
    const int ctas = gridDim.x, cta = blockIdx.x, tid = threadIdx.x;
    const int per = (p.batch + kThreads - 1) / kThreads;  // consecutive requests of a thread
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    const long long ps = p.page_size, room = min((long long)p.max_pages * ps, (long long)INT_MAX);
    const long long count0 = min(max(p.free_count[0], 0), p.pool);
    auto pages = [&](long long n) { return (n + ps - 1) / ps; };

    // Tokens and pages given back, in front of each request.
    long long tokens = 0, given = 0;
    for (int b = b0; b < b1; ++b) {
        const int len = p.lens[b], add = p.new_tokens[b];
        if (add > 0) tokens += add;
        if (add < 0) given += min(pages(max(len, 0)), (long long)p.max_pages);
    }
    long long all_tokens, all_given, all_need;
    long long start = scan(tokens, warp_sums, &all_tokens) - tokens;
    long long give = scan(given, warp_sums, &all_given) - given;
    const long long count = min(count0 + all_given, (long long)p.pool);

    // What each request needs.
    long long need = 0, at = start;
    for (int b = b0; b < b1; ++b) {
        const int len = p.lens[b], add = p.new_tokens[b];
        const bool fits = add >= 0 && len >= 0 && (long long)len + add <= room && (add == 0 || at + add <= p.n_slots);
        if (fits) need += pages((long long)len + add) - pages(len);
        if (add > 0) at += add;
    }
    if (tid == 0) taken = 0;
    long long upto = scan(need, warp_sums, &all_need) - need;
    at = start;
    for (int b = b0; b < b1; ++b) {
        const int len = p.lens[b], add = p.new_tokens[b];
        const bool fits = add >= 0 && len >= 0 && (long long)len + add <= room && (add == 0 || at + add <= p.n_slots);
        const long long n = fits ? pages((long long)len + add) - pages(len) : 0;
        const bool got = fits && (n == 0 || upto + n <= count);
        Request r;
        r.start = (int)min(at, (long long)p.n_slots);
        r.held = (int)min(pages(max(len, 0)), (long long)p.max_pages);
        r.len = got ? len : add < 0 ? kEnded : fits ? kRefusedPages : kRefusedRoom;
        r.page0 = (int)min(add < 0 ? give : upto, (long long)p.pool);
        req[b] = r;
        if (got && n > 0) atomicMax(&taken, upto + n);
        if (add < 0) give += r.held;
        if (add > 0) at += add;
        upto += n;
    }
    __syncthreads();

    // Pages given back: one warp per ended request.
    const int lane = tid & 31, gwarp = (tid >> 5) * ctas + cta, gwarps = ctas * (kThreads / 32);
    for (int b = gwarp; b < p.batch; b += gwarps) {
        const Request r = req[b];
        if (r.len != kEnded) continue;
        const long long to = count0 + r.page0;
        for (int j = lane; j < r.held; j += 32)
            if (to + j < p.pool) p.free_pages[to + j] = p.table[(long long)b * p.table_stride + j];
    }
    __syncwarp();
    ptx::cluster_sync();

    // Pages handed out: the n-th from the top of the list.
    const long long top = count - 1;
    for (int b = gwarp; b < p.batch; b += gwarps) {
        const Request r = req[b];
        const int add = p.new_tokens[b];
        if (lane == 0) {
            p.lens_out[b] = r.len == kEnded ? 0 : r.len >= 0 ? r.len + add : p.lens[b];
            p.refused[b] = r.len == kRefusedPages ? 1 : r.len == kRefusedRoom ? 2 : 0;
        }
        if (r.len < 0) continue;
        const int last = (int)pages((long long)r.len + add);
        for (int j = r.held + lane; j < last; j += 32)
            p.table[(long long)b * p.table_stride + j] = __ldcg(p.free_pages + (top - (r.page0 + j - r.held)));
    }
    if (cta == 0 && tid == 0) p.free_count_out[0] = (int)(count - taken);

    // Every token's place.
    for (long long t = (long long)cta * kThreads + tid; t < p.n_slots; t += (long long)ctas * kThreads) {
        long long slot = -1;
        int pos = 0;
        if (t < all_tokens) {
            int lo = 0, hi = p.batch - 1;  // the last request that starts at or before t
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (req[mid].start <= t) lo = mid;
                else hi = mid - 1;
            }
            const Request r = req[lo];
            if (r.len >= 0) {
                pos = r.len + (int)(t - r.start);
                const int j = (int)(pos / ps);
                const int page = j < r.held ? p.table[(long long)lo * p.table_stride + j]
                                            : __ldcg(p.free_pages + (top - (r.page0 + j - r.held)));
                slot = (long long)page * ps + pos % ps;
            }
        }
        p.slots[t] = slot;
        p.positions[t] = pos;
    }
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" w4a16_status w4a16_kv_extend(const int32_t *lens, const int32_t *new_tokens, int32_t *table,
                                        long long table_stride, int batch, int max_pages, int page_size,
                                        int32_t *free_pages, int pool, const int32_t *free_count, int32_t *lens_out,
                                        int32_t *free_count_out, int64_t *slots, int32_t *positions, int n_slots,
                                        int32_t *refused, void *stream) {
    if (batch < 0 || max_pages <= 0 || page_size <= 0 || pool <= 0 || n_slots < 0 || table_stride < max_pages)
        return W4A16_ERR_INVALID_ARG;
    if (batch > kMaxBatch) return W4A16_ERR_UNSUPPORTED;
    if (batch == 0) return W4A16_OK;
    if (!lens || !new_tokens || !table || !free_pages || !free_count || !lens_out || !free_count_out || !refused ||
        (n_slots && (!slots || !positions)))
        return W4A16_ERR_INVALID_ARG;
    for (const void *q : {(const void *)lens, (const void *)new_tokens, (const void *)table, (const void *)free_pages,
                          (const void *)free_count, (const void *)lens_out, (const void *)free_count_out,
                          (const void *)positions, (const void *)refused})
        if (!aligned(q, 4)) return W4A16_ERR_INVALID_ARG;
    if (!aligned(slots, 8)) return W4A16_ERR_INVALID_ARG;
    const ExtendParams p{lens,      new_tokens, free_count, table,        free_pages, lens_out,  free_count_out,
                         positions, refused,    slots,      table_stride, batch,      max_pages, page_size,
                         pool,      n_slots};
    cudaError_t e = ensure_max_dyn_smem((const void *)kv_extend_kernel, kMaxBatch * (int)sizeof(Request));
    if (e != cudaSuccess) return from_cuda(e);
    const int ctas = batch <= 1024 && n_slots <= 4096 ? 1 : 8;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = (size_t)batch * sizeof(Request);
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = launch_overlap() ? 2 : 1;
    return from_cuda(cudaLaunchKernelEx(&cfg, kv_extend_kernel, p));
}
