// Entry point of paged attention: argument checks and the workspace's layout. The
// kernel is in paged_attention.cuh.
#include <climits>

#include "paged_attention.cuh"

using namespace w4a16;

namespace {

// Workspace: the counters, then two partial results for each CTA, of the size of the
// largest, so that one workspace serves calls of every shape.
constexpr size_t kCounterBytes = 3 * attn::kMaxCtas * 4;

}  // namespace

// Of a call without requests only the host's values are looked at.
w4a16_status w4a16::attn::fill(Params &p, const void *q, w4a16_type type, long long q_row, long long q_head,
                               const w4a16_kv_cache *cache, const int32_t *table, long long table_stride, int max_pages,
                               const int32_t *lens, int batch, int heads, float scale, int window, float softcap, void *out,
                               long long o_row, long long o_head, float *lse, void *ws, size_t ws_bytes) {
    w4a16_status st = check_cache(cache);
    if (st != W4A16_OK) return st;
    if (type != W4A16_TYPE_F16 && type != W4A16_TYPE_BF16) return W4A16_ERR_INVALID_ARG;
    if (cache->type != type && cache->type != W4A16_TYPE_E4M3) return W4A16_ERR_UNSUPPORTED;
    if (batch < 0 || heads <= 0 || heads % cache->kv_heads || max_pages <= 0 || table_stride < max_pages || window < 0)
        return W4A16_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f) return W4A16_ERR_INVALID_ARG;
    if ((long long)batch * heads > (1 << 24)) return W4A16_ERR_UNSUPPORTED;
    // Tiles (of 32 tokens at least, 8 heads at least) are numbered in 31 bits.
    const long long room = (long long)max_pages * cache->page_size, most = room < INT_MAX ? room : INT_MAX;
    if ((most + 31) / 32 * batch * ((heads / cache->kv_heads + 7) / 8 * cache->kv_heads) > INT_MAX)
        return W4A16_ERR_UNSUPPORTED;
    if (batch == 0) return W4A16_OK;
    if (!q || !out || !table || !lens) return W4A16_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(lse, 4))
        return W4A16_ERR_INVALID_ARG;
    for (long long s : {q_row, q_head, o_row, o_head})
        if (s < 0 || s % 8) return W4A16_ERR_INVALID_ARG;
    if (!ws || !aligned(ws, 256) ||
        ws_bytes < w4a16_paged_attention_workspace_bytes(batch, heads, cache->kv_heads, cache->head_dim))
        return W4A16_ERR_WORKSPACE;
    p.q = q, p.out = out;
    p.q_row = q_row, p.q_head = q_head, p.o_row = o_row, p.o_head = o_head, p.table_stride = table_stride;
    p.c = *cache;
    p.table = table, p.lens = lens, p.lse = lse;
    p.counters = static_cast<unsigned int *>(ws);
    p.partial = reinterpret_cast<float *>(static_cast<unsigned char *>(ws) + kCounterBytes);
    p.max_pages = max_pages, p.batch = batch, p.heads = heads, p.group = heads / cache->kv_heads;
    p.one_page = cache->page_size % 16 == 0;
    p.window = window, p.scale = scale, p.softcap = softcap;
    p.err = device_error_ptr();
    if (!p.err) return W4A16_ERR_CUDA;
    return W4A16_OK;
}

extern "C" {

size_t w4a16_paged_attention_workspace_bytes(int batch, int heads, int kv_heads, int head_dim) {
    if (batch <= 0 || heads <= 0 || kv_heads <= 0 || head_dim <= 0 || heads % kv_heads) return 0;
    return kCounterBytes + (size_t)sm_count() * attn::kMostPerSm * 2 * attn::kMaxPartial * 4;
}

w4a16_status w4a16_paged_attention(const void *q, w4a16_type type, long long q_row, long long q_head,
                                   const w4a16_kv_cache *cache, const int32_t *table, long long table_stride,
                                   int max_pages, const int32_t *lens, int batch, int heads, float scale, int window,
                                   float softcap, void *out, long long o_row, long long o_head, float *lse, void *ws,
                                   size_t ws_bytes, void *stream) {
    attn::Params p{};
    const w4a16_status st = attn::fill(p, q, type, q_row, q_head, cache, table, table_stride, max_pages, lens, batch, heads,
                                       scale, window, softcap, out, o_row, o_head, lse, ws, ws_bytes);
    if (st != W4A16_OK || batch == 0) return st;
    cudaStream_t s = (cudaStream_t)stream;
    return from_cuda(type == W4A16_TYPE_F16 ? attn::launch_f16(p, sm_count(), s) : attn::launch_bf16(p, sm_count(), s));
}

w4a16_status w4a16_paged_attention_block(const w4a16_paged_attention_args *args) {
    if (!args) return W4A16_ERR_INVALID_ARG;
    const w4a16_paged_attention_args &a = *args;
    return w4a16_paged_attention(a.q, (w4a16_type)a.type, a.q_row, a.q_head, a.cache, a.table, a.table_stride,
                                 a.max_pages, a.lens, a.batch, a.heads, a.scale, a.window, a.softcap, a.out, a.o_row,
                                 a.o_head, a.lse, a.ws, a.ws_bytes, a.stream);
}

}  // extern "C"
