// Entry points of the attention of many rows: prompts, and shared prefixes. Argument
// checks and the workspaces' layouts; the kernels are in wide_attention.cuh.
#include <climits>

#include "paged_attention.cuh"
#include "wide_attention.cuh"

using namespace w4a16;

namespace {

size_t up(size_t x) { return (x + 255) / 256 * 256; }

int ctas() { return sm_count() < wide::kMaxCtas ? sm_count() : wide::kMaxCtas; }

// Floats of a row's sums.
size_t pitch(int head_dim) { return (size_t)wide::dim_of(head_dim) + 8; }

// What both calls need: the CTAs' parts of cut tiles, their flags and descriptions.
struct Layout {
    size_t cuts, odd, slots, end;
    Layout(size_t at, int head_dim) {
        cuts = at;
        odd = cuts + up(sizeof(wide::Cut) * wide::kMaxCtas);
        slots = odd + up(sizeof(int) * wide::kMaxCtas);
        end = slots + up((size_t)2 * ctas() * wide::rows_of(head_dim) * pitch(head_dim) * 4);
    }
};
// Of prefixes besides: the workspace of the requests' own attention in front (it has to be zero at first), the
// requests' places, whole tiles' sums, the requests' own sums.
struct PrefixLayout {
    size_t own, found, whole, raw, raw_lse, end;
    PrefixLayout(int batch, int heads, int kv_heads, int head_dim)
        : own(up(w4a16_paged_attention_workspace_bytes(batch, heads, kv_heads, head_dim))) {
        const Layout l(own, head_dim);
        const size_t rows = (size_t)batch * heads;
        found = l.end;
        whole = found + up((size_t)heads * batch * sizeof(wide::Found));
        raw = whole + up(rows * pitch(head_dim) * 4);
        raw_lse = raw + up(rows * head_dim * 4);
        end = raw_lse + up(rows * 4);
    }
};

bool sizes_ok(int rows, int heads, int kv_heads, int head_dim) {
    return rows > 0 && heads > 0 && kv_heads > 0 && head_dim > 0 && head_dim <= 256 && heads % kv_heads == 0 &&
           (long long)rows * heads <= (1 << 24);
}

// What both calls check alike. *nothing: there is no row.
w4a16_status check(const void *q, w4a16_type type, long long q_row, long long q_head, const w4a16_kv_cache *cache,
                   const int32_t *table, long long table_stride, int max_pages, const int32_t *lens, int rows, int batch,
                   int heads, const int32_t *ptable, long long ptable_stride, int pmax_pages, const int32_t *plens,
                   const int32_t *pof, int prefixes, float scale, int window, float softcap, const void *out, long long o_row,
                   long long o_head, const float *lse, bool prefixes_only, bool *nothing) {
    const w4a16_status st = check_cache(cache);
    if (st != W4A16_OK) return st;
    if (type != W4A16_TYPE_F16 && type != W4A16_TYPE_BF16) return W4A16_ERR_INVALID_ARG;
    if (cache->type != type && cache->type != W4A16_TYPE_E4M3) return W4A16_ERR_UNSUPPORTED;
    if (rows < 0 || batch < 0 || heads <= 0 || heads % cache->kv_heads || max_pages <= 0 || table_stride < max_pages || window < 0)
        return W4A16_ERR_INVALID_ARG;
    if (prefixes < 0 || (prefixes > 0 && (pmax_pages <= 0 || ptable_stride < pmax_pages))) return W4A16_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !std::isfinite(softcap) || softcap < 0.f) return W4A16_ERR_INVALID_ARG;
    if ((long long)rows * heads > (1 << 24) || batch > wide::kMaxSeqs || prefixes > wide::kMaxPrefixes) return W4A16_ERR_UNSUPPORTED;
    // Keys of a sequence are numbered in 31 bits.
    const long long keys = ((long long)max_pages + (prefixes > 0 ? pmax_pages : 0)) * cache->page_size;
    if (keys > INT_MAX - 1024) return W4A16_ERR_UNSUPPORTED;
    // Units of work are numbered in 31 bits: tiles of rows, at most one a sequence besides the full ones, times keys.
    const int group = heads / cache->kv_heads, most = wide::rows_of(cache->head_dim), block = group < most ? group : most;
    const long long seqs = prefixes_only ? prefixes : batch;
    const long long tiles = rows / (most / block) + seqs, hds = (long long)(group + block - 1) / block * cache->kv_heads;
    if (tiles * hds > INT_MAX / (keys / wide::keys_of(cache->head_dim) + 3 + wide::kOver)) return W4A16_ERR_UNSUPPORTED;
    *nothing = rows == 0 || batch == 0;
    if (*nothing) return W4A16_OK;
    if (!q || !out || !table || !lens || (prefixes > 0 && (!ptable || !plens || !pof))) return W4A16_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(out, 16)) return W4A16_ERR_INVALID_ARG;
    for (const void *x : {(const void *)table, (const void *)lens, (const void *)ptable, (const void *)plens, (const void *)pof,
                          (const void *)lse})
        if (!aligned(x, 4)) return W4A16_ERR_INVALID_ARG;
    for (long long s : {q_row, q_head, o_row, o_head})
        if (s < 0 || s % 8) return W4A16_ERR_INVALID_ARG;
    return W4A16_OK;
}

// Tensor maps, where rows and pages allow them: without one the kernels copy 16 bytes at a time.
void maps(wide::Params &p) {
    const w4a16_kv_cache &c = p.c;
    const int most = wide::rows_of(c.head_dim), gb = p.group < most ? p.group : most;
    p.q_tma = p.starts && p.scale != 0.f && c.type != W4A16_TYPE_E4M3 &&
              tmap_boxes(&p.q_map, p.q, {c.head_dim, p.heads, p.rows, 1}, {p.q_head, p.q_row, 0}, {64, gb, most / gb, 1});
    // Boxes of whole groups of 8 keys (the swizzle's rows), at most those that one warp brings.
    int rows = wide::keys_of(c.head_dim) / 4;
    while (rows >= 8 && c.page_size % rows) rows /= 2;
    p.kv_rows = 0;
    if (rows >= 8 && c.type != W4A16_TYPE_E4M3 &&
        tmap_boxes(&p.k_map, c.k, {c.head_dim, c.page_size, c.kv_heads, c.pages}, {c.k_token, c.k_head, c.k_page}, {64, rows, 1, 1}) &&
        tmap_boxes(&p.v_map, c.v, {c.head_dim, c.page_size, c.kv_heads, c.pages}, {c.v_token, c.v_head, c.v_page}, {64, rows, 1, 1}))
        p.kv_rows = rows;
}

}  // namespace

extern "C" {

size_t w4a16_prompt_attention_workspace_bytes(int rows, int heads, int kv_heads, int head_dim) {
    return sizes_ok(rows, heads, kv_heads, head_dim) ? Layout(0, head_dim).end : 0;
}

w4a16_status w4a16_prompt_attention(const void *q, w4a16_type type, long long q_row, long long q_head,
                                    const w4a16_kv_cache *cache, const int32_t *table, long long table_stride, int max_pages,
                                    const int32_t *starts, const int32_t *lens, int rows, int batch, int heads,
                                    const int32_t *prefix_table, long long prefix_stride, int prefix_pages,
                                    const int32_t *prefix_lens, const int32_t *prefix_of, int prefixes, float scale, int window,
                                    float softcap, void *out, long long o_row, long long o_head, float *lse, void *ws,
                                    size_t ws_bytes, void *stream) {
    bool nothing = false;
    const w4a16_status st = check(q, type, q_row, q_head, cache, table, table_stride, max_pages, lens, rows, batch, heads,
                                  prefix_table, prefix_stride, prefix_pages, prefix_lens, prefix_of, prefixes, scale, window,
                                  softcap, out, o_row, o_head, lse, false, &nothing);
    if (st != W4A16_OK || nothing) return st;
    if (!starts || !aligned(starts, 4) || q == out) return W4A16_ERR_INVALID_ARG;
    const Layout l(0, cache->head_dim);
    if (!ws || !aligned(ws, 256) || ws_bytes < l.end) return W4A16_ERR_WORKSPACE;
    unsigned char *at = static_cast<unsigned char *>(ws);
    wide::Params p{};
    p.q = q, p.out = out, p.q_row = q_row, p.q_head = q_head, p.o_row = o_row, p.o_head = o_head;
    p.c = *cache;
    p.table = table, p.table_stride = table_stride, p.max_pages = max_pages, p.lens = lens, p.starts = starts;
    if (prefixes > 0)
        p.ptable = prefix_table, p.ptable_stride = prefix_stride, p.pmax_pages = prefix_pages, p.plens = prefix_lens,
        p.pof = prefix_of, p.prefixes = prefixes;
    p.rows = rows, p.batch = batch, p.heads = heads, p.group = heads / cache->kv_heads, p.window = window;
    p.scale = scale, p.softcap = softcap, p.lse = lse;
    p.cuts = reinterpret_cast<wide::Cut *>(at + l.cuts);
    p.odd = reinterpret_cast<int *>(at + l.odd);
    p.slots = reinterpret_cast<float *>(at + l.slots);
    p.wide_out = aligned(out, 32) && o_row % 16 == 0 && o_head % 16 == 0;
    p.ctas = ctas(), p.err = device_error_ptr(), p.wait_ns = wait_limit_ns();
    if (!p.err) return W4A16_ERR_CUDA;
    maps(p);
    cudaStream_t s = (cudaStream_t)stream;
    const auto launch = type == W4A16_TYPE_F16 ? wide::launch_f16 : wide::launch_bf16;
    const cudaError_t e = launch(wide::kWide, p, s);
    return from_cuda(e != cudaSuccess ? e : launch(wide::kFinish, p, s));
}

size_t w4a16_prefix_attention_workspace_bytes(int batch, int heads, int kv_heads, int head_dim) {
    return sizes_ok(batch, heads, kv_heads, head_dim) ? PrefixLayout(batch, heads, kv_heads, head_dim).end : 0;
}

w4a16_status w4a16_prefix_attention(const void *q, w4a16_type type, long long q_row, long long q_head,
                                    const w4a16_kv_cache *cache, const int32_t *table, long long table_stride, int max_pages,
                                    const int32_t *lens, int batch, int heads, const int32_t *prefix_table,
                                    long long prefix_stride, int prefix_pages, const int32_t *prefix_lens,
                                    const int32_t *prefix_of, int prefixes, float scale, int window, float softcap, void *out,
                                    long long o_row, long long o_head, float *lse, void *ws, size_t ws_bytes, void *stream) {
    bool nothing = false;
    w4a16_status st = check(q, type, q_row, q_head, cache, table, table_stride, max_pages, lens, batch, batch, heads,
                            prefix_table, prefix_stride, prefix_pages, prefix_lens, prefix_of, prefixes, scale, window, softcap,
                            out, o_row, o_head, lse, true, &nothing);
    if (st != W4A16_OK) return st;
    if (prefixes == 0) return W4A16_ERR_INVALID_ARG;
    if (nothing) return W4A16_OK;
    if (q == out) return W4A16_ERR_INVALID_ARG;
    const PrefixLayout l(batch, heads, cache->kv_heads, cache->head_dim);
    if (!ws || !aligned(ws, 256) || ws_bytes < l.end) return W4A16_ERR_WORKSPACE;
    unsigned char *at = static_cast<unsigned char *>(ws);
    const Layout w(l.own, cache->head_dim);
    wide::Params p{};
    p.q = q, p.out = out, p.q_row = q_row, p.q_head = q_head, p.o_row = o_row, p.o_head = o_head;
    p.c = *cache;
    p.table = table, p.table_stride = table_stride, p.max_pages = max_pages, p.lens = lens;
    p.ptable = prefix_table, p.ptable_stride = prefix_stride, p.pmax_pages = prefix_pages, p.plens = prefix_lens;
    p.pof = prefix_of, p.prefixes = prefixes;
    p.rows = batch, p.batch = batch, p.heads = heads, p.group = heads / cache->kv_heads, p.window = window;
    p.scale = scale, p.softcap = softcap, p.lse = lse;
    p.odd = reinterpret_cast<int *>(at + w.odd);
    p.slots = reinterpret_cast<float *>(at + w.slots);
    p.found = reinterpret_cast<wide::Found *>(at + l.found);
    p.whole = reinterpret_cast<float *>(at + l.whole);
    p.raw = reinterpret_cast<float *>(at + l.raw), p.raw_lse = reinterpret_cast<float *>(at + l.raw_lse);
    p.wide_out = aligned(out, 32) && o_row % 16 == 0 && o_head % 16 == 0;
    p.ctas = ctas(), p.err = device_error_ptr(), p.wait_ns = wait_limit_ns();
    if (!p.err) return W4A16_ERR_CUDA;
    maps(p);
    // The requests' own tokens: paged attention, whose sums go into the workspace.
    attn::Params o{};
    st = attn::fill(o, q, type, q_row, q_head, cache, table, table_stride, max_pages, lens, batch, heads, scale, window, softcap,
                    out, o_row, o_head, nullptr, at, l.own);
    if (st != W4A16_OK) return st;
    o.raw = reinterpret_cast<float *>(at + l.raw), o.raw_lse = reinterpret_cast<float *>(at + l.raw_lse);
    cudaStream_t s = (cudaStream_t)stream;
    const auto launch = type == W4A16_TYPE_F16 ? wide::launch_f16 : wide::launch_bf16;
    cudaError_t e = launch(wide::kWide, p, s);
    if (e == cudaSuccess) e = type == W4A16_TYPE_F16 ? attn::launch_sums_f16(o, sm_count(), s) : attn::launch_sums_bf16(o, sm_count(), s);
    return from_cuda(e != cudaSuccess ? e : launch(wide::kPrefixJoin, p, s));
}

w4a16_status w4a16_prompt_attention_block(const w4a16_prompt_attention_args *args) {
    if (!args) return W4A16_ERR_INVALID_ARG;
    const w4a16_prompt_attention_args &a = *args;
    return w4a16_prompt_attention(a.q, (w4a16_type)a.type, a.q_row, a.q_head, a.cache, a.table, a.table_stride, a.max_pages,
                                  a.starts, a.lens, a.rows, a.batch, a.heads, a.prefix_table, a.prefix_stride, a.prefix_pages,
                                  a.prefix_lens, a.prefix_of, a.prefixes, a.scale, a.window, a.softcap, a.out, a.o_row, a.o_head,
                                  a.lse, a.ws, a.ws_bytes, a.stream);
}

w4a16_status w4a16_prefix_attention_block(const w4a16_prefix_attention_args *args) {
    if (!args) return W4A16_ERR_INVALID_ARG;
    const w4a16_prefix_attention_args &a = *args;
    return w4a16_prefix_attention(a.q, (w4a16_type)a.type, a.q_row, a.q_head, a.cache, a.table, a.table_stride, a.max_pages,
                                  a.lens, a.batch, a.heads, a.prefix_table, a.prefix_stride, a.prefix_pages, a.prefix_lens,
                                  a.prefix_of, a.prefixes, a.scale, a.window, a.softcap, a.out, a.o_row, a.o_head, a.lse, a.ws,
                                  a.ws_bytes, a.stream);
}

}  // extern "C"
