/*
 * w4a16.h -- C ABI of libw4a16.so: fp16-activation x int4-weight group-quantized
 * GEMM for NVIDIA GB300 (sm_103a), and the operators that stand between one such
 * GEMM and the next in a decoder layer (paged key-value cache, rotary positions,
 * attention of one new token, residual norm: second half of this file).
 *
 * Operation (github.com/justinchuby/onnx-genai pull 960, "What's landed" and
 * "Validation": fp16 x int4 MatMulNBits with per-group scales, group sizes
 * 16/32/64/128 and optional asymmetric 4-bit zero points):
 *
 *     Y[M,N] = A[M,K] . W[N,K]^T,   W[n,k] = (q[n,k] - zp[n,k/group]) * scale[n,k/group]
 *
 * Input formats (the plain reading of the "ONNX-native asymmetric-zp / nibble
 * format" named there):
 *   A       fp16 (IEEE binary16 bit patterns), row-major [M][K]
 *   q       uint8 [N][K/2]: nibble k of row n is byte k/2, low nibble for even k
 *   scales  fp16 or fp32, row-major [N][G], G = K/group
 *   zp      uint8 [N][ceil(G/2)], nibble j of row n = zero point of group j (low
 *           nibble for even j); NULL means symmetric (zero point 8)
 *   Y       fp16, row-major [M][N]; fp32 accumulation, round-to-nearest-even store
 *
 * Conventions shared by every call:
 *   - Device pointers are caller-owned device memory; host pointers are marked.
 *     The library never allocates, frees or synchronises inside a compute call;
 *     work is enqueued on `stream` (a cudaStream_t passed as void*, NULL = legacy
 *     default stream) and runs asynchronously.
 *   - Arguments are validated on the host before anything is launched; a
 *     non-OK status means nothing was enqueued. Launch failures map to
 *     W4A16_ERR_CUDA. No call throws.
 *   - Shape rules for the repacked layout and the kernels: M, N, K > 0,
 *     N % 16 == 0, K % 64 == 0, group in {16, 32, 64, 128}, K % group == 0.
 *     A, q_rep and Y must be 16-byte aligned, scales aligned to their element
 *     size. Violations return W4A16_ERR_INVALID_ARG or W4A16_ERR_UNSUPPORTED.
 *   - Results are deterministic: the same inputs and the same split factor give
 *     bit-identical Y on every run (fixed-order reductions, no atomics on data).
 */
#ifndef W4A16_H
#define W4A16_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    W4A16_OK = 0,
    W4A16_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misalignment */
    W4A16_ERR_UNSUPPORTED = 2,   /* valid but outside the supported shape rules */
    W4A16_ERR_WORKSPACE = 3,     /* workspace missing or smaller than required */
    W4A16_ERR_CUDA = 4,          /* a CUDA runtime call or launch failed */
    W4A16_ERR_TIMEOUT = 5        /* a bounded device-side wait expired */
} w4a16_status;

typedef enum { W4A16_SCALE_F16 = 0, W4A16_SCALE_F32 = 1 } w4a16_scale_dtype;

/* Which kernel family a GEMM call runs (reported by w4a16_gemm_plan). */
typedef enum {
    W4A16_PATH_SMALL_M = 0,      /* register-fed stream kernel, split-K over a cluster */
    W4A16_PATH_TCGEN05 = 1       /* TMA + tcgen05 tensor-memory kernel */
} w4a16_path;

/* Human-readable name of a status code (static storage, never NULL). */
const char *w4a16_status_string(w4a16_status s);

/* Bytes of the repacked weight buffer for an N x K int4 matrix: N*K/2. */
size_t w4a16_repacked_bytes(int N, int K);

/*
 * Repack nibble-packed int4 weights into the fragment-interleaved layout the GEMM
 * kernels read (the MatMulNBits pull request's "bijective ... reorder for
 * coalesced loads" with a device repack byte-identical to a host reference; the
 * permutation itself is this library's own):
 *   16-row sub-tile S = n/16, k-block b = k/64: piece (S, b) is 512 bytes at
 *   (S*(K/64) + b)*512, so every sub-tile is one contiguous run along K and a run
 *   of k-blocks of consecutive sub-tiles is a regular 3-D box for TMA copies;
 *   with g = n%8 and t = (k%16)/4 the 16-byte lane slot 4*g + (t + g/2)%4 of the
 *   piece at slot*16; u32 word j = (k%64)/16 at j*4; nibble p = 4*(e%2) + 2*(e/2)
 *   + h with e = k%4 and h = (n%16)/8 (byte p/2 of the word, high nibble when p
 *   is odd). Each lane slot holds one mma.sync m16n8k16 A fragment per word
 *   (rows g and g+8).
 *   q      device, uint8 [N][K/2] (input format above); not modified
 *   q_rep  device, w4a16_repacked_bytes(N, K) bytes, written; must not overlap q
 * Integer-only and bit-exact; inverse: w4a16_unpack_host.
 */
w4a16_status w4a16_repack(const uint8_t *q, uint8_t *q_rep, int N, int K, void *stream);

/*
 * Host inverse of w4a16_repack: q_rep (host, N*K/2 bytes) -> q (host, [N][K/2]).
 * Synchronous, pure host code, no CUDA calls.
 */
w4a16_status w4a16_unpack_host(const uint8_t *q_rep, uint8_t *q, int N, int K);

/*
 * Scratch bytes a w4a16_gemm call needs (0: split-K partials are reduced through
 * distributed shared memory inside a thread-block cluster, not global memory).
 * split_k: 0 = automatic, 1..8 = forced factor (small-M path).
 */
size_t w4a16_gemm_workspace_bytes(int M, int N, int K, int group, int split_k);

/*
 * Which path and split factor w4a16_gemm would use. split_k as in w4a16_gemm.
 * path / split_out are host pointers (either may be NULL).
 * Path choice: M above the small-M limit (w4a16_set_tuning, default 64) takes
 * the tensor-core path; so does M >= 33 (plain and fused SwiGLU) when that path's
 * grid (N/128 tiles, or N/64 for SwiGLU, times the token tiles) covers at least
 * two thirds of the SMs, unless split_k > 0 forces the small-M path's K split.
 * (This function reports the plain GEMM's choice.)
 */
w4a16_status w4a16_gemm_plan(int M, int N, int K, int group, int split_k,
                             int *path, int *split_out);

/*
 * Launch shape of the kernel a call would run: w4a16_gemm (swiglu_fused = 0) or
 * fused w4a16_gemm_swiglu (swiglu_fused = 1). For reports and tests; nothing is
 * launched. `info` is a host pointer. Errors as w4a16_gemm_plan.
 */
typedef struct {
    int path;          /* w4a16_path */
    int split;         /* CTAs along K per weight set (1 on the tensor-core path) */
    int ctas;          /* CTAs of the launch */
    int threads;       /* threads per CTA */
    int smem_bytes;    /* dynamic shared memory per CTA */
    int stages;        /* shared-memory ring stages of the weight stream */
} w4a16_launch_info;
w4a16_status w4a16_gemm_launch_info(int M, int N, int K, int group, int split_k, int swiglu_fused,
                                    w4a16_launch_info *info);

/*
 * Y = A . dequant(q_rep)^T  (see the operation at the top of this file).
 *   A        device fp16 [M][K], 16-byte aligned
 *   q_rep    device, repacked weights from w4a16_repack (N x K)
 *   scales   device [N][K/group], dtype sdt
 *   zp       device uint8 [N][ceil(G/2)] packed zero points, or NULL (zero point 8)
 *   Y        device fp16 [M][N], written (no read-modify-write)
 *   split_k  0 = automatic; 1..8 forces the small-M path's K split (a cluster
 *            of that many CTAs along K per run of sub-tiles) for M up to the
 *            small-M limit; ignored on the tensor-core path
 *   ws, ws_bytes  caller scratch of at least w4a16_gemm_workspace_bytes(); may be
 *            NULL when that is 0
 * Small M (see w4a16_gemm_plan for the choice) runs the stream kernel: weight
 * and activation boxes streamed by TMA through a shared-memory ring, each CTA a
 * run of 16-row sub-tiles over a K range, dequantisation in registers,
 * mma.sync m16n8k16 with fp32 accumulation and the group scale applied after
 * each group's partial sum (the pull request's "per-group scale AFTER the
 * tensor-core accumulate"); when the row split alone cannot fill the GPU, K is
 * split across a cluster and reduced in a fixed order.
 * Larger M runs the tcgen05 kernel: TMA-staged activations, int4 tiles dequantised to fp16
 * ((q - zp) * scale rounded once; fp32 scales are rounded to fp16 first) into
 * tensor memory, fp32 accumulation in tensor memory.
 */
w4a16_status w4a16_gemm(const uint16_t *A, const uint8_t *q_rep, const void *scales,
                        w4a16_scale_dtype sdt, const uint8_t *zp, uint16_t *Y,
                        int M, int N, int K, int group, int split_k,
                        void *ws, size_t ws_bytes, void *stream);

/*
 * w4a16_gemm for a caller whose activations arrive and whose outputs leave in
 * host memory (the same operation, defined at the top of this file): enqueues on
 * `stream` the copy of A_host into A_dev, the GEMM into Y_dev and the copy of
 * Y_dev into Y_host, one cudaMemcpyAsync per copy, and returns without
 * synchronising; Y_host holds the result once the stream has passed the call.
 *   A_host   host fp16 [M][K], page-locked (cudaHostAlloc, cudaHostRegister or
 *            torch pin_memory); not checked: with pageable memory the CUDA
 *            runtime performs the copies synchronously
 *   A_dev    device fp16 [M][K], 16-byte aligned, overwritten with A_host
 *   Y_dev    device fp16 [M][N], 16-byte aligned, overwritten with Y
 *   Y_host   host fp16 [M][N], page-locked as A_host, overwritten with Y
 *   q_rep, scales, sdt, zp, group, split_k as in w4a16_gemm (no workspace)
 * Every argument is validated before anything is enqueued, with the errors of
 * w4a16_gemm; a CUDA failure after the first copy was enqueued returns
 * W4A16_ERR_CUDA and may leave that copy enqueued.
 */
w4a16_status w4a16_gemm_host_io(const uint16_t *A_host, uint16_t *A_dev, const uint8_t *q_rep,
                                const void *scales, w4a16_scale_dtype sdt, const uint8_t *zp,
                                uint16_t *Y_dev, uint16_t *Y_host, int M, int N, int K, int group,
                                int split_k, void *stream);

/*
 * Scratch bytes for w4a16_gemm_swiglu: 0 when fused; 4*M*N (+alignment) when
 * unfused (the fp16 gate and up projections are materialised).
 */
size_t w4a16_swiglu_workspace_bytes(int M, int N, int K, int group, int fused);

/*
 * Y = silu(A . Wg^T) * (A . Wu^T), silu(x) = x / (1 + exp(-x)) (the pull
 * request's gate_up SwiGLU MLP fusion: paired gate/up int4 GEMMs followed by a
 * SiluMul epilogue). Gate and up share A, K, N, group and the scale dtype.
 *   fused = 1  one pass: both accumulators kept in fp32, silu*mul in the
 *              epilogue, only Y is written
 *   fused = 0  the unfused chain: gate -> fp16 G, up -> fp16 U (both in ws),
 *              then an elementwise silu_mul(G, U) -> Y
 * The two modes come from one source with this switch, for fusion benchmarks.
 */
w4a16_status w4a16_gemm_swiglu(const uint16_t *A,
                               const uint8_t *qg_rep, const void *sg, const uint8_t *zg,
                               const uint8_t *qu_rep, const void *su, const uint8_t *zu,
                               w4a16_scale_dtype sdt, uint16_t *Y,
                               int M, int N, int K, int group, int fused,
                               void *ws, size_t ws_bytes, void *stream);

/*
 * RMS-norm prologue (the pull request's "Update -- fused RMS-norm epilogue + e2e
 * PASS" and "Update -- P1 COMPLETE": the normalised activation is staged in
 * scratch, then the GEMM runs on it; gate_up SwiGLU has the same optional
 * prologue). The pages give no formula; the reading taken is the ONNX
 * SimplifiedLayerNormalization that the prologue replaces:
 *     An[m,k] = A[m,k] / sqrt(mean_k A[m,k]^2 + eps) * gamma[k]
 * computed in fp32 per row (fixed-order sum of squares) and stored as fp16 in
 * the caller's workspace; the GEMM (or SwiGLU) then runs on An exactly as
 * w4a16_gemm (w4a16_gemm_swiglu) would. With launch overlap on, the GEMM is a
 * programmatic dependent of the prologue and streams weights while it runs.
 *   gamma    device fp16 [K], 16-byte aligned
 *   eps      >= 0 (finite)
 *   ws       device scratch of w4a16_rmsnorm_workspace_bytes(M, N, K, group,
 *            mode) bytes, 256-byte aligned; mode 0 = w4a16_gemm_rmsnorm,
 *            1 = fused SwiGLU, 2 = unfused SwiGLU (An followed by the unfused
 *            chain's intermediates). Too small -> W4A16_ERR_WORKSPACE.
 * Other arguments, layouts and errors as w4a16_gemm / w4a16_gemm_swiglu.
 */
size_t w4a16_rmsnorm_workspace_bytes(int M, int N, int K, int group, int mode);
w4a16_status w4a16_gemm_rmsnorm(const uint16_t *A, const uint16_t *gamma, float eps, const uint8_t *q_rep,
                                const void *scales, w4a16_scale_dtype sdt, const uint8_t *zp, uint16_t *Y,
                                int M, int N, int K, int group, int split_k, void *ws, size_t ws_bytes,
                                void *stream);
w4a16_status w4a16_gemm_swiglu_rmsnorm(const uint16_t *A, const uint16_t *gamma, float eps,
                                       const uint8_t *qg_rep, const void *sg, const uint8_t *zg,
                                       const uint8_t *qu_rep, const void *su, const uint8_t *zu,
                                       w4a16_scale_dtype sdt, uint16_t *Y, int M, int N, int K, int group,
                                       int fused, void *ws, size_t ws_bytes, void *stream);

/*
 * Unfused SwiGLU (as w4a16_gemm_swiglu with fused = 0) for callers that cannot
 * allocate device memory -- code inside another framework's memory pool, hot
 * paths where an allocation that may synchronise the device is not allowed, or
 * plug-ins that are handed only input and output buffers. No counterpart in the
 * MatMulNBits pull request; this is a library convenience.
 *   The fp16 gate and up intermediates (4*M*N bytes) live in a fixed array
 *   compiled into the library, w4a16_swiglu_static_scratch_bytes() = 8 MiB,
 *   one per GPU that loads the library, kept until the process exits. Shapes
 *   whose 4*M*N exceeds it return W4A16_ERR_WORKSPACE and launch nothing.
 *   The call allocates and frees nothing. Its first call on a device looks up the
 *   array's device address (a runtime query, no allocation); make that first
 *   call before any stream capture on that device.
 *   Every call on a device shares the array, which keeps the last call's
 *   intermediates: calls that can overlap on the GPU (different streams without
 *   ordering between them) race and must not be issued that way. Nothing in the
 *   array needs to start at zero.
 *   Arguments, layouts and errors otherwise as w4a16_gemm_swiglu.
 */
size_t w4a16_swiglu_static_scratch_bytes(void);
w4a16_status w4a16_gemm_swiglu_unfused_static(const uint16_t *A,
                                              const uint8_t *qg_rep, const void *sg, const uint8_t *zg,
                                              const uint8_t *qu_rep, const void *su, const uint8_t *zu,
                                              w4a16_scale_dtype sdt, uint16_t *Y,
                                              int M, int N, int K, int group, void *stream);

/*
 * Tuning knobs (process-wide, not thread-safe; for tests and benchmarks).
 *   smallm_max  largest M that may take the small-M path (0 = default 64, max 64;
 *               -1 routes every M to the tensor-core path); see w4a16_gemm_plan
 */
w4a16_status w4a16_set_tuning(int smallm_max);

/*
 * Overlap of consecutive small-M GEMM calls (process-wide, not thread-safe;
 * default 0 = off). With enable = 1 each small-M launch is a programmatic
 * dependent of the work before it on the stream: its CTAs may start while that
 * work finishes, stage scales and zero points and start streaming q_rep, and
 * wait for it to complete before they read A or write Y. So A and Y may be the
 * previous call's output or input, as in a chain of layers, but q_rep, scales
 * and zp must not be written by the work that directly precedes the call on
 * the stream (weights loaded once and reused satisfy this; a w4a16_repack
 * followed at once by a GEMM on the same weights does not). Results are
 * identical with the switch on or off. The pages describe no such launch mode;
 * it is a GB300 launch-latency measure.
 * Returns W4A16_ERR_INVALID_ARG unless enable is 0 or 1.
 */
w4a16_status w4a16_set_launch_overlap(int enable);

/*
 * Limit of every bounded device-side wait (process-wide, not thread-safe; for
 * tests of the failure path). Each wait for an mbarrier phase (a copy landing,
 * a pipeline slot freeing up, the accumulator completing) gives up once it has
 * waited limit_ns or longer: the kernel then records W4A16_ERR_TIMEOUT in the
 * device error word (see w4a16_device_error), stops issuing work, waits for the
 * copies and tensor-core operations it already issued (with a fixed limit of
 * 0.2 s), releases its tensor memory and returns; its output is undefined.
 * Default 2000000000 (2 s). 0 gives up at the first poll that finds a phase
 * incomplete, which makes any call whose copies are still in flight fail; this
 * exists so that tests can run the expiry path without a stuck barrier.
 * Always returns W4A16_OK.
 */
w4a16_status w4a16_set_wait_limit_ns(unsigned long long limit_ns);

/*
 * Read and clear the device-side error word that bounded waits set when they
 * expire (W4A16_ERR_TIMEOUT), and the operators between the projections when a
 * value on the GPU is out of range (W4A16_ERR_INVALID_ARG), on the device current
 * for the calling thread.
 * Synchronises `stream`. Returns W4A16_OK when no kernel reported an error.
 */
w4a16_status w4a16_device_error(void *stream);

/* ------------------------------------------------------------------------
 * Operators between the int4 projections of a decoder layer.
 *
 * The conventions above hold (host validation first, no allocation, no
 * synchronisation, everything enqueued on `stream`), with these of their own:
 *   - Zero rows (rows, batch or M = 0) is a valid call that enqueues nothing.
 *   - Strides are counted in elements of the tensor and may be larger than the
 *     row they step over; the innermost dimension is contiguous. Offsets are
 *     computed in 64 bits.
 *   - Values that only the GPU sees (lengths, page numbers, slots) are checked
 *     by the kernels: one that is out of range is never used as an address, is
 *     treated as the call's comment says, and leaves W4A16_ERR_INVALID_ARG in
 *     the device error word (w4a16_device_error), unless that comment gives it
 *     a status of its own.
 *   - The calls may be launched as programmatic dependents of the work before
 *     them on the stream; they touch no memory before that work has completed, so
 *     they have no rule to keep. With w4a16_set_launch_overlap(1) captured calls
 *     are too, and all but paged_attention let the work behind them begin early.
 *   - Sums, softmax statistics and norms are held in fp32; every output element
 *     is rounded once, to nearest even. Softmax weights are matrix operands of 16
 *     bits: w4a16_paged_attention says what that leaves of them.
 * ------------------------------------------------------------------------ */
typedef enum {
    W4A16_TYPE_F16 = 0,
    W4A16_TYPE_BF16 = 1,
    W4A16_TYPE_E4M3 = 2,         /* 8-bit float, 4 exponent bits, largest 448 (cache only) */
    W4A16_TYPE_F32 = 3           /* residual stream only */
} w4a16_type;

/*
 * A paged key-value cache. Keys and values are two pools of `pages` pages of
 * `page_size` tokens of kv_heads x head_dim elements; element d of head h of
 * token t of page p is at p*page + t*token + h*head + d of its pool, so pages
 * laid out tokens first, heads first, or both pools in one allocation are all
 * described by the strides. Slot s is token s % page_size of page s / page_size.
 * Heads whose rows are no multiple of 128 bytes are read faster from pages laid out
 * heads first.
 *   type      F16, BF16 or E4M3. E4M3 stores e4m3(x / scale[h]), the quotient in
 *             fp32 first, and stands for that times scale[h], with one positive fp32
 *             scale for each kv head. Beyond 448 it saturates
 *   k_scale, v_scale  device fp32 [kv_heads], E4M3 only; NULL means 1
 * Rules: pages, page_size, kv_heads > 0; head_dim a multiple of 8 (E4M3: 16), at
 * most 256; pools 16-byte aligned; strides multiples of 16 bytes, below 2^31 elements.
 */
typedef struct {
    void *k, *v;
    const float *k_scale, *v_scale;
    long long k_page, k_token, k_head;
    long long v_page, v_token, v_head;
    int type;
    int pages, page_size, kv_heads, head_dim;
} w4a16_kv_cache;

/*
 * Places for a step's new tokens, from the requests' lengths: one call takes
 * pages from a free list, grows the block table and names every token's slot.
 *   lens        device [batch]: tokens that each request holds now
 *   new_tokens  device [batch]: tokens that it gets in this step (0: none);
 *               negative: the request has ended and gives its pages back
 *   table       device [batch][max_pages] (rows table_stride apart): entry j of
 *               request b is the page of its tokens j*page_size...; read and written
 *   free_pages  device [pool]: the free list, a stack of page numbers, of which
 *   free_count  device [1]: the first free_count are free
 * In this order:
 *   1. ended requests' pages go onto the stack, in the order of (request, j);
 *   2. the requests are served in their order: one that needs pages gets them
 *      from the top of the stack if the needs of all requests up to it, itself
 *      included, can be met; otherwise it is refused (refused[b] = 1). One whose
 *      tokens do not fit its table row or the slots buffer, or whose length is
 *      negative, is refused too (refused[b] = 2) and counts as needing none.
 *      The n-th page handed out is the n-th from the top.
 * Outputs:
 *   lens_out    [batch]: the new lengths (0 for ended, unchanged for refused)
 *   free_count_out [1]
 *   refused     [batch]: 0, 1 or 2 as above
 *   slots       int64 [n_slots], positions int32 [n_slots]: slot and position in
 *               the request of the step's tokens; -1 and 0 for refused requests'
 *               tokens and where there is no token
 *   spacing     0: the tokens follow each other, request after request, refused
 *               ones included (prompts packed into a step); > 0: request b's
 *               begin at entry b*spacing, and more than spacing of them do not
 *               fit (a batch whose rows stay with their requests: 1)
 * lens_out may be lens and free_count_out may be free_count. Table entries of
 * ended requests stay as they are. batch <= 8192; free_count is clamped to
 * [0, pool], and pages given back beyond the pool's size are dropped.
 * In the device error word: an ended request's length that is negative (it gives
 * nothing back) or beyond its table row (it gives the row back), and a negative page
 * number that is given back, handed out or gets a token of the step; it goes where a
 * page would, and its tokens have slot -1. How many pages the cache has is not known
 * here: numbers beyond it are named by the calls that use the slots and the table.
 */
w4a16_status w4a16_kv_extend(const int32_t *lens, const int32_t *new_tokens, int32_t *table,
                             long long table_stride, int batch, int max_pages, int page_size,
                             int32_t *free_pages, int pool, const int32_t *free_count,
                             int32_t *lens_out, int32_t *free_count_out, int64_t *slots,
                             int32_t *positions, int n_slots, int32_t *refused, int spacing, void *stream);

/*
 * Host helper: the rot_dim/2 inverse frequencies base^(-2i/rot_dim) in fp32,
 * scaled for contexts longer than `context`, the one that a model was made for.
 *   scaling  0 as they are
 *            1 all divided by factor (positions squeezed)
 *            2 base * factor^(rot_dim/(rot_dim-2)) in place of base: the lowest
 *              frequency is divided by factor, the highest stays
 *            3 by bands: with t = context * f / (2 pi) turns in the context, f stays
 *              for t >= high, is divided by factor for t <= low, and goes linearly
 *              in t from one to the other between
 * (The ramp of 3 is over turns, not over the pair's index i.)
 * rot_dim positive and even (at least 4 for scaling 2), base > 0, factor >= 1,
 * for scaling 3 context > 0 and high > low. Computed in fp64.
 */
w4a16_status w4a16_rope_frequencies(float *inv_freq, int rot_dim, double base, int scaling,
                                    double factor, double context, double low, double high);

/*
 * Rotary positions for a step's queries and keys, and its keys and values into
 * the cache. For each row r and each head of q and k, on the first rot_dim
 * elements, with x = input + bias and angle = positions[r] * inv_freq[i]:
 *     (x_a, x_b) -> m * (x_a cos - x_b sin, x_b cos + x_a sin)
 * interleaved = 0: a = i, b = i + rot_dim/2; interleaved = 1: a = 2i, b = 2i+1.
 * The other elements of q and k, and v, only get their bias.
 *   q, k, v   device, `type` (F16 or BF16), [rows][heads or kv_heads][head_dim]
 *             with row and head strides (the joined QKV projection's output is
 *             three such views); kv_heads and head_dim are the cache's
 *   bias      device, `type`, [(heads + 2*kv_heads) * head_dim] in the order q,
 *             k, v, or NULL
 *   positions device int32 [rows]; inv_freq device fp32 [rot_dim/2]
 *   mscale    the m above (1 unless the frequencies are scaled with one)
 *   q_out     device, `type`, [rows][heads][head_dim], may be q itself
 *   slots     device int64 [rows]: where k and v go; a negative slot is not
 *             written, one beyond the cache is an error and not written. Two
 *             rows with one slot leave either row's values there.
 * The product of position and frequency is reduced to a part of one turn in
 * 64-bit fixed point before it is rounded to fp32, so the angle is as exact at
 * far positions as at near ones. A frequency that is infinite or NaN gives NaN.
 * rot_dim: 0 <= rot_dim <= head_dim, a multiple of 4. Pointers 4-byte aligned,
 * strides even; 16-byte alignment throughout and rot_dim % 16 == 0 are faster.
 * The cache's type is `type` or E4M3.
 */
w4a16_status w4a16_rope_append(const void *q, const void *k, const void *v, w4a16_type type,
                               long long q_row, long long q_head, long long k_row, long long k_head,
                               long long v_row, long long v_head, const void *bias,
                               const int32_t *positions, const float *inv_freq, int rot_dim,
                               int interleaved, float mscale, void *q_out, long long qo_row,
                               long long qo_head, const w4a16_kv_cache *cache, const int64_t *slots,
                               int rows, int heads, void *stream);

/*
 * Attention of one new token of each request over its pages:
 *     s_j = scale * q . K_j,  s_j = softcap * tanh(s_j / softcap) if softcap > 0,
 *     out = sum_j exp(s_j - m) V_j / sum_j exp(s_j - m),  lse = m + log sum_j exp(s_j - m)
 * over the tokens j < lens[b] (the new one is already in the cache), and of these
 * only the last `window` if window > 0. Query head h reads kv head
 * h / (heads/kv_heads). A request with no token gets out = 0 and lse = -inf.
 * What the cache holds behind lens[b] is not used, whatever it is.
 *   q, out    device, `type` (F16 or BF16), [batch][heads][head_dim], 16-byte
 *             aligned rows and heads; out may be q
 *   cache     of `type` or E4M3; heads a multiple of its kv_heads
 *   table     device int32 [batch][max_pages], rows table_stride apart
 *   lens      device int32 [batch]. A length beyond max_pages*page_size is an
 *             error and counts as that; a page number out of range is an error,
 *             and its tokens are left out
 *   lse       device fp32 [batch][heads], or NULL
 *   ws        device scratch of w4a16_paged_attention_workspace_bytes(), 256-byte
 *             aligned. It has to be zero before its first use; every call leaves
 *             it ready for the next, of whatever shape (its size is the same for
 *             all). Calls that can overlap on the GPU need one each.
 * The result does not depend on timing: how a request's tokens are divided among
 * the SMs follows from all lengths of the call, and the parts are joined in the
 * tokens' order.
 * Scores, their maximum and the sums are fp32. Weights are rounded as operands: with a
 * 16-bit cache to two of them (2^-21 of a weight in fp16, 2^-16 in bf16), with E4M3 to
 * one of fp16 (2^-11), whose sum is also what the output is divided by. In fp16 they
 * end at 2^-35 of the largest: smaller ones count in lse, not in out. bf16 queries of
 * an E4M3 cache lose what is below 2^-25 of their head's largest. A visible infinity of
 * a 16-bit cache gives that infinity (NaN beside one of the other sign), as long as its
 * weight is not below 2^-35 of the largest.
 * Refused as unsupported: batch * heads above 2^24; batch * (32-token tiles of a table
 * row) * kv_heads * (blocks of 8 query heads) of 2^31 and more.
 */
size_t w4a16_paged_attention_workspace_bytes(int batch, int heads, int kv_heads, int head_dim);
w4a16_status w4a16_paged_attention(const void *q, w4a16_type type, long long q_row, long long q_head,
                                   const w4a16_kv_cache *cache, const int32_t *table,
                                   long long table_stride, int max_pages, const int32_t *lens,
                                   int batch, int heads, float scale, int window, float softcap,
                                   void *out, long long o_row, long long o_head, float *lse, void *ws,
                                   size_t ws_bytes, void *stream);

/*
 * A block's output into the residual stream, and the norm that the next block
 * begins with, in one pass over M rows of K elements:
 *     t = y,  t = t / sqrt(mean_k t^2 + eps) * post_gamma if post_gamma,
 *     t = t * gate if gate,
 *     h_out = h + alpha * t,
 *     n_out = h_out / sqrt(mean_k h_out^2 + eps) * gamma     (of the unrounded h_out)
 *   h, h_out  device, h_type (F16, BF16 or F32), rows h_row and ho_row apart;
 *             h_out may be h
 *   y, n_out  device, `type` (F16 or BF16); n_out may be y. gamma and n_out are
 *             both NULL where only the residual stream is wanted
 *   post_gamma, gamma  device, `type`, [K], or NULL
 *   gate      device, `type`: [K] for all rows (gate_row = 0) or [M][K] with rows
 *             gate_row apart; or NULL
 *   eps       >= 0, finite
 * K % 8 == 0, K <= 32768; all rows 16-byte aligned.
 */
w4a16_status w4a16_residual_rmsnorm(const void *h, w4a16_type h_type, long long h_row, const void *y,
                                    w4a16_type type, long long y_row, const void *post_gamma,
                                    const void *gate, long long gate_row, float alpha,
                                    const void *gamma, float eps, void *h_out, long long ho_row,
                                    void *n_out, long long no_row, int M, int K, void *stream);

/*
 * The four calls above with their arguments in one block, in the order of the
 * parameters: for callers to whom every argument of a foreign call costs time (a
 * Python program spends more of it on 24 arguments than on the launch). Same
 * checks, same results; a NULL block is W4A16_ERR_INVALID_ARG. The block is read
 * before the call returns.
 */
typedef struct {
    const int32_t *lens, *new_tokens;
    int32_t *table;
    long long table_stride;
    int batch, max_pages, page_size;
    int32_t *free_pages;
    int pool;
    const int32_t *free_count;
    int32_t *lens_out, *free_count_out;
    int64_t *slots;
    int32_t *positions;
    int n_slots;
    int32_t *refused;
    int spacing;
    void *stream;
} w4a16_kv_extend_args;
typedef struct {
    const void *q, *k, *v;
    int type;
    long long q_row, q_head, k_row, k_head, v_row, v_head;
    const void *bias;
    const int32_t *positions;
    const float *inv_freq;
    int rot_dim, interleaved;
    float mscale;
    void *q_out;
    long long qo_row, qo_head;
    const w4a16_kv_cache *cache;
    const int64_t *slots;
    int rows, heads;
    void *stream;
} w4a16_rope_append_args;
typedef struct {
    const void *q;
    int type;
    long long q_row, q_head;
    const w4a16_kv_cache *cache;
    const int32_t *table;
    long long table_stride;
    int max_pages;
    const int32_t *lens;
    int batch, heads;
    float scale;
    int window;
    float softcap;
    void *out;
    long long o_row, o_head;
    float *lse;
    void *ws;
    size_t ws_bytes;
    void *stream;
} w4a16_paged_attention_args;
typedef struct {
    const void *h;
    int h_type;
    long long h_row;
    const void *y;
    int type;
    long long y_row;
    const void *post_gamma, *gate;
    long long gate_row;
    float alpha;
    const void *gamma;
    float eps;
    void *h_out;
    long long ho_row;
    void *n_out;
    long long no_row;
    int M, K;
    void *stream;
} w4a16_residual_rmsnorm_args;
w4a16_status w4a16_kv_extend_block(const w4a16_kv_extend_args *args);
w4a16_status w4a16_rope_append_block(const w4a16_rope_append_args *args);
w4a16_status w4a16_paged_attention_block(const w4a16_paged_attention_args *args);
w4a16_status w4a16_residual_rmsnorm_block(const w4a16_residual_rmsnorm_args *args);

#ifdef __cplusplus
}
#endif

#endif /* W4A16_H */
