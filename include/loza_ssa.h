/*
 * loza_ssa.h - C ABI of the B200 (sm_100a) streaming sparse attention library.
 *
 * Streaming sparse attention (SSA) is the sparse branch of LongCat ZigZag
 * Attention (Efficient Context Scaling with LongCat ZigZag Attention, page 1,
 * section 01 (1) "calibration"): every query token attends, by softmax
 * attention, only to selected and blocked keys/values K*, V*, defined by the
 * block size b, the number of sink blocks s and the number of local blocks l.
 * Page 1 section 01 (2) fixes b = 128, s = 1, l = 7, a 1,024-token window;
 * page 5 (QbitAI article) describes it as one global block and seven local
 * blocks of 128 tokens. With query position i in block j = floor(i/b), the keys
 * of a query are
 *     t <= i  with  floor(t/b) in {0 .. s-1} U {j-l+1 .. j}
 * i.e. the sink blocks, the l most recent blocks including its own, and
 * token-causal inside its own block (the "streaming" pattern). Blocks restart
 * at every sequence start of a packed batch; a sequence's last block may be
 * short.
 *
 * The operator runs inside MLA modules (page 1 section 01 (1); page 2 section
 * 1.2). Two layouts are supported:
 *   - per-head K/V ("non-absorbed" MLA, MHA): n_kv_heads == n_heads,
 *     (d_qk, d_v) in {(64, 64), (192, 128)};
 *   - one latent KV row shared by all heads ("absorbed" MLA): n_kv_heads == 1,
 *     d_qk = 576 (512 latent + 64 rope) and d_v = 512, where V is the first 512
 *     columns of the latent row (pass v == k).
 *
 * Conventions for every entry point:
 *   - All pointers named q, k, v, out, dout, dq, dk, dv, lse, workspace,
 *     cu_seqlens and seqlens are DEVICE pointers. bf16 tensors are raw bf16
 *     bit patterns. The caller owns and allocates every buffer; the library
 *     never allocates, frees or synchronises.
 *   - Calls are asynchronous on `stream` (0 = legacy default stream).
 *   - Validation errors return a negative status BEFORE anything is launched.
 *     A launch failure returns LOZA_ERR_CUDA. Kernels never trap; a kernel
 *     that gives up on a bounded wait records LOZA_ERR_TIMEOUT, which
 *     loza_device_status() reports.
 *   - Strides are in elements. Rows (tokens) may be strided; within a row,
 *     heads are contiguous with head stride = head dim.
 *   - Every row stride times 2 bytes and every base pointer must be 16-byte
 *     aligned (TMA requirement); otherwise LOZA_ERR_INVALID_ARG.
 *   - Window: block_size b a power of two from 1 to 65,536; n_sink >= 0,
 *     n_local >= 1 (n_sink * b and n_local * b at most 2^30), or n_local ==
 *     LOZA_UNBOUNDED for full causal attention (n_sink ignored). The keys of
 *     query position i are then {t <= i : t < n_sink * b or t >= lo(i)}, lo(i)
 *     = max(0, (floor(i / b) - n_local + 1) * b). b = 1 makes every token a
 *     block: {1, 16, 1024} is the fixed part of the streaming-aware index of
 *     page 4 ("LongCat Sparse Attention ...", agihunt.info), 16 sink tokens
 *     and a 1,024-token sliding window that includes the query. The prefill
 *     and decode entry points take any such window, and so does
 *     loza_ssa_backward (bounded windows only) and loza_ssa_prefill_host.
 *     Keys are read in tiles of 128 (64 in
 *     the half-block decode): the cache rows of positions below seqlens[n]
 *     that share a tile with a visible key are read and must hold finite
 *     values (they are the sequence's own context); rows at or past
 *     seqlens[n] never reach the result, whatever they hold.
 */
#ifndef LOZA_SSA_H
#define LOZA_SSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t without the CUDA headers: the same opaque pointer. */
typedef struct CUstream_st *loza_stream_t;

/* Window parameters {b, s, l, scale}; the pages' configuration is
 * {128, 1, 7, scale}; {1, 16, 1024, scale} is page 4's token-granular sink
 * and sliding window. scale multiplies q.k before the softmax. */
typedef struct {
    int32_t block_size;
    int32_t n_sink;
    int32_t n_local;
    float scale;
} loza_ssa_params;

/* n_local value selecting full causal attention (the dense baseline). */
#define LOZA_UNBOUNDED (-1)

typedef enum {
    LOZA_OK = 0,
    LOZA_ERR_INVALID_ARG = -1,
    LOZA_ERR_UNSUPPORTED = -2,
    LOZA_ERR_WORKSPACE = -3,
    LOZA_ERR_CUDA = -4,
    LOZA_ERR_TIMEOUT = -5
} loza_status;

/* Operation codes for loza_ssa_workspace_size. */
#define LOZA_OP_PREFILL 0
#define LOZA_OP_DECODE 1
#define LOZA_OP_BACKWARD 2
#define LOZA_OP_PREFILL_HOST 3

/*
 * Bytes of device workspace the operation needs for this shape (0 if none).
 * batch: number of sequences; total_tokens: packed tokens (prefill/backward);
 * max_seqlen: longest sequence (decode: longest context). Returns 0 for an
 * unsupported shape as well; the entry point then reports the error.
 */
size_t loza_ssa_workspace_size(int op, int32_t batch, int64_t total_tokens, int32_t max_seqlen,
                               int32_t n_heads, int32_t n_kv_heads, int32_t d_qk, int32_t d_v,
                               loza_ssa_params p);

/*
 * Prefill / training forward over a packed variable-length batch.
 *   q   [T, n_heads, d_qk]     bf16, token stride q_row_stride (>= n_heads*d_qk)
 *   k   [T, n_kv_heads, d_qk]  bf16, token stride k_row_stride
 *   v   [T, n_kv_heads, d_v]   bf16, token stride v_row_stride (absorbed: v == k,
 *                              v_row_stride == k_row_stride, V = first d_v columns)
 *   cu_seqlens int32 [batch+1], cu_seqlens[0] = 0, non-decreasing,
 *               cu_seqlens[batch] == total_tokens (T)
 *   total_tokens T, the packed row count of q, k, v, out and lse (the bound the
 *               TMA descriptors are built with; rows past T read as zero)
 *   max_seqlen  >= every sequence length (sizes the launch grid)
 *   out [T, n_heads, d_v] bf16 contiguous; lse [T, n_heads] fp32, natural log of
 *   the sum of exp(scale * q.k) over the visible keys.
 *   workspace: optional. For the absorbed shapes (n_kv_heads 1, 576 / 512,
 *               even n_heads) with a bounded window of at most 32 blocks
 *               (n_sink + n_local <= 32), a workspace of at least
 *               loza_ssa_workspace_size(LOZA_OP_PREFILL, ...) bytes lets the
 *               kernel compute S once for both halves of the value dimension
 *               (it keeps P there between the two halves); with NULL or fewer
 *               bytes it recomputes S per half. Same results either way up to
 *               rounding order; the workspace is scratch owned by the caller
 *               and must not be used by other work running at the same time.
 * Definition: page 1 section 01 (1) and (2) of the LoZA pages (see above).
 */
loza_status loza_ssa_prefill(const void *q, const void *k, const void *v,
                             const int32_t *cu_seqlens, int32_t batch, int64_t total_tokens,
                             int32_t max_seqlen,
                             int32_t n_heads, int32_t n_kv_heads, int32_t d_qk, int32_t d_v,
                             int64_t q_row_stride, int64_t k_row_stride, int64_t v_row_stride,
                             loza_ssa_params p, void *out, float *lse,
                             void *workspace, size_t workspace_bytes, loza_stream_t stream);

/*
 * Prefill of a packed batch whose tensors live in host memory: the operation
 * and results of loza_ssa_prefill (same kernels; every output row is computed
 * exactly as in a device-resident call with the same cu_seqlens), with the
 * host-to-device copies of the inputs and the device-to-host copies of the
 * outputs inside the call. (The LoZA pages have no counterpart to this entry
 * point; it exists for callers whose activations are on the host.)
 *   q   [T, n_heads, d_qk]     bf16, contiguous rows
 *   k   [T, n_kv_heads, d_qk]  bf16, contiguous rows
 *   v   [T, n_kv_heads, d_v]   bf16, contiguous rows; absorbed MLA: v == k
 *                              (V = the first d_v columns of the latent row)
 *   out [T, n_heads, d_v] bf16 and lse [T, n_heads] fp32 (written)
 *   cu_seqlens: HOST int32 [batch+1], 0 = cu_seqlens[0] <= ... <=
 *               cu_seqlens[batch] = total_tokens (T); no sequence longer than
 *               max_seqlen; empty sequences are allowed
 * These five tensors may be host memory (page-locked memory lets the copies
 * run asynchronously and overlap; pageable memory gives the same results but
 * the copies serialise) or device memory; they are addressed through the
 * unified address space.
 * How it runs: each sequence's query rows are cut into chunks of whole units
 * of U = max(b, 128) rows (about 16 chunks per sequence, of 1,024 to 8,192
 * rows, at least as many as the prefix below; the unbounded window is one
 * chunk per sequence). A chunk's own rows [q0, q1) run as the local sequence
 * [sink rows | zero rows | rows q0-(l-1)b .. q0-1 | own rows] with zero query
 * rows before the own ones; the prefix is the smallest multiple of U that
 * holds the sink rows rounded up to whole 128-row tiles plus the (l-1)b halo
 * rows (exactly s + l - 1 blocks for b = 128). By the window rule (page 1
 * section 01 (1) of the LoZA pages) every own query then sees exactly its
 * keys of the whole sequence, each in the same place of its 128-row tile, so
 * the kernels read them in the same order. Up to three chunks are in flight: the
 * copy-in of one, the kernels of the next and the copy-out of a third
 * overlap, on two copy streams that the library creates on the first call per
 * device and keeps until exit. The call is asynchronous on `stream`: when
 * `stream` reaches this point of its work, out and lse hold the results.
 * Supported shapes are those of loza_ssa_prefill with n_kv_heads in
 * {1, n_heads}: (d_qk, d_v) in {(64, 64), (192, 128)} and the absorbed
 * (576, 512) with an even n_heads.
 *   workspace: device memory, 256-byte aligned, of at least
 *   loza_ssa_workspace_size(LOZA_OP_PREFILL_HOST, batch, T, max_seqlen, ...)
 *   bytes (chunk slots sized for the longest sequence, and the chunks' local
 *   cu_seqlens), owned by the caller and used by nothing else until `stream`
 *   has passed this call.
 *   Errors: LOZA_ERR_INVALID_ARG / LOZA_ERR_UNSUPPORTED / LOZA_ERR_WORKSPACE
 *   before anything is enqueued; LOZA_ERR_CUDA if enqueueing fails part way
 *   (synchronise `stream` before reusing any buffer in that case).
 */
loza_status loza_ssa_prefill_host(const void *q, const void *k, const void *v, const int32_t *cu_seqlens,
                                  int32_t batch, int64_t total_tokens, int32_t max_seqlen,
                                  int32_t n_heads, int32_t n_kv_heads, int32_t d_qk, int32_t d_v,
                                  loza_ssa_params p, void *out, float *lse,
                                  void *workspace, size_t workspace_bytes, loza_stream_t stream);

/*
 * Decode: one new query token per sequence against its KV cache.
 *   q        [batch, n_heads, d_qk] bf16 contiguous; the query of sequence n is
 *            its last token, position seqlens[n]-1, whose KV row is already in
 *            the cache (page 1 section 02: the streaming kernel in decode)
 *   k_cache  sequence n's row t at k_cache + (n*cache_batch_stride + t*cache_row_stride)
 *            elements, [n_kv_heads, d_qk] bf16 per row
 *   v_cache  absorbed MLA: NULL (or == k_cache): V is the first d_v columns of
 *            the latent row. Per-head K/V: a second cache whose strides are the
 *            K strides scaled by d_v / d_qk (both caches are [batch, Lcap,
 *            n_kv_heads, d] arrays with the same Lcap).
 *   The cache must hold at least max_seqlen rows per sequence
 *   (cache_batch_stride >= max_seqlen * cache_row_stride); rows at or past
 *   seqlens[n] are never used, whatever they contain.
 *   seqlens  int32 [batch], 1 <= seqlens[n] <= max_seqlen
 *   out [batch, n_heads, d_v] bf16; lse [batch, n_heads] fp32
 *   workspace: loza_ssa_workspace_size(LOZA_OP_DECODE, ...) bytes (split-KV
 *   partial results); contents on entry are ignored.
 * Compiled shapes: absorbed MLA (n_kv_heads == 1, 64 heads, (576, 512)) on
 * tensor cores, with split-KV partials merged in-kernel; per-head K/V
 * ((64, 64) or (192, 128)) on CUDA cores, which needs no workspace.
 */
loza_status loza_ssa_decode(const void *q, const void *k_cache, const void *v_cache,
                            const int32_t *seqlens, int32_t batch, int32_t max_seqlen,
                            int64_t cache_batch_stride, int64_t cache_row_stride,
                            int32_t n_heads, int32_t n_kv_heads, int32_t d_qk, int32_t d_v,
                            loza_ssa_params p, void *out, float *lse,
                            void *workspace, size_t workspace_bytes, loza_stream_t stream);

/*
 * Hierarchical index decode (page 4, "LongCat Sparse Attention: Taming the
 * Lightning via Streaming-aware Hierarchical Cross-Layer Indexing",
 * agihunt.info: its streaming-aware index gives every query fixed sink and
 * window tokens plus dynamically selected tokens, and its hierarchical index
 * selects those in two stages, top pages of 128 tokens first, then top tokens
 * within them). The fixed part is the SSA window `p` of this library; the
 * dynamic part is chosen among the tokens outside it, so the parts are
 * disjoint, and the query attends to both at once (one softmax over their
 * union, the same as merging the two parts by their log-sum-exp).
 * Scoring (the pages give none): the dot product of the sequence's index
 * query with a token's index key, both supplied by the caller (as an indexer
 * produces them); a page is scored by the mean of its 128 index keys. Scores
 * are fp32 fused multiply-adds over the index dimension in order, so the
 * selection is one exact set; ties go to the lower page / token index.
 * Common arguments:
 *   k_index   index keys: token t of sequence n at k_index + n *
 *             index_batch_stride + t * index_row_stride elements, d_index bf16
 *             each (d_index a multiple of 64, at most 512; 16-byte aligned;
 *             strides * 2 multiples of 16; index_batch_stride >= max_seqlen *
 *             index_row_stride)
 *   q_index   [batch, d_index] bf16 contiguous, one index query per sequence
 *   page_keys [batch, d_index, max_seqlen / 128] fp32, the page dimension
 *             innermost (from loza_hi_page_keys)
 *   seqlens   device int32 [batch], 1 <= seqlens[n] <= max_seqlen; the decode
 *             query is position seqlens[n] - 1, as in loza_ssa_decode
 *   p         the window: as loza_ssa_decode's, with at most 65,536 rows
 *             ((n_sink + n_local) * block_size); LOZA_UNBOUNDED leaves no
 *             token outside the window, so nothing is selected
 * Limits: max_seqlen / 128 <= 8192 pages; 1 <= top_k <= 2048; top_pages >= 1.
 *
 * loza_hi_page_keys: the mean index key of every whole page (tokens 128p ..
 * 128p+127 all below seqlens[n]): fp32 sums in token order times 1/128. Pages
 * past a sequence's end are not written. Maintained by the caller as its cache
 * fills (a page's mean never changes once the page is whole).
 */
loza_status loza_hi_page_keys(const void *k_index, int64_t index_batch_stride, int64_t index_row_stride,
                              const int32_t *seqlens, int32_t batch, int32_t max_seqlen, int32_t d_index,
                              float *page_keys, loza_stream_t stream);

/* Bytes of device workspace loza_hi_select and loza_hi_decode need (0 for an
 * unsupported request); loza_ssa_decode_selected needs the size for
 * top_pages = 1. */
size_t loza_hi_workspace_size(int32_t batch, int32_t max_seqlen, int32_t top_pages, int32_t top_k,
                              loza_ssa_params p);

/*
 * The tokens the hierarchical index selects for each sequence's decode query:
 * the top_pages whole pages holding a token outside the window, by page score,
 * then the top_k tokens outside the window in those pages, by token score.
 *   selected  device int32 [batch, top_k]: the tokens in ascending order, then
 *             -1 where fewer than top_k were available
 *   workspace loza_hi_workspace_size(...) bytes, 256-byte aligned
 */
loza_status loza_hi_select(const void *q_index, const void *k_index, int64_t index_batch_stride,
                           int64_t index_row_stride, const float *page_keys, const int32_t *seqlens, int32_t batch,
                           int32_t max_seqlen, int32_t d_index, loza_ssa_params p, int32_t top_pages, int32_t top_k,
                           int32_t *selected, void *workspace, size_t workspace_bytes, loza_stream_t stream);

/*
 * Softmax attention of each sequence's decode query (position seqlens[n] - 1)
 * over its window p and the tokens of a given selection (absorbed MLA: 64
 * heads, the 576-wide latent row as K, its first 512 columns as V): out
 * [batch, 64, 512] bf16, lse [batch, 64] fp32 (natural log). q [batch, 64,
 * 576] bf16 contiguous; the cache layout is loza_ssa_decode's.
 *   selected  device int32 [batch, top_k] (0 <= top_k <= 2048): entries that
 *             name a token before the query and outside the window are
 *             attended, every other entry (negative, past the query, inside
 *             the window) is ignored; the entries must be distinct
 *   workspace loza_hi_workspace_size(batch, max_seqlen, 1, top_k, p) bytes,
 *             256-byte aligned
 * The window rows and the selected rows are packed per sequence in the
 * workspace and attended by the tensor-core decode.
 */
loza_status loza_ssa_decode_selected(const void *q, const void *kv_cache, int64_t cache_batch_stride,
                                     int64_t cache_row_stride, const int32_t *seqlens, int32_t batch,
                                     int32_t max_seqlen, loza_ssa_params p, const int32_t *selected, int32_t top_k,
                                     void *out, float *lse, void *workspace, size_t workspace_bytes,
                                     loza_stream_t stream);

/*
 * The whole decode: loza_hi_select, then loza_ssa_decode_selected over the
 * window p and that selection, into out [batch, 64, 512] bf16 and lse
 * [batch, 64]. Same cache arguments as loza_ssa_decode (absorbed MLA, 64
 * heads, 576 / 512).
 *   workspace loza_hi_workspace_size(...) bytes, 256-byte aligned
 */
loza_status loza_hi_decode(const void *q, const void *kv_cache, int64_t cache_batch_stride, int64_t cache_row_stride,
                           const void *q_index, const void *k_index, int64_t index_batch_stride,
                           int64_t index_row_stride, const float *page_keys, const int32_t *seqlens, int32_t batch,
                           int32_t max_seqlen, int32_t d_index, loza_ssa_params p, int32_t top_pages, int32_t top_k,
                           void *out, float *lse, void *workspace, size_t workspace_bytes, loza_stream_t stream);

/*
 * Decode without any caller-provided device memory. (The LoZA pages have no
 * counterpart to this entry point; it exists for callers of this library.)
 *
 * Some callers cannot allocate device memory at the point where they decode:
 * a host application that owns the device allocator and gives plug-ins no
 * access to it, a serving runtime that has reserved all device memory for its
 * own KV-cache pool up front, or a latency-critical loop that must not pay
 * for cudaMalloc/cudaFree. For them this entry point takes the same arguments
 * as loza_ssa_decode minus the workspace. The absorbed decode needs scratch
 * only when a few sequences have long windows (more than 8 selected blocks
 * and batch * 16 <= number of SMs): its split-KV partial results then go to a
 * fixed 16 MiB array that is part of the library itself. Every other call
 * merges its partials on chip and needs none.
 *   - The library never allocates: every GPU that loads the library holds the
 *     16 MiB array until the process exits. With CUDA's lazy module loading
 *     (the default since CUDA 12.2) the array is placed on a device at the
 *     first call into this library on that device, whichever entry point it
 *     is; a runtime that reserves nearly all device memory for its own pool
 *     should make one call into the library on each device before it does so.
 *   - Limit: a call that needs scratch needs batch * nsplit * 132,096 bytes
 *     plus 256 for the counters, with nsplit = min(selected blocks,
 *     ceil(SMs / batch)), so it fits when batch * nsplit <= 127; e.g. with
 *     the unbounded window on a 148-SM B200, one sequence of up to 16,256
 *     tokens or four of up to 3,968 tokens. A larger call returns
 *     LOZA_ERR_WORKSPACE before anything is launched; use loza_ssa_decode with
 *     a workspace instead, or split the batch.
 *   - Every call that needs scratch looks up the array's device address on
 *     the current device (the first such call on a device also loads the
 *     library's device code there, if no earlier call did); make that first
 *     call before any stream capture on that device. After cudaDeviceReset
 *     the next call finds the array at its new address.
 *   - Every call uses the same array and leaves its last contents there; the
 *     arrival counters are cleared on the caller's stream at the start of each
 *     call. Two calls whose kernels can overlap on the GPU (different streams
 *     without ordering between them) race on the array and give wrong results.
 *   - Per-head K/V shapes need no scratch and behave exactly like
 *     loza_ssa_decode.
 */
loza_status loza_ssa_decode_noalloc(const void *q, const void *k_cache, const void *v_cache,
                                    const int32_t *seqlens, int32_t batch, int32_t max_seqlen,
                                    int64_t cache_batch_stride, int64_t cache_row_stride,
                                    int32_t n_heads, int32_t n_kv_heads, int32_t d_qk, int32_t d_v,
                                    loza_ssa_params p, void *out, float *lse, loza_stream_t stream);

/*
 * Training backward of loza_ssa_prefill (page 1 section 01 "training": the
 * model is mid-trained with SSA in place). Given q, k, v, the forward out and
 * lse, and the upstream gradient dout [T, n_heads, d_v] (bf16, contiguous),
 * writes dq [T, n_heads, d_qk], dk [T, n_kv_heads, d_qk], dv [T, n_kv_heads, d_v]
 * (bf16, contiguous); q, k, v, out and dout are contiguous [T, heads, dim]
 * tensors here. Gradients of a key block are owned by one CTA (no
 * atomics); the sink block, which every query block reads, is reduced from
 * fp32 partials in the workspace in a fixed order.
 * Only per-head K/V (n_kv_heads == n_heads) with (d_qk, d_v) in
 * {(64,64), (192,128)} is compiled for the backward.
 */
loza_status loza_ssa_backward(const void *q, const void *k, const void *v, const void *out,
                              const void *dout, const float *lse, const int32_t *cu_seqlens,
                              int32_t batch, int64_t total_tokens, int32_t max_seqlen,
                              int32_t n_heads,
                              int32_t n_kv_heads, int32_t d_qk, int32_t d_v,
                              loza_ssa_params p, void *dq, void *dk, void *dv,
                              void *workspace, size_t workspace_bytes, loza_stream_t stream);

/*
 * Absorbed decode (n_kv_heads 1, d_qk 576, d_v 512, n_heads 64) from a paged
 * latent cache: the pool holds num_pages pages of 128 rows (one 128-row tile
 * each), row r of page g at kv_pool + (g * 128 + r) * pool_row_stride
 * elements; logical block kb of sequence n (rows 128kb .. 128kb+127 of its
 * context) is page block_table[n * bt_stride + kb]. Every block the window
 * selects must have a page; other table entries are never read. Same
 * operation, outputs, workspace (loza_ssa_workspace_size(LOZA_OP_DECODE, ...)
 * with the same batch and max_seqlen) and errors as loza_ssa_decode; in
 * addition LOZA_ERR_INVALID_ARG if block_table is NULL, bt_stride <
 * ceil(max_seqlen / 128), num_pages < 1 or num_pages * 128 > INT32_MAX. A page
 * number outside [0, num_pages) reads zeros (it is not detected).
 *   block_table: device int32 [batch, bt_stride]; kv_pool: device bf16,
 *   16-byte aligned, pool_row_stride >= 576 and a multiple of 8.
 */
loza_status loza_ssa_decode_paged(const void *q, const void *kv_pool, int32_t num_pages, int64_t pool_row_stride,
                                  const int32_t *block_table, int32_t bt_stride, const int32_t *seqlens,
                                  int32_t batch, int32_t max_seqlen, int32_t n_heads, loza_ssa_params p,
                                  void *out, float *lse, void *workspace, size_t workspace_bytes,
                                  loza_stream_t stream);

/*
 * Combine two attention branches of the same (token, head) rows, each given
 * as O [rows, d_v] bf16 and LSE [rows] fp32 (natural log; -inf = a branch
 * without keys), where the branches attend to disjoint key sets (for example
 * SSA's sink + local blocks and a second set of selected blocks). Writes the
 * attention over the union of the two key sets:
 *     lse_out = ln(exp(lse_a) + exp(lse_b))
 *     out     = exp(lse_a - lse_out) o_a + exp(lse_b - lse_out) o_b
 * (both branches empty: out = 0, lse_out = -inf). This is the LSE combine of
 * the split-KV decode applied to two whole outputs.
 *   rows >= 0 (0 launches nothing); d_v a positive multiple of 8.
 *   o_a, o_b, out: device, 16-byte aligned, contiguous [rows, d_v] bf16;
 *   lse_a, lse_b, lse_out: device [rows] fp32. out may alias o_a or o_b
 *   (each element is read before it is written by the same thread).
 * Returns LOZA_ERR_INVALID_ARG for a bad size, alignment or null pointer.
 */
loza_status loza_ssa_merge(const void *o_a, const float *lse_a, const void *o_b, const float *lse_b,
                           int64_t rows, int32_t d_v, void *out, float *lse_out, loza_stream_t stream);

/*
 * Calibration mix of a module's full-attention and SSA outputs (page 1
 * section 01 (1) of the LoZA pages; the formula is lost in the page text, the
 * plain reading is used): out = alpha * o_full + (1 - alpha) * o_ssa,
 * elementwise over n bf16 values (n a multiple of 8; device pointers, 16-byte
 * aligned; out may alias either input).
 */
loza_status loza_ssa_mix(const void *o_full, const void *o_ssa, int64_t n, float alpha, void *out,
                         loza_stream_t stream);

/*
 * Serving and training around the attention: the bookkeeping of a paged
 * cache, the position rotation, norms of query and key heads, and decode over
 * paged K and V pools. (The LoZA pages name rotary dimensions (the 64 of 192
 * and 576) and paged caches only as part of the models the attention runs in;
 * these entry points are for the callers of this library.) They take their
 * arguments in a struct, which is read before the call returns; the general
 * conventions above hold (device pointers, caller's buffers, status codes).
 */

/* Element types of these entry points (the other ones are bf16). */
#define LOZA_BF16 0
#define LOZA_FP16 1
#define LOZA_FP32 2

/*
 * A paged cache: two pools of num_pages pages of page_size rows (a power of
 * two up to 65,536; num_pages * page_size <= INT32_MAX). Head h of row r of page
 * g is at base + g * page_stride + r * row_stride + h * head_stride elements,
 * its columns contiguous; so [pages, rows, heads, d] and [pages, heads, rows,
 * d] arrays, and K and V side by side in one array, are all pools. Strides are
 * in elements and >= 0. A row's number in the pool (its slot) is g *
 * page_size + r.
 */
typedef struct {
    void *k;
    void *v;               /* NULL: the latent cache, whose values are columns of k */
    int32_t num_pages;
    int32_t page_size;
    int64_t k_page_stride, k_row_stride, k_head_stride;
    int64_t v_page_stride, v_row_stride, v_head_stride;
} loza_kv_pool;

/*
 * Which columns of a head are rotated, and how: rope_dim columns (even; 0: no
 * rotation) from rope_offset. Pair i of them is (i, i + rope_dim / 2) or, if
 * interleaved is 1, (2i, 2i + 1). Pair i of a token at position t turns by t *
 * inv_freq[i]; cos and sin are multiplied by scale (1 unless the frequencies
 * were stretched by a method that asks for it).
 */
typedef struct {
    int32_t rope_dim;
    int32_t rope_offset;
    int32_t interleaved;
    float scale;
} loza_rope_params;

/* How loza_rope_frequencies stretches the frequencies for long contexts. */
#define LOZA_ROPE_NONE 0
#define LOZA_ROPE_LINEAR 1   /* every frequency divided by factor */
#define LOZA_ROPE_NTK 2      /* theta * factor ^ (rope_dim / (rope_dim - 2)) */
#define LOZA_ROPE_YARN 3     /* frequencies that make fewer than beta_slow turns over original_max
                                positions are divided by factor, those with more than beta_fast
                                turns kept, a linear ramp over the pair index between; scale
                                0.1 ln(factor) + 1 */

/*
 * The step's bookkeeping of a paged cache. Request r has ctx_lens[r] tokens in
 * the cache, in pages block_table[r * bt_stride + 0 ...], and appends
 * new_lens[r] tokens (0: it is idle in this step). Pages that the new tokens
 * need are taken from free_pages[0 .. n_free) in request order and entered in
 * the table after the ones it holds; entries before them and behind them are
 * left as they were. Written:
 *   cu_seqlens [batch + 1]  offsets of the requests' new tokens in the packed rows
 *   seqlens    [batch]      ctx + new, the cached lengths after the step
 *   positions, slots [capacity]  position and pool row of each packed token;
 *                           rows past the last token get position 0, slot -1
 *                           (which loza_qk_norm_rope does not write), so a
 *                           captured step can run at a fixed capacity
 *   counts     [3]          new tokens, pages taken, requests that were short
 * A request is short if its pages would not fit the table's max_pages columns
 * or reach past n_free: it gets no page, its new tokens slot -1 and its
 * seqlens stays ctx. Pages are dealt as if nobody were short, so pages taken
 * can exceed n_free; the caller that sees counts[2] > 0 frees pages and calls
 * again (the same call with the same lengths gives the same result). Tokens
 * past capacity are counted but not written. A negative page number in the
 * part of the table that a request holds (a page handed back because the
 * window left it) gives slot -1. Lengths outside [0, 2^30) count as 0.
 * All pointers are device memory, on their type's alignment, positions and
 * slots on 16 bytes. What is written (the table's rows included) must share no
 * memory with what is read nor with each other (LOZA_ERR_INVALID_ARG): lengths
 * do not advance in place. Page numbers in free_pages must be distinct and not
 * in use. max_pages <= bt_stride; page_size a power of two up to 65,536; at
 * most 16,384 requests (LOZA_ERR_UNSUPPORTED beyond).
 */
typedef struct {
    const int32_t *ctx_lens, *new_lens, *free_pages;
    int32_t *block_table;
    int32_t *cu_seqlens, *seqlens, *positions;
    int64_t *slots;
    int32_t *counts;
    int64_t bt_stride, capacity;
    int32_t batch, n_free, page_size, max_pages;
} loza_page_plan_args;
loza_status loza_page_plan(const loza_page_plan_args *args, loza_stream_t stream);

/*
 * Host function: the angles per position of rope_dim / 2 pairs,
 * theta^(-2i / rope_dim) stretched by `scaling`, into inv_freq (HOST memory,
 * rope_dim / 2 doubles), and the factor for loza_rope_params.scale. factor >= 1
 * is the ratio of the extended to the original context length; original_max,
 * beta_fast and beta_slow are read by LOZA_ROPE_YARN only (usually 32 and 1).
 * Angles are 64-bit throughout: a 32-bit product is off by 0.03 rad at
 * position 10^6. Any other table of frequencies may be used as well.
 */
loza_status loza_rope_frequencies(double theta, int32_t rope_dim, int32_t scaling, double factor,
                                  double original_max, double beta_fast, double beta_slow,
                                  double *inv_freq, float *scale);

/*
 * Rotation of one tensor: out[t, h] = x[t, h] with the columns of `rope` turned
 * by positions[t]. x, out [tokens, n_heads, d] (0 <= tokens <= 2^30, n_heads
 * <= 65,535, d <= 1024), rows x_row_stride and out_row_stride elements apart (at
 * least n_heads * d), heads contiguous within a row, dtype any of the three;
 * positions device int32 [tokens] (any value, any order); inv_freq DEVICE
 * double [rope_dim / 2]. out may be x with the same stride (then only the
 * rotated columns are touched) or must not overlap it. transposed = 1 applies
 * the transposed map, which is the gradient: dx from dout. 32-bit arithmetic,
 * one rounding. Where the head's size, rope_offset, HALF of rope_dim (and
 * norm_dim below), strides and pointers are all multiples of 16 bytes, rows move
 * in 16-byte vectors; else, for 16-bit types, in vectors of 4 bytes if they are
 * all multiples of that, else element by element: two to five times as long.
 */
typedef struct {
    const void *x;
    const int32_t *positions;
    const double *inv_freq;
    void *out;
    int64_t tokens, x_row_stride, out_row_stride;
    int32_t n_heads, d;
    loza_rope_params rope;
    int32_t transposed, dtype;
} loza_rope_args;
loza_status loza_rope(const loza_rope_args *args, loza_stream_t stream);

/*
 * Norm of each query and key head, the rotation, and the write into a paged
 * cache, in one pass. Per head row x of q [tokens, n_heads, d] and k [tokens,
 * n_kv_heads, d]:
 *     n_c = weight_c x_c / sqrt(mean(x_0 .. x_{norm_dim-1} squared) + eps)  for c < norm_dim
 *     n_c = x_c  for the other columns, and for a side whose weight is NULL
 * then the rotation of loza_rope; 32-bit arithmetic (squares above 3.4e38
 * overflow), one rounding; eps >= 0; sizes as there.
 *   q, k, v   rows q_row_stride, k_row_stride, v_row_stride elements apart, so
 *             they may be slices of one projection's rows; n_heads or
 *             n_kv_heads may be 0 (that side's arguments are then not read)
 *   q_weight, k_weight  [norm_dim] of the same dtype, or NULL
 *   q_out, k_out  as q and k, with their own row strides; each may be its
 *             input with the same stride, or must not overlap any input.
 *             k_out may be NULL when a pool is given
 *   pool      none (pool.k NULL), or the cache: token t's key heads (after norm and
 *             rotation) and v's rows [n_kv_heads, d_v] go to row slots[t];
 *             a slot outside [0, num_pages * page_size) writes nothing.
 *             pool.v and v are both given or both NULL (the latent cache:
 *             d = 576, norm_dim = 512, rope_offset = 512). Slots must be
 *             distinct (except those that write nothing); every page_size
 *             from 1 on is taken here
 *   slots     device int64 [tokens] (from loza_page_plan), NULL without a pool
 */
typedef struct {
    const void *q, *k, *v;
    const int32_t *positions;
    const double *inv_freq;
    const void *q_weight, *k_weight;
    void *q_out, *k_out;
    const int64_t *slots;
    loza_kv_pool pool;      /* pool.k NULL: none */
    int64_t tokens;
    int64_t q_row_stride, k_row_stride, v_row_stride, q_out_row_stride, k_out_row_stride;
    int32_t n_heads, n_kv_heads, d, d_v, norm_dim;
    float eps;
    loza_rope_params rope;
    int32_t dtype;
} loza_qk_norm_rope_args;
loza_status loza_qk_norm_rope(const loza_qk_norm_rope_args *args, loza_stream_t stream);

/* Bytes of workspace loza_qk_norm_rope_backward needs when a weight is given (0: norm_dim out of range). */
size_t loza_qk_norm_rope_workspace_size(int32_t norm_dim);

/*
 * Gradient of loza_qk_norm_rope: from dq_out and dk_out (the gradients of
 * q_out and k_out) and the forward's inputs, dq, dk (same dtype) and the
 * weights' gradients dq_weight, dk_weight ([norm_dim] fp32, written, summed
 * over all tokens and heads; each given exactly if its weight is, and in memory
 * of its own: the gradient of a weight of both sides is their sum). A side
 * without weight needs no q (k). The sums' order is fixed: no atomics, the
 * same bits every run on one kind of GPU. dq may replace dq_out or q, and dk
 * dk_out or k, with the same row strides.
 *   workspace: loza_qk_norm_rope_workspace_size(norm_dim) bytes, 16-byte
 *   aligned, unless both weights are NULL; contents on entry are ignored
 */
typedef struct {
    const void *dq_out, *dk_out, *q, *k;
    const int32_t *positions;
    const double *inv_freq;
    const void *q_weight, *k_weight;
    void *dq, *dk;
    float *dq_weight, *dk_weight;
    void *workspace;
    size_t workspace_bytes;
    int64_t tokens;
    int64_t dq_out_row_stride, dk_out_row_stride, q_row_stride, k_row_stride, dq_row_stride, dk_row_stride;
    int32_t n_heads, n_kv_heads, d, norm_dim;
    float eps;
    loza_rope_params rope;
    int32_t dtype;
} loza_qk_norm_rope_backward_args;
loza_status loza_qk_norm_rope_backward(const loza_qk_norm_rope_backward_args *args, loza_stream_t stream);

/* Bytes of workspace loza_ssa_decode_paged_kv needs, whatever the batch and the lengths (0: unsupported shape). */
size_t loza_decode_paged_kv_workspace_size(int32_t n_heads, int32_t n_kv_heads, int32_t d_qk, int32_t d_v);

/*
 * Decode over paged K and V pools with heads of their own or shared by groups:
 * the operation of loza_ssa_decode (`window` at the sequence's last position,
 * LOZA_UNBOUNDED included) for n_heads a multiple of n_kv_heads, (d_qk, d_v) in
 * {(64,64), (128,128), (192,128)}, bf16 or fp16. The work is split over the
 * keys of all sequences together, so one long sequence and many ragged ones
 * both fill the GPU.
 *   q       [batch, n_heads, d_qk], rows q_row_stride elements apart
 *   pool    both pools given, 16-byte aligned (as q and out), every stride a
 *           multiple of 8 elements, page_size >= 16
 *   block_table  device int32, page of key t of sequence n: block_table[n *
 *           bt_stride + t / page_size]; bt_stride >= ceil(max_seqlen /
 *           page_size). Only entries of pages that hold a key below
 *           seqlens[n] within 64 keys of the window are read. A page number
 *           outside [0, num_pages) holds no keys: they get no weight
 *   seqlens device int32 [batch], 0 <= seqlens[n] <= max_seqlen <= 2^30 (taken
 *           to be in that range if it is not); the query of sequence n is its key
 *           seqlens[n] - 1. A sequence of length 0 (an idle row of a padded
 *           batch), or none of whose pages is there, gives out 0 and lse -inf
 *   Rows at or past seqlens[n], and rows outside the window, are not read.
 *   An infinity or NaN in a visible row of v leaves an infinity or NaN in its
 *   column, also where the row's weight has underflowed to 0
 *   out     [batch, n_heads, d_v] of the same dtype; lse [batch, n_heads] fp32
 *   workspace  loza_decode_paged_kv_workspace_size(...) bytes, 16-byte
 *           aligned, contents on entry ignored; calls that can overlap on the
 *           GPU need one each
 */
typedef struct {
    const void *q;
    loza_kv_pool pool;
    const int32_t *block_table, *seqlens;
    void *out;
    float *lse;
    void *workspace;
    size_t workspace_bytes;
    int64_t q_row_stride, bt_stride;
    int32_t batch, max_seqlen, n_heads, n_kv_heads, d_qk, d_v;
    loza_ssa_params window;
    int32_t dtype;
} loza_decode_paged_kv_args;
loza_status loza_ssa_decode_paged_kv(const loza_decode_paged_kv_args *args, loza_stream_t stream);

/* Human-readable name of a status code (static string). */
const char *loza_status_string(loza_status s);

/*
 * Synchronises `stream`, then returns and clears the library's device-side
 * status word: LOZA_OK, or LOZA_ERR_TIMEOUT if a kernel gave up on a bounded
 * wait since the last call. LOZA_ERR_CUDA if the synchronisation failed.
 */
loza_status loza_device_status(loza_stream_t stream);

/* Number of kernel launches the library issued since load (all entry points). */
uint64_t loza_launch_count(void);

/*
 * Self-test of the bounded waits: launches one thread that waits on an
 * mbarrier nothing completes; after limit_us microseconds (1 ... 2,000,000)
 * it gives up and records a timeout exactly as a kernel's own wait would, so
 * the next loza_device_status returns LOZA_ERR_TIMEOUT and the context stays
 * usable. (Every wait in the library's kernels has the same bound, 2 s.)
 * LOZA_ERR_INVALID_ARG for a limit out of range.
 */
loza_status loza_wait_selftest(uint32_t limit_us, loza_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LOZA_SSA_H */
