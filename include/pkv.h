/*
 * pkv.h - C ABI of libpkv: attention over a paged KV cache on GB300 (sm_103a).
 *
 * The KV cache of one attention layer is one contiguous physical pool per
 * tensor, K and V, each bf16 [num_pages * page_size, H_kv, D] (token-major,
 * row-major, contiguous). A page table, int32 [max_batch, max_blocks]
 * row-major, maps (batch slot, logical block) to a physical page. Batch slot 0
 * and page 0 are reserved as no-op padding; an entry of -1 means "no page
 * reserved". Source: "flex_paged_attention.py" commit log, section "Why this
 * works", items 1 and 3.
 *
 * Three stream-ordered calls replace the pages' PagedKVCache.update followed
 * by flex_attention(q, k, v, scale, block_mask, enable_gqa=True)
 * ("qwen3_flex_inference.py", attention forward, _decode_step_eager,
 * _prefill):
 *   pkv_append            - write new tokens' K/V rows through the page table
 *   pkv_append_rope       - the same with k_norm and the rotary embedding
 *                           applied to K
 *   pkv_prefill_paged_attention - chunked prefill / mixed prefill + decode
 *                           tokens attending their slots' keys through pages
 *   pkv_decode_attention  - one query token per row, GQA, over the pages
 *   pkv_prefill_attention - packed document-causal attention over fresh k/v
 * and, for serving with drafted tokens and shared prefixes over the same
 * cache (the pages have no counterpart; these are operators of this library):
 *   pkv_tree_attention    - a tree of drafted tokens over the cached context
 *   pkv_verify_tree       - which drafted tokens the target accepts, and the
 *                           next token
 *   pkv_commit_path       - the accepted path's K/V rows moved next to the
 *                           committed context
 *   pkv_update_pages      - fork, reserve, copy on write, truncate and free
 *   pkv_compact_pages     - live pages moved to the low end of the pool
 * and, for attention whose keys and values come from one latent vector a token
 * that all heads share (further operators of this library):
 *   pkv_rotate            - the rotary embedding, interleaved or in halves
 *   pkv_latent_append     - new tokens' rows, normalised and rotated, written
 *                           through the page table
 *   pkv_latent_gather     - cached rows read back through the page table
 *   pkv_latent_decode_attention  - the absorbed form, over the cached rows
 *   pkv_latent_prefill_attention - the expanded form, packed sequences
 *
 * Conventions for every call:
 *  - All tensor pointers are DEVICE pointers owned by the caller. The library
 *    keeps no pointer after the call returns and allocates no device memory;
 *    scratch space, where needed, is a caller-provided workspace.
 *  - Arguments are validated on the host, synchronously, before anything is
 *    launched; a failed check returns its status and launches nothing.
 *  - Problems only visible on the device (a page entry outside [0, num_pages),
 *    a slot outside [0, max_batch), a position past the table) never trap:
 *    the affected work is skipped and a PKV_DEV_ERR_* bit is OR-ed into the
 *    optional int32 word dev_err (device memory, may be NULL). The caller
 *    reads it after synchronising the stream. Results of affected rows are
 *    unspecified; everything else is still computed.
 *  - Calls only enqueue work on `stream` (NULL = the legacy default stream),
 *    never synchronise it, and keep no state between calls, so they may be
 *    captured into a CUDA graph.
 *  - head_dim must be 128 (the pkv_latent_* calls: 576, with num_kv_heads 1);
 *    num_q_heads / num_kv_heads (the GQA group) must be 1, 2, 4 or 8; page_size
 *    must be a positive multiple of 16; bf16 tensors must be 16-byte aligned;
 *    int32/fp32 arrays 4-byte aligned.
 */
#ifndef PKV_H
#define PKV_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PKV_OK = 0,
  PKV_ERR_ARG = 1,        /* bad size, null pointer or unsupported shape   */
  PKV_ERR_ALIGN = 2,      /* a pointer misses its required alignment       */
  PKV_ERR_BAD_PAGE = 3,   /* pkv_status_from_device_error: bad page entry  */
  PKV_ERR_WORKSPACE = 4,  /* workspace missing or smaller than required    */
  PKV_ERR_CUDA = 5,       /* a CUDA runtime call failed (launch, query)    */
  PKV_ERR_DEVICE = 6,     /* current device is not a supported sm_103 GPU  */
  PKV_ERR_BAD_INPUT = 7   /* pkv_status_from_device_error: other device err */
} pkv_status;

/* Bits OR-ed into *dev_err by the kernels. */
#define PKV_DEV_ERR_BAD_PAGE   0x1  /* page entry not in [0, num_pages)          */
#define PKV_DEV_ERR_BAD_SLOT   0x2  /* batch_idx not in [0, max_batch)           */
#define PKV_DEV_ERR_BAD_POS    0x4  /* position/seq_len < 0 or past max_blocks   */
#define PKV_DEV_ERR_LAYOUT     0x8  /* prefill packing precondition violated     */
#define PKV_DEV_ERR_TIMEOUT    0x10 /* a bounded wait inside a kernel gave up    */
#define PKV_DEV_ERR_BAD_TREE   0x20 /* tree size, parent, path or token invalid  */
#define PKV_DEV_ERR_NO_PAGES   0x40 /* not enough free pages for a row           */
#define PKV_DEV_ERR_BAD_PROBS  0x80 /* a probability row sums to 0, inf or NaN   */

/* Most nodes of a tree of drafted tokens (a node's ancestors are one 64-bit
 * mask). */
#define PKV_MAX_TREE_NODES 64

/* Geometry of one layer's paged cache. */
typedef struct {
  int num_pages;     /* P: physical pages per pool (page 0 reserved)          */
  int page_size;     /* ps: token slots per page, multiple of 16               */
  int num_kv_heads;  /* H_kv                                                   */
  int head_dim;      /* D, must be 128                                         */
  int max_batch;     /* rows of page_table (slot 0 reserved)                   */
  int max_blocks;    /* columns of page_table: logical blocks per sequence     */
} pkv_cache_desc;

/*
 * pkv_append - KV append through the page table.
 * Source: "qwen3_flex_inference.py", attention forward ("Write to paged KV
 * cache"), capture_decode_cudagraph (the k_cache[addr] = k_val write); the
 * crash on an unreserved entry: "flex_paged_attention.py" commit log, "Files".
 *
 * For each token i in [0, n_tokens) with slot b = batch_idx[i] and position
 * p = input_pos[i], copies the bytes of k_new[i] and v_new[i] (each bf16
 * [H_kv, D], contiguous rows of a [n_tokens, H_kv, D] tensor) to pool row
 *     page_table[b, p / ps] * ps + p % ps
 * of k_pool and v_pool. Bit-exact byte copy. Tokens with b == 0 (padding
 * slot) are skipped without error. A token whose slot, block or page entry is
 * out of range is skipped and sets PKV_DEV_ERR_BAD_SLOT / _BAD_POS / _BAD_PAGE.
 * Two tokens that address the same row race (the last writer is unspecified).
 * Decode passes n_tokens = B (one new token per row), prefill passes the
 * packed tokens.
 */
pkv_status pkv_append(const pkv_cache_desc* cache, void* k_pool, void* v_pool,
                      const int32_t* page_table, const void* k_new,
                      const void* v_new, const int32_t* batch_idx,
                      const int32_t* input_pos, int n_tokens, int32_t* dev_err,
                      cudaStream_t stream);

/*
 * pkv_append_rope - pkv_append with the model's per-head k_norm (optional)
 * and the rotary position embedding applied to each new K row on the way
 * into the pool (V rows are copied unchanged).
 * Source: "qwen3_flex_inference.py", attention forward (k = k_norm(k_proj(..)
 * per head), then _apply_rotary: x * cos + rotate_half(x) * sin with
 * rotate_half(x) = cat(-x2, x1), right before the cache write).
 *
 * rope_cos, rope_sin: fp32 [rope_len, D/2] row-major, 16-byte aligned; row p
 * holds the cos/sin of the angles of position p (the full-width tables repeat
 * them for the second half of D). For each kv head of token i at position
 * p = input_pos[i], with x1 = k_new[i][h][0:D/2], x2 = k_new[i][h][D/2:D],
 * c = rope_cos[p], s = rope_sin[p]:
 *     K row = bf16_rne(concat(x1*c - x2*s, x2*c + x1*s))   (computed in fp32)
 * k_norm_weight: null (no normalisation) or fp32 [D], 16-byte aligned. When
 * given, each head x of k_new[i] is first replaced by
 *     x_d * k_norm_weight[d] / sqrt(mean_d(x_d^2) + k_norm_eps)
 * (the pages name the k_norm module; this is the Qwen3 family's RMSNorm over
 * the head dims), kept in fp32 and rotated, with one rounding to bf16 at the
 * end. k_norm_eps must be finite and >= 0 (else PKV_ERR_ARG); it is ignored
 * without a weight.
 * A position outside [0, rope_len) sets PKV_DEV_ERR_BAD_POS and skips the
 * token; everything else (slots, pages, errors, races) is as pkv_append.
 */
pkv_status pkv_append_rope(const pkv_cache_desc* cache, void* k_pool, void* v_pool,
                           const int32_t* page_table, const void* k_new,
                           const void* v_new, const int32_t* batch_idx,
                           const int32_t* input_pos, int n_tokens,
                           const float* rope_cos, const float* rope_sin, int rope_len,
                           const float* k_norm_weight, float k_norm_eps,
                           int32_t* dev_err, cudaStream_t stream);

/*
 * pkv_decode_workspace_size - bytes of workspace pkv_decode_attention needs
 * on the CURRENT device for `batch` rows and `num_q_heads` query heads.
 * max_seq_len is accepted for interface stability; the split-KV schedule
 * balances work over the device's SMs and its scratch does not grow with
 * sequence length. A batch above 512 rows runs as equal launches of at most
 * 512 rows that reuse the workspace, so the size is that of one launch.
 * Returns 0 for invalid arguments.
 */
size_t pkv_decode_workspace_size(const pkv_cache_desc* cache, int batch,
                                 int num_q_heads, int max_seq_len);

/*
 * pkv_decode_attention - split-KV GQA decode over the paged cache.
 * Source: "qwen3_flex_inference.py", _decode_block_mask (causal_offset:
 * keys kv_idx <= input_pos of the row's own slot), attention forward
 * (enable_gqa); zero-safe padded rows: "flex_vs_vllm.md", "What broke
 * correctness and had to be dropped" (ROWS_GUARANTEED_SAFE).
 *
 * batch may be any count >= 0. Above 512 rows (the kernels' row tables in
 * shared memory) the call enqueues equal launches of at most 512 rows each,
 * in row order on `stream`, sharing the workspace.
 * Row b in [0, batch) has one query token q[b] (bf16 [num_q_heads, D] within
 * a contiguous [batch, num_q_heads, D] tensor) and attends the first
 * n = seq_lens[b] logical keys of slot c = batch_idx[b] (for a decode step
 * seq_lens[b] = input_pos[b] + 1, the new token included). Query head h reads
 * kv head h / (num_q_heads / num_kv_heads). Writes
 *   lse[b, h] = ln sum_{t<n} exp(scale * q[b,h] . K[c,t,kvh])       (fp32)
 *   out[b, h] = sum_{t<n} exp(scale * q[b,h] . K[c,t,kvh] - lse) V[c,t,kvh]
 * out: bf16 [batch, num_q_heads, D] (rounded to nearest even); lse: fp32
 * [batch, num_q_heads], natural log. Rows with c == 0 or n == 0 give out = 0
 * and lse = -inf (never NaN). A row with c outside [0, max_batch) or
 * n > max_blocks * page_size (or n < 0) sets a PKV_DEV_ERR bit and gives
 * 0 / -inf; a page entry out of range within the first n keys sets
 * PKV_DEV_ERR_BAD_PAGE and leaves that row unspecified.
 * out and lse are only written, with plain stores (no bulk copies): besides
 * device memory they may be pinned host memory mapped into the device's
 * address space (unified addressing), so that the results land on the host
 * without a separate copy; the caller synchronises the stream before reading.
 *
 * q, batch_idx and seq_lens (and k_new, v_new of the fused call) may
 * likewise be pinned host memory mapped into the device's address space:
 * the kernels then read them over the host link (q's rows by ordinary
 * asynchronous copies, the rest by plain loads), so a step needs no input
 * copy; the host must not rewrite them before the call has completed. q in
 * pageable host memory, which the GPU cannot read, returns PKV_ERR_ARG. The
 * pools, the page table, the workspace and dev_err stay in device memory.
 *
 * workspace: device scratch of at least pkv_decode_workspace_size() bytes,
 * 256-byte aligned, owned by the caller; its contents need no initialisation
 * and are overwritten; calls that share a workspace must be stream-ordered.
 * Each launch runs two kernels: the split-KV pass and the LSE merge.
 */
pkv_status pkv_decode_attention(const pkv_cache_desc* cache, const void* k_pool,
                                const void* v_pool, const int32_t* page_table,
                                const void* q, int num_q_heads,
                                const int32_t* batch_idx,
                                const int32_t* seq_lens, int batch, float scale,
                                void* out, float* lse, void* workspace,
                                size_t workspace_bytes, int32_t* dev_err,
                                cudaStream_t stream);

/*
 * pkv_decode_append_attention - one decode step's KV append fused into the
 * decode attention (one launch fewer than pkv_append + pkv_decode_attention).
 * Source: the pages' decode step writes the new token's K/V into the paged
 * cache, then attends over the cache including it ("qwen3_flex_inference.py",
 * forward "Write to paged KV cache" then flex_attention with
 * _decode_block_mask); fused, a step is one call and one launch fewer.
 *
 * Same arguments and results as pkv_decode_attention, plus k_new, v_new:
 * bf16 [batch, num_kv_heads, D], 16-byte aligned. Row b's new token is
 * written to position seq_lens[b] - 1 of slot batch_idx[b] (a decode step has
 * seq_lens[b] = input_pos[b] + 1), exactly as pkv_append would write it
 * (bit-exact byte copy), and the attention of row b includes it. Rows that
 * attend nothing (batch_idx 0, seq_lens 0, or rejected entries) write
 * nothing. A page entry for the new position outside [0, num_pages) skips
 * that write and sets PKV_DEV_ERR_BAD_PAGE. The pools are written, so they
 * are non-const here; k_pool/v_pool must not alias k_new/v_new.
 */
pkv_status pkv_decode_append_attention(const pkv_cache_desc* cache, void* k_pool,
                                       void* v_pool, const int32_t* page_table,
                                       const void* q, int num_q_heads,
                                       const void* k_new, const void* v_new,
                                       const int32_t* batch_idx,
                                       const int32_t* seq_lens, int batch,
                                       float scale, void* out, float* lse,
                                       void* workspace, size_t workspace_bytes,
                                       int32_t* dev_err, cudaStream_t stream);

/*
 * pkv_decode_attention_static_scratch - pkv_decode_attention for callers that
 * cannot allocate device memory. The source pages have no counterpart: this
 * is a deployment convenience of this library.
 *
 * Some callers cannot hand pkv_decode_attention a workspace, because they may
 * not call cudaMalloc at all: code that runs inside a custom allocator's own
 * hooks, processes whose device memory is reserved entirely at start-up, or
 * plug-in hosts that forbid allocations once running. This entry point takes
 * the same arguments minus the workspace and uses a scratch array compiled
 * into the library instead: a file-scope __device__ array of 8 MiB, held on
 * every GPU that loads the library until the process exits. It allocates
 * nothing and calls no allocating routine.
 *  - A call whose pkv_decode_workspace_size() exceeds 8 MiB returns
 *    PKV_ERR_WORKSPACE without launching (one launch of more than about 350
 *    rows at 8 KV heads and a GQA group of 4 on a 152-SM GB300; a batch above
 *    512 rows runs as equal launches, so whether it fits depends on their
 *    size, which pkv_decode_workspace_size() reflects; use
 *    pkv_decode_attention where it does not fit).
 *  - The first call on a device looks up the array's device address
 *    (cudaGetSymbolAddress) with that device current and caches it; make that
 *    first call before any stream capture. A failed lookup returns
 *    PKV_ERR_CUDA (its text in pkv_last_cuda_error_string()). The cached
 *    address does not survive cudaDeviceReset: after a reset, do not use
 *    this entry point on that device again in the same process.
 *  - Other argument errors give the status pkv_decode_attention gives for
 *    them (an empty batch is validated the same way and returns PKV_OK).
 *  - All calls share the one array. Its contents from the previous call are
 *    never read before being overwritten, so nothing needs clearing, but two
 *    calls whose kernels overlap on the GPU (different streams, or different
 *    host threads without ordering) race on it: keep them stream-ordered.
 * Results are those of pkv_decode_attention on the same inputs.
 */
pkv_status pkv_decode_attention_static_scratch(
    const pkv_cache_desc* cache, const void* k_pool, const void* v_pool,
    const int32_t* page_table, const void* q, int num_q_heads,
    const int32_t* batch_idx, const int32_t* seq_lens, int batch, float scale,
    void* out, float* lse, int32_t* dev_err, cudaStream_t stream);

/*
 * pkv_prefill_paged_attention - chunked prefill over the paged cache, on
 * tcgen05 tensor cores. Source: the step the pages leave on the table
 * ("flex_vs_vllm.md", "What's left on the table": chunked prefill, prefill
 * and decode interleaved in one pass, reading earlier context from the
 * pages); the per-token rule is the decode rule ("qwen3_flex_inference.py",
 * _decode_block_mask, causal_offset: keys kv_idx <= input_pos).
 *
 * q: bf16 [n_tokens, num_q_heads, D], 16-byte aligned; batch_idx, input_pos:
 * int32 [n_tokens]. Token i attends the logical keys 0..input_pos[i] of slot
 * batch_idx[i], read through page_table from k_pool/v_pool:
 *   lse[i, h] = ln sum_{t<=p} exp(scale * q[i,h] . K[slot,t,kvh])       (fp32)
 *   out[i, h] = sum_{t<=p} exp(scale * q[i,h] . K[slot,t,kvh] - lse) V[slot,t,kvh]
 * with kvh = h / (num_q_heads / num_kv_heads). The keys of the token's own
 * chunk must be in the pools already (pkv_append first). Tokens need no order
 * or packing: a chunk of a prompt is its tokens with consecutive positions, a
 * decode token is a chunk of one, and both can share a call. Tokens of slot 0
 * give out 0, lse -inf. A slot outside [0, max_batch) or a position outside
 * [0, max_blocks * page_size) sets PKV_DEV_ERR_BAD_SLOT / _BAD_POS and gives
 * 0 / -inf; an unreserved page entry among a token's keys sets
 * PKV_DEV_ERR_BAD_PAGE and leaves that token's result unspecified.
 * page_size must be 16, 32, 64 or a multiple of 128 (PKV_ERR_ARG otherwise);
 * scale must be finite and > 0. out: bf16 [n_tokens, num_q_heads, D] and
 * lse: fp32 [n_tokens, num_q_heads], 16- and 4-byte aligned. The pools are
 * only read. A decode token costs a full 128-row product per key tile of its
 * prefix here: in a step that mixes chunks and decode tokens, the decode
 * tokens are cheaper through pkv_decode_append_attention.
 */
pkv_status pkv_prefill_paged_attention(const pkv_cache_desc* cache, const void* k_pool,
                                       const void* v_pool, const int32_t* page_table,
                                       const void* q, int num_q_heads,
                                       const int32_t* batch_idx,
                                       const int32_t* input_pos, int n_tokens,
                                       float scale, void* out, float* lse,
                                       int32_t* dev_err, cudaStream_t stream);

/*
 * pkv_prefill_attention - packed document-causal prefill on tcgen05 tensor
 * cores. Source: "qwen3_flex_inference.py", _prefill (prompts concatenated
 * into one sequence with a document-causal mask; the mask built without
 * paging, so attention reads the packed fresh k/v).
 *
 * q: bf16 [n_tokens, num_q_heads, D]; k, v: bf16 [n_tokens, num_kv_heads, D];
 * batch_idx, input_pos: int32 [n_tokens]. Token i may attend token j iff
 * batch_idx[j] == batch_idx[i] != 0 and input_pos[j] <= input_pos[i].
 * Precondition (the pages' packing): each document's tokens are contiguous
 * and numbered input_pos = 0, 1, 2, ...; padding tokens carry batch_idx 0.
 * A token that breaks it sets PKV_DEV_ERR_LAYOUT (its row is unspecified).
 * Writes out bf16 [n_tokens, num_q_heads, D] and lse fp32
 * [n_tokens, num_q_heads] with the same formulas as decode; padding tokens
 * give 0 / -inf. scale must be finite and > 0. q, k, v and out are
 * 16-byte aligned device memory (out is written with bulk tensor stores).
 * Writing the k/v into the pages is a separate pkv_append.
 */
pkv_status pkv_prefill_attention(const void* q, const void* k, const void* v,
                                 int num_q_heads, int num_kv_heads,
                                 int head_dim, const int32_t* batch_idx,
                                 const int32_t* input_pos, int n_tokens,
                                 float scale, void* out, float* lse,
                                 int32_t* dev_err, cudaStream_t stream);

/*
 * pkv_mixed_workspace_size - bytes of device scratch pkv_mixed_attention
 * needs for n_tokens tokens (0 for invalid arguments).
 */
size_t pkv_mixed_workspace_size(const pkv_cache_desc* cache, int n_tokens,
                                int num_q_heads);

/*
 * pkv_mixed_attention - one call for a step that interleaves prefill chunks
 * and decode tokens, each token attending its slot's keys 0..input_pos
 * through the page table. Source: the step the pages leave on the table,
 * prefill and decode served in one pass ("flex_vs_vllm.md", "What's left on
 * the table"); the rule per token is the decode rule
 * ("qwen3_flex_inference.py", _decode_block_mask, causal_offset).
 *
 * Arguments, results and error behaviour are those of
 * pkv_prefill_paged_attention (the same out and lse, within rounding), plus
 * a workspace: device scratch of at least pkv_mixed_workspace_size() bytes,
 * 256-byte aligned, owned by the caller, no initialisation needed; calls
 * sharing one must be stream-ordered. Inside, tokens that are a run of one
 * in the packing (a live slot different from both neighbours' slots: decode
 * tokens) are routed to the split-KV decode kernels, up to 512 of them in
 * token order; every other token goes through the chunked prefill, where a
 * lone token would cost a full 128-row product per key tile of its prefix.
 * Four kernels run on `stream`: the routing, the chunked prefill, the
 * split-KV decode and its merge. The chunks' and decode tokens' own K/V must
 * be in the pools already (pkv_append first). page_size must be 16, 32, 64
 * or a multiple of 128.
 */
pkv_status pkv_mixed_attention(const pkv_cache_desc* cache, const void* k_pool,
                               const void* v_pool, const int32_t* page_table,
                               const void* q, int num_q_heads,
                               const int32_t* batch_idx, const int32_t* input_pos,
                               int n_tokens, float scale, void* out, float* lse,
                               void* workspace, size_t workspace_bytes,
                               int32_t* dev_err, cudaStream_t stream);

/*
 * pkv_stage_from_host - copies a step's inputs from pinned host memory into
 * device memory with the GPU's own loads. Source: the pages' decode step
 * copies each step's inputs into the static buffers its captured graph reads,
 * then replays the graph ("qwen3_flex_inference.py", _decode_step and
 * capture_decode_cudagraph). On GB300 a copy-engine transfer of such a step's
 * inputs (under 1 MB) costs ~14 us of mostly fixed latency; read by the SMs
 * over the coherent host link it takes a few microseconds.
 *
 * dst: device (or managed) memory; src: pinned host memory (cudaHostAlloc,
 * cudaMallocHost or cudaHostRegister; device memory also works); bytes a
 * multiple of 16, both pointers 16-byte aligned (PKV_ERR_ARG /
 * PKV_ERR_ALIGN otherwise, nothing launched). Memory the GPU cannot reach
 * (pageable host memory) is rejected with PKV_ERR_ARG before any launch.
 * The copy is one kernel on `stream`; a kernel that starts after it on the
 * stream (a programmatic dependent such as the decode kernels included)
 * sees the copied bytes. src must not change until the copy has run.
 */
pkv_status pkv_stage_from_host(void* dst, const void* src, size_t bytes,
                               cudaStream_t stream);

/*
 * pkv_tree_workspace_size - bytes of workspace pkv_tree_attention needs on the
 * CURRENT device for `batch` rows of n_nodes nodes (0 for invalid arguments).
 */
size_t pkv_tree_workspace_size(const pkv_cache_desc* cache, int batch, int n_nodes,
                               int num_q_heads);

/*
 * pkv_tree_attention - attention of a tree of drafted tokens per sequence over
 * the paged cache, on tcgen05 tensor cores.
 *
 * Row b is one sequence: slot c = batch_idx[b] holds ctx = ctx_lens[b]
 * committed tokens, and the K/V of its tree's nodes 0 .. tree_lens[b]-1 are in
 * the pools at positions ctx + 0, ctx + 1, ... (pkv_append first; whatever
 * position the rotary embedding used is the caller's affair). parents:
 * int32 [batch, n_nodes]; parents[b, i] in [-1, i) is the node that node i
 * follows, -1 for one that follows the context (any number of nodes may).
 * Node i attends the context, itself and its ancestors:
 *   T(i) = {0 .. ctx-1} + {ctx + a : a = i, parent(i), parent(parent(i)), ..}
 *   lse[b, i, h] = ln sum_{t in T(i)} exp(scale * q[b,i,h] . K[c,t,kvh])   (fp32)
 *   out[b, i, h] = sum_{t in T(i)} exp(scale * q[b,i,h] . K[c,t,kvh] - lse) V[c,t,kvh]
 * with kvh = h / (num_q_heads / num_kv_heads).
 * q: bf16 [batch, n_nodes, num_q_heads, D]; batch_idx, ctx_lens, tree_lens:
 * int32 [batch]; out: bf16 like q; lse: fp32 [batch, n_nodes, num_q_heads].
 * Nodes at or past tree_lens[b] (padding) and every node of a row with slot 0
 * give out 0, lse -inf. n_nodes is 1 .. PKV_MAX_TREE_NODES; ctx_lens[b] may be
 * 0. Scores, softmax sums and products are held in fp32; the weights exp(..) are
 * rounded to bf16 for the product with V, as in the decode and the prefills (their
 * sum takes them unrounded), and out is rounded once: each is off by at most 2^-8
 * of its value. A slot outside [0, max_batch) sets PKV_DEV_ERR_BAD_SLOT, a tree_lens[b]
 * outside [0, n_nodes] PKV_DEV_ERR_BAD_TREE, a negative ctx_lens[b] or
 * ctx + tree_lens[b] past the table PKV_DEV_ERR_BAD_POS: the row gives 0 /
 * -inf. A parent outside [-1, i) sets PKV_DEV_ERR_BAD_TREE; that node and
 * every node below it give 0 / -inf, the others are computed. An unreserved
 * page entry among a row's keys sets PKV_DEV_ERR_BAD_PAGE and leaves the row
 * unspecified. The pools are only read; slots past the last node may hold any
 * bits. The K/V of a row's own nodes and context must be finite: a NaN or
 * infinity in one node's V reaches the other nodes of its row.
 * page_size must be 16, 32, 64 or a multiple of 128; scale finite and > 0.
 * batch may be any count >= 0 (above 128 rows the call runs as equal launches
 * that share the workspace). workspace: at least pkv_tree_workspace_size()
 * bytes, 256-byte aligned, owned by the caller, no initialisation needed;
 * calls that share one must be stream-ordered. All tensors are device memory.
 */
pkv_status pkv_tree_attention(const pkv_cache_desc* cache, const void* k_pool,
                              const void* v_pool, const int32_t* page_table, const void* q,
                              int num_q_heads, const int32_t* parents,
                              const int32_t* tree_lens, const int32_t* batch_idx,
                              const int32_t* ctx_lens, int batch, int n_nodes, float scale,
                              void* out, float* lse, void* workspace, size_t workspace_bytes,
                              int32_t* dev_err, cudaStream_t stream);

/* Element types of probabilities. */
#define PKV_PROBS_FP32 0
#define PKV_PROBS_BF16 1

/*
 * pkv_verify_tree - acceptance of a tree of drafted tokens against the
 * target's probabilities, from given random numbers.
 *
 * target_probs: [batch, n_nodes, vocab]; row (b, i) is the target's
 * distribution of the token that follows node i. draft_probs: the same shape,
 * row (b, i) the distribution that node i's children were drawn from one after
 * another, or null: then every drafted token counts as drawn from a point mass
 * on it (guessed tokens). Both have the element type `probs_type`
 * (PKV_PROBS_*) and are 16-byte aligned; rows sum to 1 up to rounding; an entry
 * that is negative or NaN counts as 0. draft_tokens, parents: int32 [batch,
 * n_nodes]; tree_lens: int32 [batch]. Node 0 is the sequence's last token: it
 * is accepted as it stands and its draft_tokens entry is not read; node i >= 1
 * follows node parents[b, i] in [0, i).
 *
 * The walk starts at node 0. At node c its children x are tried in order of
 * their number. With p, q the rows of c, r = p and R = 1 to begin with:
 *   x is accepted iff u_accept[b, x] * q(tok x) * R < r(tok x)   (q(..) = 1 without
 *   draft_probs); the walk goes on at x.
 *   Otherwise r and R become those of the rest: with draft_probs
 *     r(v) = max(r(v) - R q(v), 0), R = sum_v r(v);
 *   without, R = max(R - r(tok x), 0), r(tok x) = 0.
 * Where no child is accepted the next token is drawn from r: the lowest v with
 * r(v) > 0 and sum_{w <= v} r(w) > u_sample[b] * sum_w r(w), or the highest v
 * with r(v) > 0 where rounding leaves none; from p where r has no mass. (The
 * accepted tokens and the next one are then distributed as the target's.)
 * Sums are held to about 2^-40 and decisions to 2^-45 of their terms, so that
 * they do not depend on an order of summation in fp32.
 *
 * path: int32 [batch, n_nodes], the accepted nodes (0 first), -1 behind them;
 * n_accepted: int32 [batch], their number (>= 1); tokens: int32 [batch,
 * n_nodes], the tokens of the accepted nodes after node 0, then the drawn one
 * (n_accepted in all), -1 behind them. tree_lens[b] = 0 (a padding row) gives
 * n_accepted 0 and -1 throughout. A tree_lens[b] outside [0, n_nodes] sets
 * PKV_DEV_ERR_BAD_TREE and is treated as 0; a parent outside [-1, i) or a
 * drafted token outside [0, vocab) sets it too and leaves that node and all
 * below it out (so does, without an error, a parent of -1 at i >= 1). A row
 * to draw from that sums to 0 or is not finite sets PKV_DEV_ERR_BAD_PROBS and
 * gives the token -1. n_nodes is 1 .. PKV_MAX_TREE_NODES. Results are the same
 * on every run.
 */
pkv_status pkv_verify_tree(const void* target_probs, const void* draft_probs, int probs_type,
                           int vocab, const int32_t* draft_tokens, const int32_t* parents,
                           const int32_t* tree_lens, const float* u_accept,
                           const float* u_sample, int batch, int n_nodes, int32_t* path,
                           int32_t* tokens, int32_t* n_accepted, int32_t* dev_err,
                           cudaStream_t stream);

/*
 * pkv_commit_path - moves the K/V rows of an accepted path next to the
 * committed context, in place.
 *
 * For row b with slot c = batch_idx[b], ctx = ctx_lens[b] and n =
 * n_accepted[b]: the rows at position ctx + path[b, i] of the slot go to
 * position ctx + i, for 0 <= i < n (bit-exact byte copies; each row is read
 * before anything overwrites it). path: int32 [batch, n_nodes] with
 * path[b, 0..n) strictly increasing in [0, n_nodes), as pkv_verify_tree
 * writes it. new_lens: int32 [batch] or null; new_lens[b] = ctx + n (it may be
 * ctx_lens itself; where several layers' calls share ctx_lens, in the last one's
 * only). Rows with slot 0 or n = 0 move nothing and give ctx. A
 * slot out of range sets PKV_DEV_ERR_BAD_SLOT, an n or a path that breaks the
 * above PKV_DEV_ERR_BAD_TREE, a position past the table PKV_DEV_ERR_BAD_POS, a
 * page entry out of range at a moved position PKV_DEV_ERR_BAD_PAGE: the row
 * moves nothing and gives ctx. A live slot must appear at most once, and no
 * page that a row writes may belong to another slot as well (reserve the
 * drafts' positions with pkv_update_pages).
 */
pkv_status pkv_commit_path(const pkv_cache_desc* cache, void* k_pool, void* v_pool,
                           const int32_t* page_table, const int32_t* path,
                           const int32_t* n_accepted, const int32_t* batch_idx,
                           const int32_t* ctx_lens, int batch, int n_nodes, int32_t* new_lens,
                           int32_t* dev_err, cudaStream_t stream);

/*
 * pkv_update_workspace_size - bytes of workspace pkv_update_pages needs for n
 * rows (0 for invalid arguments).
 */
size_t pkv_update_workspace_size(const pkv_cache_desc* cache, int n);

/*
 * pkv_update_pages - fork, reserve, copy on write, truncate and free.
 *
 * page_refs: int32 [num_pages], owned by the caller like the page table: how
 * many table entries (and holds of the caller's own) use each page. A page
 * with count 0 is free; page 0 is never handed out, whatever its count.
 * Row i gives slot d = dst_slots[i] the first keep = keep_lens[i] tokens of
 * slot s = src_slots[i] and makes positions keep .. new_lens[i]-1 writable:
 *   s == d, new > keep : room for the next tokens (reserve)
 *   s == d, new = keep : truncation; keep = 0 frees the slot
 *   s != d             : fork: whole pages are shared, counted once more
 *   s = 0, keep = 0    : a new sequence
 * A block that holds one of the positions [keep, new) gets a page that is the
 * slot's alone: the one it has when s == d and its count is 1, else a free
 * page, into which the rows before `keep` of a partly kept block are copied
 * (K and V, byte for byte). The slot's other entries up to new are the
 * source's, those past new are -1; every entry that the slot gives up counts
 * its page down. Writing only such positions, no sequence ever changes
 * another's tokens.
 *
 * Counts are those at the start of the call: two slots that share a partly
 * filled page and both reserve in one call both get a copy, and a page that
 * one row gives up is free from the next call on. Free pages are handed out
 * lowest number first, in row order and block order within a row, so the
 * result does not depend on timing.
 * A row with d = 0 is padding and does nothing. A row that cannot be served
 * changes nothing, sets its bit, and the others go on: PKV_DEV_ERR_BAD_SLOT (a
 * slot outside [0, max_batch); s = 0 with keep > 0; a destination that an
 * earlier row has; a source, with keep > 0, that is another row's destination),
 * PKV_DEV_ERR_BAD_POS (keep < 0, new < keep, new past the table),
 * PKV_DEV_ERR_BAD_PAGE (a kept block without a page in [1, num_pages), or a
 * page in use with a count below 1), PKV_DEV_ERR_NO_PAGES (a row that needs
 * pages where the needs of the rows up to it exceed the free ones). Entries of
 * the destination outside [1, num_pages) count as unreserved.
 * page_size x num_kv_heads must be below 2^25. page_table, page_refs, k_pool and
 * v_pool are updated in place.
 *
 * One call serves one pool pair, and its copies follow from the table and counts
 * that it finds. A second layer's call on the updated state would find the pages
 * handed out already and leave its own rows behind, without an error. So every
 * layer's call takes the state as it was before the first one's: layers with a
 * table and counts each have that; where layers share them, all calls but the last
 * are made on copies (device to device, before the first call; the result depends
 * on the state alone, so every copy ends as the shared state does, and can be
 * dropped).
 *
 * workspace: at least pkv_update_workspace_size()
 * bytes, 256-byte aligned, no initialisation needed; calls that share one must
 * be stream-ordered.
 */
pkv_status pkv_update_pages(const pkv_cache_desc* cache, void* k_pool, void* v_pool,
                            int32_t* page_table, int32_t* page_refs, const int32_t* dst_slots,
                            const int32_t* src_slots, const int32_t* keep_lens,
                            const int32_t* new_lens, int n, void* workspace,
                            size_t workspace_bytes, int32_t* dev_err, cudaStream_t stream);

/*
 * pkv_compact_workspace_size - bytes of workspace pkv_compact_pages needs
 * (0 for invalid arguments).
 */
size_t pkv_compact_workspace_size(const pkv_cache_desc* cache);

/*
 * pkv_compact_pages - moves the live pages to the low end of the pool.
 *
 * With L the number of live pages (count > 0; page 0 always is), the k-th live
 * page numbered L or more, in ascending order, moves to the k-th free page
 * below L: its K and V rows are copied, every entry of page_table that names
 * it is rewritten, and its count goes with it. Pages below L that are live
 * stay where they are; afterwards the live pages are 0 .. L-1. Pages that only
 * the caller's own holds keep alive move like the others, and nothing says where
 * to: a page that has to be found again belongs in a slot of the table. Several
 * layers that share a table and counts: as for pkv_update_pages, all calls but the
 * last on copies of the state before the first.
 * num_live: int32 [1] or null, receives L. page_refs as for pkv_update_pages, none
 * negative. An entry of page_table that names a free page at or past L sets
 * PKV_DEV_ERR_BAD_PAGE and is left as it is; entries outside [0, num_pages) are
 * left without an error, and so are those of free pages below L, which then name
 * what has moved there (pkv_update_pages leaves no such entries). workspace: at
 * least pkv_compact_workspace_size() bytes, 256-byte aligned, no initialisation
 * needed; calls that share one must be stream-ordered.
 */
pkv_status pkv_compact_pages(const pkv_cache_desc* cache, void* k_pool, void* v_pool,
                             int32_t* page_table, int32_t* page_refs, int32_t* num_live,
                             void* workspace, size_t workspace_bytes, int32_t* dev_err,
                             cudaStream_t stream);

/* Sizes of the pkv_latent_* calls: a cache row is a token's latent, then its
 * rotated part; expanded, a head's key is its own part, then the token's
 * rotated part. */
#define PKV_LATENT_DIM 512
#define PKV_LATENT_ROTATED 64
#define PKV_LATENT_ROW 576
#define PKV_LATENT_KEY 128
#define PKV_LATENT_VALUE 128

/*
 * pkv_rotate - the rotary position embedding of tokens' heads, in place or into
 * another tensor.
 *
 * x: bf16, the value d of head h of token i at x[i * x_token_stride + h *
 * x_head_stride + d], 0 <= d < dims; out likewise with its own strides (in
 * values, >= 0). So the rotated dims may be a part of a longer head: x points at
 * its first. dims is even; rope_cos, rope_sin: fp32 [rope_len, dims / 2]
 * row-major, the cosines and sines of position p in row p (whatever scaling for
 * long contexts they hold is the caller's). With j < dims / 2, c and s of
 * (positions[i], j), the pair (a, b) = (x_j, x_{j + dims/2}), or (x_{2j},
 * x_{2j+1}) with interleaved = 1, becomes
 *     (a c - b s, b c + a s)
 * computed in fp32 and rounded to nearest even once. out may be x itself with the
 * same strides; otherwise no value of out may lie on one of x that the call
 * reads. Values of out must not lie on one another: strides for which the inner
 * axis's rows do not end before the outer one's next are PKV_ERR_ARG (x may
 * repeat values: a stride of 0). The stride of an axis of length 1 is ignored. A
 * token whose position is outside [0, rope_len) is not written and sets
 * PKV_DEV_ERR_BAD_POS. Infinite values give what the formula gives. Pointers need 2-byte (x, out) and
 * 4-byte alignment; with 16-byte alignment of all four tensors, strides that are
 * multiples of 8 and dims of 16 (8 if interleaved) the call moves 16 bytes at a
 * time. n_tokens >= 0, num_heads >= 1.
 */
pkv_status pkv_rotate(const void* x, int64_t x_token_stride, int64_t x_head_stride, void* out,
                      int64_t out_token_stride, int64_t out_head_stride, int n_tokens,
                      int num_heads, int dims, int interleaved, const int32_t* positions,
                      const float* rope_cos, const float* rope_sin, int rope_len,
                      int32_t* dev_err, cudaStream_t stream);

/*
 * pkv_latent_append - new tokens' latents and position parts into the paged cache.
 *
 * The cache of a layer is one pool, bf16 [num_pages * page_size, 576] contiguous,
 * described by a pkv_cache_desc with num_kv_heads = 1, head_dim = 576; page table,
 * slots and positions are as for pkv_append. x_new: bf16, token i's 576 values at
 * x_new + i * x_token_stride (a multiple of 8, of one token too; >= 0): its latent l, then its position
 * part. With norm_weight (fp32 [512], 16-byte aligned) the latent becomes
 *     l_d * norm_weight[d] / sqrt(mean_d(l_d^2) + norm_eps)
 * (norm_eps finite and >= 0, else PKV_ERR_ARG; ignored without a weight), without
 * it is copied bit for bit. The position part is rotated as by pkv_rotate with
 * dims = 64 and tables [rope_len, 32], 16-byte aligned. Each value is rounded to bf16
 * once. Tokens of slot 0 are skipped; a bad slot, position (also one past
 * rope_len) or page entry skips the token and sets its bit. Two tokens that
 * address one row race.
 */
pkv_status pkv_latent_append(const pkv_cache_desc* cache, void* pool, const int32_t* page_table,
                             const void* x_new, int64_t x_token_stride,
                             const int32_t* batch_idx, const int32_t* input_pos, int n_tokens,
                             const float* rope_cos, const float* rope_sin, int rope_len,
                             int interleaved, const float* norm_weight, float norm_eps,
                             int32_t* dev_err, cudaStream_t stream);

/*
 * pkv_latent_gather - sequences' cached rows, one after another.
 *
 * Row starts[b] + t of out (bf16 [total, 576], contiguous, 16-byte aligned), for 0 <= t <
 * starts[b + 1] - starts[b], becomes the pool row of position t of slot slots[b]
 * (byte for byte). slots: int32 [n_seqs]; starts: int32 [n_seqs + 1], ascending
 * (equal neighbours: an empty sequence) from 0 or more to at most total, else
 * PKV_DEV_ERR_LAYOUT is set and what is written is unspecified (never outside
 * out). Rows before starts[0], from starts[n_seqs] on, and those of slot 0 stay as
 * they were. A bad slot, a position past the table or a bad page entry sets its
 * bit and leaves the row as it was.
 */
pkv_status pkv_latent_gather(const pkv_cache_desc* cache, const void* pool,
                             const int32_t* page_table, const int32_t* slots,
                             const int32_t* starts, int n_seqs, int total, void* out,
                             int32_t* dev_err, cudaStream_t stream);

/*
 * pkv_latent_decode_workspace_size - bytes of workspace pkv_latent_decode_attention
 * needs on the CURRENT device (0 for invalid arguments).
 */
size_t pkv_latent_decode_workspace_size(const pkv_cache_desc* cache, int batch, int n_q,
                                        int num_heads);

/*
 * pkv_latent_decode_attention - attention of new tokens over the cached rows (the
 * absorbed form: queries and results live in the latent's space), on tcgen05
 * tensor cores.
 *
 * q: bf16 [batch, n_q, num_heads, 576], contiguous: a head's query times its
 * up-projection of keys (512), then its rotated part (64). Row b's n_q tokens are
 * the last of the first n = seq_lens[b] positions of slot c = batch_idx[b] (their
 * own rows are in the pool: pkv_latent_append first); token j sees the rows
 * t < e = n - (n_q - 1 - j). With C[t] the row of position t:
 *   lse[b, j, h] = ln sum_{t<e} exp(scale * q[b,j,h] . C[t])                    (fp32)
 *   out[b, j, h] = sum_{t<e} exp(scale * q[b,j,h] . C[t] - lse) C[t][0:512]
 * out: bf16 [batch, n_q, num_heads, 512], 16-byte aligned; lse: fp32 [batch, n_q,
 * num_heads]. e <= 0, slot 0 and n = 0 give out 0, lse -inf. Scores, sums and
 * products are held in fp32; the weights exp(..) are rounded to bf16 for the product
 * (their sum takes them unrounded) and out is rounded once. A slot outside [0,
 * max_batch) sets PKV_DEV_ERR_BAD_SLOT, an n < 0 or past the table
 * PKV_DEV_ERR_BAD_POS: the row gives 0 / -inf. A page entry out of range within the
 * first n rows sets PKV_DEV_ERR_BAD_PAGE and leaves the row unspecified. The pool is
 * only read; rows past n may hold any bits. A query among whose scores there is a NaN
 * or +infinity gives NaN for out and lse, never 0 / -inf; one all of whose scores are
 * -infinity gives 0 / -inf. Of the tokens that do not see a row below n, lse is as
 * without it, but a NaN or infinity in its latent may reach their out in that dim.
 * n_q 1 .. 64; num_heads 1 .. 1024; the tiles of 128 keys that a slot can have, times
 * ceil(n_q * num_heads / 128), at most 2^30, else PKV_ERR_ARG (page tables of more than
 * 2^28 keys with the most query rows); batch any count >= 0 (above 512 rows the call runs
 * as equal launches that share the workspace); page_size any multiple of 16; scale
 * finite and > 0. workspace: at least pkv_latent_decode_workspace_size() bytes,
 * 256-byte aligned, owned by the caller, no initialisation needed; calls that
 * share one must be stream-ordered. All tensors are device memory. The
 * same inputs give the same bits on every run.
 */
pkv_status pkv_latent_decode_attention(const pkv_cache_desc* cache, const void* pool,
                                       const int32_t* page_table, const void* q, int num_heads,
                                       const int32_t* batch_idx, const int32_t* seq_lens,
                                       int batch, int n_q, float scale, void* out, float* lse,
                                       void* workspace, size_t workspace_bytes,
                                       int32_t* dev_err, cudaStream_t stream);

/*
 * pkv_latent_prefill_attention - causal attention of packed sequences in the
 * expanded form, on tcgen05 tensor cores: each head has its own keys and values,
 * up-projected from the latents, and all heads share a token's rotated part.
 *
 * Sequence s has the queries q_starts[s] .. q_starts[s+1]-1 and the keys k_starts[s]
 * .. k_starts[s+1]-1 (its cached prefix, as pkv_latent_gather returns it, then its
 * own tokens). With n queries and m keys, query i sees the keys t <= m - n + i:
 *   x[t] = scale (q[i,h][0:128] . k_own[t,h] + q[i,h][128:192] . k_rot[t])
 *   lse[i, h] = ln sum_t exp(x[t])   (fp32),
 *   out[i, h] = sum_t exp(x[t] - lse) v[t, h]
 * A query that sees no key gives out 0, lse -inf. q: bf16, 192 values a head; k_own,
 * v: bf16, 128 a head; k_rot: bf16, 64 a token; strides of tokens and heads in values,
 * multiples of 8, >= 0 and below 2^38 (so slices of wider rows and stride-0 heads do;
 * those of an axis of length 1 are ignored);
 * the four tensors 16-byte aligned. out: bf16 [n_queries, num_heads, 128], 32-byte
 * aligned; lse: fp32 [n_queries, num_heads]. q_starts, k_starts: int32 [n_seqs + 1], ascending
 * (equal neighbours: no queries, no keys) from 0 or more to at most n_queries and
 * n_keys, else PKV_DEV_ERR_LAYOUT is set and rows are unspecified (nothing is read or
 * written outside the tensors). Rows of out and lse outside all sequences stay as
 * they were. Scores, sums and products are held in fp32; the weights are rounded to
 * bf16 for the product (their sum takes them unrounded) and out is rounded once. A query
 * among whose scores there is a NaN or +infinity gives NaN for out and lse, never 0 / -inf;
 * one all of whose scores are -infinity gives 0 / -inf. A NaN or infinity in v may reach,
 * in its dim, out of any query of that sequence and head, also of those before the key; one
 * in k reaches only queries that see it. Other sequences are never reached. num_heads 1 .. 65535; scale finite and > 0. A sequence has at most
 * 2^26 keys (with more, an item of work may pass the kernel's limit on waits, which sets
 * PKV_DEV_ERR_TIMEOUT and leaves rows unspecified). The same inputs give the same bits on
 * every run.
 */
pkv_status pkv_latent_prefill_attention(
    const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k_own,
    int64_t k_token_stride, int64_t k_head_stride, const void* k_rot, int64_t r_token_stride,
    const void* v, int64_t v_token_stride, int64_t v_head_stride, int num_heads,
    const int32_t* q_starts, const int32_t* k_starts, int n_seqs, int n_queries, int n_keys,
    float scale, void* out, float* lse, int32_t* dev_err, cudaStream_t stream);

/* Static, human-readable name of a status. */
const char* pkv_status_string(pkv_status status);

/* Text of the CUDA runtime error behind the calling thread's most recent
 * PKV_ERR_CUDA (static storage; "no error" if there was none). */
const char* pkv_last_cuda_error_string(void);

/* Maps a dev_err word read back by the caller to a status: PKV_OK when 0,
 * PKV_ERR_BAD_PAGE when the bad-page bit is set, PKV_ERR_BAD_INPUT else. */
pkv_status pkv_status_from_device_error(int32_t dev_err_value);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H */
