/*
 * llama_block.h — C ABI of the GB300 (sm_103a) Llama-3-style decoder block library.
 *
 * One pre-norm decoder block, forward pass only, in causal prefill and in
 * KV-cached decode:
 *
 *     h = x + Attn(RMSNorm_1(x))          y = h + SwiGLU_FFN(RMSNorm_2(h))
 *
 * as defined by "Llama 3.1 70B" (ainfra.dev LLM architecture diagram:
 * Transformer layer, RMSNorm, Grouped-Query Attention, Residual add, SwiGLU
 * MLP), "How Llama 3.1 Generates the Next Token" (The transformer blocks,
 * What's RMSNorm?, What's the SWIGLU block?, RoPE) and "Llama 3 8B · Prepare
 * Q, K, V" (decode mode: Q/K/V projections, RoPE, K and V cached at KV-head
 * size).
 *
 * Conventions shared by every entry point
 *   - All pointers to tensors are DEVICE pointers owned by the caller; the
 *     library never frees them.  Weights are borrowed by the handle and must
 *     outlive it.  Nothing is copied.
 *   - Matrices are row-major [out, in] (torch.nn.Linear's storage: y = x W^T).
 *   - Activations are row-major [B, T, d_model].  The KV cache is two
 *     buffers K, V of shape [batch, n_kv_heads, max_seq, head_dim].
 *   - Element type is bf16 (LLAMA_BF16) or fp32 (LLAMA_F32) throughout one
 *     handle; token ids are int32.
 *   - Device pointers must be 16-byte aligned; every row length in bytes must
 *     be a multiple of 16.
 *   - Work is enqueued on the caller's stream (a cudaStream_t passed as
 *     void*; NULL = legacy default stream).  No host synchronisation, no
 *     device allocation and no device-wide barrier happens inside
 *     prefill/decode, so they may be captured into a CUDA graph.
 *   - Every function returns LLAMA_OK (0) or a negative LLAMA_ERR_* code;
 *     nothing throws across the ABI.  llama_block_last_error() returns a
 *     message for the last failure on that handle.
 */
#ifndef LLAMA_BLOCK_H_
#define LLAMA_BLOCK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LLAMA_OK 0
#define LLAMA_ERR_INVALID_ARG (-1)      /* null / misaligned pointer, bad size */
#define LLAMA_ERR_UNSUPPORTED_DIMS (-2) /* dims outside what the kernels implement */
#define LLAMA_ERR_POS_RANGE (-3)        /* position outside [0, max_seq) */
#define LLAMA_ERR_WORKSPACE (-4)        /* workspace missing or too small */
#define LLAMA_ERR_CUDA (-5)             /* a CUDA runtime call failed */
#define LLAMA_ERR_DEVICE_TIMEOUT (-6)   /* a bounded device-side wait expired */
#define LLAMA_ERR_NO_PAGES (-7)         /* the page pool holds too few (or no room for the) pages */

typedef enum { LLAMA_F32 = 0, LLAMA_BF16 = 1 } llama_dtype;

/* Block shape.  n_heads query heads share n_kv_heads K/V heads in groups of
 * n_heads / n_kv_heads ("Llama 3.1 70B", Grouped-Query Attention).  eps sits
 * inside the square root of RMSNorm; rope_theta is the RoPE base (omega_i =
 * theta^(-2i/head_dim), "How Llama 3.1 Generates the Next Token", Why use
 * different rotation speeds?).  max_seq bounds positions and sizes the
 * cos/sin table built at create.
 * bf16 handles need head_dim == 128 and d_model, d_ff multiples of 128;
 * fp32 handles accept head_dim in {32, 64, 128} and d_model, d_ff multiples
 * of 4. */
typedef struct {
    int32_t d_model, n_heads, n_kv_heads, head_dim, d_ff, max_seq;
    float eps, rope_theta;
    int32_t dtype; /* llama_dtype */
} llama_block_dims;

/* Device pointers, element type = dims.dtype.
 *   g_attn, g_ffn   [d_model]                 RMSNorm gains
 *   wq              [n_heads*head_dim, d]     wk, wv [n_kv_heads*head_dim, d]
 *   wo              [d, n_heads*head_dim]
 *   w_gate, w_up    [d_ff, d]                 w_down [d, d_ff]
 * ("How Llama 3.1 Generates the Next Token", Weight dimensions, transposed to
 * [out, in] as in "Llama 3 8B · Prepare Q, K, V", layers.py excerpt.) */
typedef struct {
    const void *g_attn, *wq, *wk, *wv, *wo, *g_ffn, *w_gate, *w_up, *w_down;
} llama_block_weights;

/* K and V rows are stored after RoPE (K) at KV-head size ("Llama 3 8B ·
 * Prepare Q, K, V", Explanation).  batch and max_seq describe the buffers;
 * max_seq may differ from the handle's but positions must fit both. */
typedef struct {
    void *k, *v;
    int32_t batch, max_seq;
} llama_kv_cache;

typedef struct llama_block_s* llama_block;

/* Validate dims, borrow weight pointers, build the TMA descriptors over the
 * weights and upload the fp32 cos/sin table [max_seq, head_dim/2] (computed
 * in fp64 on the host).  This is the only call that allocates device memory
 * (the table and a 4-byte error word).  On success *out holds the handle. */
int llama_block_create(const llama_block_dims* dims, const llama_block_weights* w, llama_block* out);

/* Llama 3.1's long-context RoPE schedule ("How Llama 3.1 Generates the Next
 * Token", Why use different rotation speeds?: the fastest rotations unchanged,
 * the slowest slowed by a factor, a middle range blended; "Llama 3.1 70B",
 * highlights: llama3 x8).  Pair i turns omega_i = rope_theta^(-2i/head_dim)
 * radians per position in the base schedule; with wavelength 2 pi / omega_i:
 *   wavelength < original_max_pos / high_freq_factor  ->  omega_i (unchanged)
 *   wavelength > original_max_pos / low_freq_factor   ->  omega_i / factor
 *   otherwise  (1 - s) omega_i / factor + s omega_i,
 *              s = (original_max_pos / wavelength - low_freq_factor)
 *                  / (high_freq_factor - low_freq_factor).
 * The pages give the factor (8) but not the band edges; Llama 3.1's released
 * configuration is factor 8, low 1, high 4, original_max_pos 8192.  Requires
 * factor >= 1, 0 < low_freq_factor < high_freq_factor, original_max_pos > 0. */
typedef struct {
    float factor, low_freq_factor, high_freq_factor;
    int32_t original_max_pos;
} llama_rope_scaling;

/* llama_block_create with the long-context RoPE schedule above in the handle's
 * cos/sin table (scaling = NULL: the base schedule, same as
 * llama_block_create).  Only the table differs; every call on the handle then
 * rotates q and k with the scaled angles.  LLAMA_ERR_INVALID_ARG for scaling
 * values outside the ranges above. */
int llama_block_create_scaled(const llama_block_dims* dims, const llama_block_weights* w,
                              const llama_rope_scaling* scaling, llama_block* out);

/* Free the handle's table, error word and host state.  NULL is a no-op. */
void llama_block_destroy(llama_block blk);

/* Bytes of device workspace that prefill (tokens = T) or decode (tokens = 1)
 * needs for batch B.  Returns 0 for invalid arguments. */
size_t llama_block_workspace_bytes(llama_block blk, int batch, int tokens);

/* Where a call's intermediates sit in its workspace, for inspection after the
 * call (stage-by-stage checks, callers that reuse a stage's output).  For a
 * call with this batch and tokens (tokens = 1: decode), offsets[i] receives the
 * byte offset from the workspace start of
 *   [0] xn  = RMSNorm_1(x)                    [batch*tokens, d_model]
 *   [1] q   after RoPE                        [batch*tokens, n_heads*head_dim]
 *   [2] o   attention output, heads merged    [batch*tokens, n_heads*head_dim]
 *   [3] h   = x + o Wo^T                      [batch*tokens, d_model]
 *   [4] hn  = RMSNorm_2(h)                    [batch*tokens, d_model]
 *   [5] u   = SiLU(hn W_gate^T) * (hn W_up^T) [batch*tokens, d_ff]
 * row-major, element type dims.dtype ("Llama 3.1 70B", Transformer layer: the
 * steps of the block in order).  n must be at least LLAMA_BLOCK_INTERMEDIATES.
 * Returns LLAMA_BLOCK_INTERMEDIATES, or LLAMA_ERR_INVALID_ARG. */
#define LLAMA_BLOCK_INTERMEDIATES 6
int llama_block_workspace_offsets(llama_block blk, int batch, int tokens, size_t* offsets, int n);

/* Causal prefill of T tokens per sequence at positions 0..T-1.
 *   x  [batch, T, d]   input residual stream
 *   y  [batch, T, d]   output; may alias x
 *   kv cache rows 0..T-1 of sequences 0..batch-1 are overwritten with the
 *      rotated keys and the values.
 * Attention follows "Llama 3.1 70B", Grouped-Query Attention (scaled dot
 * product, causal, 1/sqrt(head_dim)); the query at position p sees keys 0..p. */
int llama_block_prefill(llama_block blk, const void* x, int batch, int tokens, const llama_kv_cache* kv, void* y,
                        void* workspace, size_t workspace_bytes, void* stream);

/* Prefill of `tokens` new tokens per sequence at positions start_pos ..
 * start_pos + tokens - 1 on a cache that already holds the earlier tokens
 * (prefill in chunks).  kv rows 0 .. start_pos - 1 must hold their keys and
 * values; rows start_pos .. start_pos + tokens - 1 are written; the query at
 * position p sees keys 0..p.  llama_block_prefill is this call with
 * start_pos = 0.  Each row equals, bit for bit, the same row of one prefill of
 * all start_pos + tokens tokens.  start_pos + tokens must not exceed max_seq
 * (LLAMA_ERR_POS_RANGE otherwise). */
int llama_block_prefill_at(llama_block blk, const void* x, int batch, int tokens, int start_pos,
                           const llama_kv_cache* kv, void* y, void* workspace, size_t workspace_bytes, void* stream);

/* One decode step at position pos for every sequence of the batch.
 *   x [batch, 1, d] in, y [batch, 1, d] out (may alias x).
 *   kv rows 0..pos-1 must hold the cached keys/values; row pos is written;
 *   attention reads keys 0..pos (L = pos + 1, "Llama 3 8B · Prepare Q, K, V",
 *   decode mode) and nothing beyond.
 * The result for position pos is bit-identical to row pos of a prefill of
 * the same tokens (both paths share one reduction schedule). */
int llama_block_decode(llama_block blk, const void* x, int batch, const llama_kv_cache* kv, int pos, void* y,
                       void* workspace, size_t workspace_bytes, void* stream);

/* Same as llama_block_decode with the position read on the device from
 * *pos_dev (int32) when the kernels run, so one captured CUDA graph can be
 * replayed for successive positions.  The value must lie in [0, max_seq);
 * a value outside that range makes the kernels record LLAMA_ERR_POS_RANGE in
 * the handle's error word (read it with llama_block_poll_error); no cache row
 * is written and y is left undefined. */
int llama_block_decode_devpos(llama_block blk, const void* x, int batch, const llama_kv_cache* kv,
                              const int32_t* pos_dev, void* y, void* workspace, size_t workspace_bytes,
                              void* stream);

/* One decode step with a position per sequence: sequence b sits at position
 * pos_seq[b] (int32, device memory, read by the kernels when they run, so a
 * captured graph can be replayed as the positions move).  Sequence b reads its
 * cache rows 0..pos_seq[b] and writes row pos_seq[b]; its result equals, bit for
 * bit, what llama_block_decode at that position gives for it.  Each value must lie
 * in [0, max_seq): otherwise the kernels record LLAMA_ERR_POS_RANGE in the error
 * word, write no cache row and leave y undefined.  Supported for bf16 handles
 * with at most 8 query heads per KV head and batch <= 32; otherwise
 * LLAMA_ERR_UNSUPPORTED_DIMS. */
int llama_block_decode_seqpos(llama_block blk, const void* x, int batch, const llama_kv_cache* kv,
                              const int32_t* pos_seq, void* y, void* workspace, size_t workspace_bytes,
                              void* stream);

/* Synchronise `stream`, read and clear the handle's device error word.
 * Returns LLAMA_OK or the first code that a kernel recorded (LLAMA_ERR_POS_RANGE;
 * of paged steps also LLAMA_ERR_INVALID_ARG); LLAMA_ERR_DEVICE_TIMEOUT replaces
 * any other code. */
int llama_block_poll_error(llama_block blk, void* stream);

/* Per-CTA timeline of the block's kernels (RMSNorm, the projections, their
 * reductions, RoPE, attention and its combine), in the trace build of the
 * library (libllama_block_trace.so, the same sources compiled with
 * LLAMA_TRACE); the product library returns LLAMA_ERR_UNSUPPORTED_DIMS from
 * llama_trace_begin and carries no tracing code in its kernels.  Between
 * llama_trace_begin and llama_trace_end every CTA of those kernels claims one
 * record with an atomic
 * increment of *count and, while the index is below `capacity`, writes four
 * uint64 words at records[4 * index]:
 *   [0] kernel id (bits 0..7: 1 RMSNorm, 2 weight-streaming projection, 3
 *       token-tiled projection, 4..7 the QKV / residual / SwiGLU / residual +
 *       RMSNorm reductions, 8 decode attention, 9 its combine, 10 prefill
 *       attention, 11 RoPE, 12 wide-group decode attention; bits 8..11 the
 *       projection's epilogue: 0 QKV, 1 residual, 2 SwiGLU, 4 logits; bit 12
 *       a token-tiled projection whose K-segments run on separate CTAs),
 *       bits 16..31 the SM, bits 32..63 the CTA's linear index;
 *   [1] %globaltimer (ns) when the CTA started;
 *   [2] when its grid-dependency wait returned (0 if that CTA's recording
 *       thread does not wait);
 *   [3] when the CTA's thread 0 finished.
 * records (capacity x 32 bytes) and count (zeroed by the caller) are device
 * memory owned by the caller and must stay valid until llama_trace_end.  The
 * setting is process-wide and applies to kernels that run after the call
 * (graph replays included); with it on, each CTA reads it from the constant
 * bank at its start (a traced step runs about 3 us longer).  Returns LLAMA_OK,
 * LLAMA_ERR_INVALID_ARG, LLAMA_ERR_CUDA or (product build)
 * LLAMA_ERR_UNSUPPORTED_DIMS. */
int llama_trace_begin(unsigned long long* records, unsigned int* count, unsigned int capacity);
int llama_trace_end(void);

/* Failure-path self-test.  Launches on `stream` one warp that waits, through the
 * same bounded mbarrier wait every tensor-core kernel of the library uses, on a
 * barrier nothing arrives on.  After budget_ns nanoseconds (0 or more than 2 s:
 * the kernels' own 2 s budget) the wait gives up, records
 * LLAMA_ERR_DEVICE_TIMEOUT in the handle's error word and the kernel returns:
 * llama_block_poll_error then reports it, and the handle and the CUDA context stay
 * usable.  Returns LLAMA_OK once the launch is queued. */
int llama_block_selftest_wait_timeout(llama_block blk, unsigned long long budget_ns, void* stream);

/* Message of the last failure on this handle ("" if none).  Valid until the
 * next call on the handle. */
const char* llama_block_last_error(llama_block blk);

/* Stage timing.  events = NULL disables it; otherwise an array of 8 cudaEvent_t
 * (passed as void*) that every later prefill/decode on this handle records on
 * its stream: events[i] before stage i and events[7] after the last, for the
 * stages RMSNorm_1, QKV+RoPE+append, attention, O+residual, RMSNorm_2,
 * gate/up+SwiGLU, down+residual.  The array is borrowed until disabled. */
#define LLAMA_BLOCK_STAGES 7
int llama_block_set_stage_events(llama_block blk, void* const* events, int n_events);

/* Number of kernels the last successful prefill/decode call on this handle
 * enqueued (0 before the first call, after a failed call, or for NULL).  It
 * depends on the shape (the K-segment schedule fixed at create decides which
 * projections need a reduction kernel) and on the call (decode or prefill). */
int llama_block_launch_count(llama_block blk);

/* Device address of pinned host memory (cudaHostAlloc / cudaHostRegister; with
 * unified addressing every such allocation is mapped).  x and y of prefill and
 * decode may be given this way: the kernels then read x from and write y to host
 * memory directly (over NVLink-C2C on a Grace host), with no copy calls around
 * the block.  Only x and y take host memory: weights, the cache and the
 * workspace are read by TMA and must be device memory.  *dev = NULL and
 * LLAMA_ERR_INVALID_ARG if `host` is not pinned and mapped. */
int llama_device_ptr_of_host(const void* host, void** dev);

/* ---------------------------------------------------------------------------
 * Stack head (32-layer generation loop): embedding gather, final RMSNorm,
 * LM head with greedy choice.  bf16 only.
 * ------------------------------------------------------------------------- */

/* x[n, :] = w_embed[ids[n], :] for n < n_tokens ("Llama 3.1 70B", Token
 * embedding: a row gather, no positional term).  ids int32 in [0, vocab);
 * an id outside that range writes a zero row and records
 * LLAMA_ERR_INVALID_ARG in *err_dev (may be NULL). */
int llama_embed(const int32_t* ids, int n_tokens, const void* w_embed, int vocab, int d_model, void* x,
                int32_t* err_dev, void* stream);

/* ids[b] = argmax_v (RMSNorm_final(h[b]) . w_out[v]), fp32 logits, ties to the
 * lowest index ("How Llama 3.1 Generates the Next Token", Unembedding and
 * Sampling: greedy choice).  h [batch, d_model] (stride h_stride elements
 * between rows), g_final [d_model], w_out [vocab, d_model].  logits, if not
 * NULL, receives [batch, vocab] fp32.  workspace: llama_lmhead_workspace_bytes
 * (it also holds the call's device error word).  Every wait inside the kernels
 * is bounded; if one expires, ids[b] receives LLAMA_ERR_DEVICE_TIMEOUT (a
 * negative value, never a token id) for every row and the logits are undefined. */
size_t llama_lmhead_workspace_bytes(int batch, int d_model, int vocab);
int llama_lmhead_argmax(const void* h, int batch, int h_stride, const void* g_final, const void* w_out, int vocab,
                        int d_model, float eps, int32_t* ids, float* logits, void* workspace,
                        size_t workspace_bytes, void* stream);

/* Same result as llama_lmhead_argmax, for callers that cannot allocate device
 * memory (no workspace to pass: code running where cudaMalloc is not allowed or
 * must not happen on the hot path).  There is no counterpart on the pages; it is
 * a deployment variant.  The normalised rows live in a library-owned device
 * array of 32 x 8192 bf16 (512 KiB), held by every GPU that loads the library
 * until the process exits; batch > 32 or d_model > 8192 returns
 * LLAMA_ERR_WORKSPACE.  logits [batch, vocab] fp32 is required (it is an
 * output).  Nothing is allocated.  The first call on a device looks up the
 * array's device address (with that device current) and caches it: make that
 * first call before any stream capture.  Every call shares the one array, which
 * keeps the last call's rows; calls that overlap on the GPU (other streams,
 * other threads) race on it.  The cached address belongs to the device's
 * context: after cudaDeviceReset (or a reset of the primary context) the
 * library must be reloaded before this call is used again.  A device wait that
 * expires is reported as in llama_lmhead_argmax: ids[b] =
 * LLAMA_ERR_DEVICE_TIMEOUT (the error word is a second library-owned device
 * int, cleared by every call). */
int llama_lmhead_argmax_noalloc(const void* h, int batch, int h_stride, const void* g_final, const void* w_out,
                                int vocab, int d_model, float eps, int32_t* ids, float* logits, void* stream);

/* Next-token sampling from fp32 logits [batch, vocab] ("How Llama 3.1
 * Generates the Next Token", Temperature, Softmax, Top-k and top-p sampling):
 * divide by the temperature, softmax over the whole vocabulary, keep the top_k
 * most probable tokens and the smallest set of most probable tokens whose
 * probability reaches top_p (both restrictions: the smaller set), renormalise,
 * and draw: with the kept tokens in order of decreasing logit (equal logits by
 * increasing index), ids[b] is the first token whose cumulative renormalised
 * probability exceeds uniforms[b] (device fp32 in [0, 1), one per row, supplied
 * by the caller; values outside are clamped).  temperature = 0 or top_k = 1
 * gives the greedy choice (first maximum); top_k = 0 means no top-k limit and
 * top_p = 1 no top-p limit.  Weights e^{(z - max)/T} are computed in fp32 and
 * summed exactly in 2^-40 fixed point, top_p and the uniforms are taken to 24
 * bits: the result does not depend on thread scheduling.  Logits must be finite
 * (-inf allowed, weight zero).  Requires temperature >= 0, top_k >= 0,
 * 0 < top_p <= 1, 1 <= vocab <= 2^20, batch <= 65535; otherwise
 * LLAMA_ERR_INVALID_ARG.  No workspace, nothing allocated. */
int llama_sample(const float* logits, int batch, int vocab, float temperature, int top_k, float top_p,
                 const float* uniforms, int32_t* ids, void* stream);

/* Log probabilities of given tokens under fp32 logits [rows, vocab] ("How Llama 3.1
 * Generates the Next Token", Softmax), with the entropy and the top alternatives:
 *   logprobs[r] = logits[r][tokens[r]] - log sum_v e^(logits[r][v])
 *   entropy[r]  = - sum_v p_v log p_v (natural logarithm; a logit of -inf adds nothing)
 *   top_ids, top_logprobs [rows, n_top]: the n_top largest logits in decreasing order, equal
 *     ones by increasing token, and their log probabilities.
 * A row with tokens[r] < 0 takes no part: its logits are not read and its outputs are left
 * as they were; one with tokens[r] >= vocab too, and it is recorded (LLAMA_ERR_INVALID_ARG in
 * err_dev).  tokens may be NULL (every row takes part; logprobs is NULL too), entropy may be
 * NULL, n_top 0 (top_ids and top_logprobs are then not used).  Logits of -inf have
 * probability 0; a row of them alone has log probabilities of -inf, entropy 0 and the lowest
 * tokens on top.  A row with a NaN or +inf gets NaN log probabilities and entropy, and tokens
 * of its own vocabulary as alternatives.  Everything is held in fp32, the sums in a
 * tree over threads and without the largest term, so that small probabilities beside a large one keep
 * their digits.  0 <= n_top <= 32, n_top <= vocab <= 2^20. */
int llama_token_logprobs(const float* logits, int rows, int vocab, const int32_t* tokens, int n_top, float* logprobs,
                         float* entropy, int32_t* top_ids, float* top_logprobs, int32_t* err_dev, void* stream);

/* ---------------------------------------------------------------------------
 * Paged KV cache: serving ragged requests from one pool of pages.  The pages give
 * the cache's contents ("Llama 3 8B · Prepare Q, K, V", Explanation: K and V per
 * position at KV-head size) and no layout; paging is a deployment variant.
 *
 * Shared by the calls below: positions, lengths, tables, slots and counts are
 * int32 device arrays.  err_dev (device int32, may be NULL) receives the first
 * error that a kernel finds (LLAMA_ERR_DEVICE_TIMEOUT replaces any other); the
 * caller clears it.  All tensors live on the
 * current device.  Calls that read or write the same cache, table or pool must be
 * ordered by the caller (one stream, or events).
 * ------------------------------------------------------------------------- */

/* One layer's cache: k, v [n_pages, n_kv_heads, page_size, head_dim], page_size a
 * power of two in 16 .. 1024, n_pages * page_size * n_kv_heads < 2^31.  Position p
 * of a sequence lies in row p % page_size of page table[p / page_size] of its block
 * table row.  bf16 caches have head_dim 128, fp32 caches 32, 64 or 128. */
typedef struct {
    void *k, *v;
    int32_t n_pages, page_size;
} llama_paged_cache;

/* Block tables and slot maps of a batch of requests.  Request b holds positions
 * 0 .. start[b] - 1 and receives count[b] new ones (0 .. tokens):
 *   - it needs ceil((start + count) / page_size) pages and holds ceil(start /
 *     page_size); the difference is taken from the stack of free pages, requests
 *     in order and each request's pages in order, from the top entry
 *     free_pages[pool[0] - 1] downward, into the following entries of its row of
 *     table [batch, table_stride];
 *   - slots [batch, tokens] receives page * page_size + row of each new position
 *     start[b] + t, and -1 for t >= count[b].
 * pool is {number of free pages, any value}; pool_out receives {the new number, 0}
 * and may be pool (or two other words).
 * Entries of table that are not filled, and free_pages, are left as they are.  A
 * request with start < 0, count outside 0 .. tokens or more positions than its
 * table row holds gets no page and slots of -1 (LLAMA_ERR_POS_RANGE in err_dev);
 * with too few free pages for all requests nothing is taken and every slot is -1
 * (LLAMA_ERR_NO_PAGES); a page id outside [0, n_pages) gives slots of -1
 * (LLAMA_ERR_INVALID_ARG). */
int llama_paged_plan(const int32_t* start, const int32_t* count, int batch, int tokens, int page_size, int n_pages,
                     const int32_t* free_pages, const int32_t* pool, int32_t* pool_out, int32_t* table,
                     int table_stride, int32_t* slots, int32_t* err_dev, void* stream);

/* The inverse of llama_paged_plan with the same start and count: the pages that
 * it took go back on the stack, in the order that restores it exactly (free_pages
 * has n_pages entries).  start = 0 and count = the length gives back all pages of
 * a request.  Nothing is given back when the stack has no room for all of them
 * (LLAMA_ERR_NO_PAGES); a request out of range is left out (LLAMA_ERR_POS_RANGE).
 * Every page is released once: pages that the beams of a llama_beam_reorder share are
 * released through the row that planned them.  Pages that llama_paged_fork shared are
 * not released here (no count is read: other rows may still hold them) but given up
 * with llama_paged_free; the pages of such rows behind the shared ones may be released
 * (drafts that were rejected). */
int llama_paged_release(const int32_t* start, const int32_t* count, int batch, int page_size, int n_pages,
                        int32_t* free_pages, const int32_t* pool, int32_t* pool_out, const int32_t* table,
                        int table_stride, int32_t* err_dev, void* stream);

/* Rows of a contiguous cache k, v [batch, n_kv_heads, src_seq, head_dim] (as
 * llama_block_prefill leaves them) to their pages: row src_pos + t of sequence b
 * goes to slot slots[b][t], t < tokens.  A negative slot is skipped, a slot beyond
 * the cache is skipped and recorded (LLAMA_ERR_INVALID_ARG).  Slots must differ
 * from one another; rows that no slot names are left as they are. */
int llama_paged_store(const void* k, const void* v, int batch, int tokens, int src_seq, int src_pos,
                      const int32_t* slots, int n_kv_heads, int head_dim, int dtype, const llama_paged_cache* kv,
                      int32_t* err_dev, void* stream);

/* Attention of one new token per sequence over its pages: q, o [batch, n_heads,
 * head_dim]; sequence b attends its first lens[b] positions (the new token's among
 * them), query head h reads KV head h / (n_heads / n_kv_heads) ("Llama 3.1 70B",
 * Grouped-Query Attention; scores scaled by 1/sqrt(head_dim)).  lens[b] = 0 gives a
 * row of zeros.  max_len bounds the lengths (it sizes the workspace): a length
 * outside 0 .. max_len, or beyond the table row, is recorded (LLAMA_ERR_POS_RANGE)
 * and gives a row of zeros; a page id outside [0, n_pages) among the pages that a
 * sequence attends is recorded (LLAMA_ERR_INVALID_ARG) and leaves that sequence's
 * row undefined.  Cache rows and table entries behind the length are not used,
 * whatever they hold.  At most 64 query heads per KV head.  The result is, bit for
 * bit, the attention that llama_block_decode computes from the same rows: where that
 * runs on the tensor cores (bf16, groups that divide 128), softmax weights are rounded
 * to bf16 before their product with V and their sum (both held in fp32). */
size_t llama_paged_attention_workspace_bytes(int batch, int n_heads, int n_kv_heads, int head_dim, int max_len);
int llama_paged_attention(const void* q, int batch, int n_heads, int n_kv_heads, int head_dim, int dtype,
                          const llama_paged_cache* kv, const int32_t* table, int table_stride, const int32_t* lens,
                          int max_len, void* o, void* workspace, size_t workspace_bytes, int32_t* err_dev,
                          void* stream);

/* llama_block_decode_seqpos on a paged cache: sequence b at position pos_seq[b],
 * its rows found through row b of table [batch, table_stride]; the page of the
 * position must be in the table (llama_paged_plan).  Same result, bit for bit, as
 * on a contiguous cache.  For bf16 handles whose number of query heads per KV head
 * divides 128 (at most 64), and batch <= 32; otherwise LLAMA_ERR_UNSUPPORTED_DIMS.
 * A position outside [0, max_seq) or beyond the table row is recorded in the
 * handle's error word (LLAMA_ERR_POS_RANGE), and so is a page id outside
 * [0, n_pages) (LLAMA_ERR_INVALID_ARG): that sequence's cache row is not written
 * and its y is undefined.  Rows of table may share pages that no position of the
 * call is written to. */
int llama_block_decode_paged(llama_block blk, const void* x, int batch, const llama_paged_cache* kv,
                             const int32_t* table, int table_stride, const int32_t* pos_seq, void* y,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Attention of a chunk of new tokens per sequence over its pages: q, o [batch, tokens,
 * n_heads, head_dim].  Sequence b has count[b] new tokens (0 .. tokens) at positions
 * start[b] .. start[b] + count[b] - 1, the start and count of its llama_paged_plan; their
 * keys and values are in the cache already (llama_paged_store).  Token t attends
 * positions 0 .. start[b] + t; heads and scale as in llama_paged_attention.  Rows of o at
 * t >= count[b] are left as they were, and those of q are not used.  max_len bounds
 * start + count.  A sequence with start < 0, a count outside 0 .. tokens, or more positions
 * than max_len, its table row or 2^30 is recorded (LLAMA_ERR_POS_RANGE) and its rows are left
 * as they were; a page id outside [0, n_pages) among the pages that it attends is recorded
 * (LLAMA_ERR_INVALID_ARG) and leaves that sequence's rows undefined.  Cache rows and table
 * entries behind the last position are not used, and a token's row does not depend on the
 * keys and values behind its position, whatever they hold (infinities and NaN included).  A
 * row is NaN where no finite softmax exists.  bf16 (head_dim 128): products on the tensor
 * cores, weights rounded to bf16 before their product with V (held in fp32) and summed as
 * rounded, in fp32, so that keys of like values give that value whatever their weights'
 * roundings; fp32 (head_dim 32, 64, 128): fp32 throughout.  A row's sums are carried over to
 * second ones, in fp32, every few thousand keys (bf16: 65536), so that their roundings do not
 * grow with the cache.  At most 64 query heads per KV head, batch * tokens < 2^31, batch <=
 * 65535.  Where there are fewer query rows than the device has room for, the positions of a
 * row are split and joined: the split follows from the call's sizes, starts and counts, so
 * equal calls give equal bits, and a row's last bit may depend on the other sequences of the
 * call.  workspace: llama_paged_chunk_attention_workspace_bytes (0 for sizes that the call
 * refuses). */
size_t llama_paged_chunk_attention_workspace_bytes(int batch, int tokens, int n_heads, int n_kv_heads, int head_dim,
                                                   int max_len);
int llama_paged_chunk_attention(const void* q, int batch, int tokens, int n_heads, int n_kv_heads, int head_dim,
                                int dtype, const llama_paged_cache* kv, const int32_t* table, int table_stride,
                                const int32_t* start, const int32_t* count, int max_len, void* o, void* workspace,
                                size_t workspace_bytes, int32_t* err_dev, void* stream);

/* The block on a chunk of new tokens per sequence, on a paged cache: prompts in chunks, further turns of a
 * conversation, drafted tokens.  x, y [batch, tokens, d_model] (y may alias x); sequence b has count[b] new tokens
 * (0 .. tokens) at positions start[b] on, the start and count of its llama_paged_plan; positions 0 .. start[b] - 1 are in
 * the pages, those of the new tokens are written.  Cache rows have the bits that llama_block_prefill_at writes for the
 * same x; the attention is llama_paged_chunk_attention's, so y agrees with that call's to the attention's last
 * rounding, not bit for bit.  Rows of y at t >= count[b] are undefined.  bf16 handles; batch * tokens < 2^30.  A sequence
 * with start or count out of range, or positions beyond max_seq or its table row, is recorded in the handle's error word
 * (LLAMA_ERR_POS_RANGE), and so is a page id outside [0, n_pages) (LLAMA_ERR_INVALID_ARG): its rows of the cache are not
 * written (those of the bad page) and its rows of y are undefined.  workspace:
 * llama_block_prefill_paged_workspace_bytes (0 for invalid arguments). */
size_t llama_block_prefill_paged_workspace_bytes(llama_block blk, int batch, int tokens);
int llama_block_prefill_paged(llama_block blk, const void* x, int batch, int tokens, const llama_paged_cache* kv,
                              const int32_t* table, int table_stride, const int32_t* start, const int32_t* count,
                              void* y, void* workspace, size_t workspace_bytes, void* stream);

/* Samples of one prompt share its pages.  refs [n_pages] counts, for each page, the rows
 * that hold it beside the first: all zeros at first.  Only the two calls below read or
 * write it.  From a fork on, therefore, the full pages of its first lens[i] positions are,
 * in both of its rows,
 *   - given up with llama_paged_free alone: llama_paged_release would hand a page out
 *     again that other rows still read;
 *   - not written (a plan of either row starts behind them);
 *   - not in rows that go through llama_beam_reorder, which moves table entries and
 *     counts nothing.
 * No call can tell when this is broken.  All other pages of the rows are as before.
 *
 * Fork i (of n): row dst[i] of table [table_rows, table_stride] continues the first lens[i]
 * positions of row src[i], c = lens / page_size full pages and r = lens % page_size rows of
 * the page after them.  Entries 0 .. c-1 become those of the source row, and refs of each
 * of these pages grows by one; if r > 0, entry c becomes a page from the top of the stack
 * of free pages (in the order of the forks, as in llama_paged_plan) and receives rows
 * 0 .. r-1 of the source's page c in the caches of all n_layers (as in
 * llama_beam_reorder).  Other entries are left as they are.  pool and pool_out as in
 * llama_paged_plan.  A fork whose rows lie outside the table, whose dst is listed twice or is
 * also listed as a source is left out (LLAMA_ERR_INVALID_ARG in err_dev), one whose length
 * lies outside 0 .. table_stride * page_size too (LLAMA_ERR_POS_RANGE); with too few free
 * pages nothing is changed (LLAMA_ERR_NO_PAGES); an entry that is no page of the cache
 * is recorded (LLAMA_ERR_INVALID_ARG), passed on and nothing else is done with it.  n <= 65535,
 * table_rows <= 65536.  workspace: llama_paged_fork_workspace_bytes(n). */
size_t llama_paged_fork_workspace_bytes(int n);
int llama_paged_fork(const int32_t* src, const int32_t* dst, const int32_t* lens, int n, int32_t* refs,
                     const int32_t* free_pages, const int32_t* pool, int32_t* pool_out, int32_t* table, int table_rows,
                     int table_stride, const llama_paged_cache* caches, int n_layers, int n_kv_heads, int head_dim,
                     int dtype, void* workspace, size_t workspace_bytes, int32_t* err_dev, void* stream);

/* Rows rows[i] (of n) give up the pages of their first lens[i] positions: a page with
 * further holders (refs > 0) loses one of them, a page without goes back on the stack.
 * Several rows that hold a page may give it up in one call; it goes back at the last of
 * them in the order of rows and of pages within a row, and the pages that go back lie on
 * the stack in that order, the first on top: for rows without shared pages this is
 * llama_paged_release with start = 0 and count = lens.  Entries of table are left as
 * they are.  A row outside the table or listed twice is left out (LLAMA_ERR_INVALID_ARG),
 * one with a length outside 0 .. table_stride * page_size too (LLAMA_ERR_POS_RANGE); an
 * entry that is no page is recorded (LLAMA_ERR_INVALID_ARG) and skipped, and so is what a
 * page is given up more often than it is held; when the stack has no room for all pages
 * nothing is changed (LLAMA_ERR_NO_PAGES).  n * table_stride < 2^31, n <= 65536, table_rows <=
 * 65536.  workspace: llama_paged_free_workspace_bytes(n, n_pages). */
size_t llama_paged_free_workspace_bytes(int n, int n_pages);
int llama_paged_free(const int32_t* rows, const int32_t* lens, int n, int page_size, int n_pages, int32_t* refs,
                     int32_t* free_pages, const int32_t* pool, int32_t* pool_out, const int32_t* table, int table_rows,
                     int table_stride, void* workspace, size_t workspace_bytes, int32_t* err_dev, void* stream);

/* ---------------------------------------------------------------------------
 * Beam search ("How Llama 3.1 Generates the Next Token", Sampling, names greedy
 * choice and sampling; beam search keeps the best few continuations instead).
 * ------------------------------------------------------------------------- */

/* The n_out best continuations of each group's beams.  logits [groups * beams,
 * vocab] fp32, scores [groups * beams] the beams' cumulative log probabilities
 * (-inf: the beam takes no part).  Token v after beam k has the score
 *   scores[k] + logits[k][v] - log sum_u e^(logits[k][u]);
 * a beam with last[k] == eos has ended: its only continuation is eos, at scores[k]
 * (last may be NULL: no beam ends).  Outputs [groups, n_out] in decreasing score,
 * equal scores by increasing beam and then token: parents (row of the beam, in
 * 0 .. groups * beams - 1), tokens, out_scores.  With n_out == beams, out_scores may
 * be scores and tokens may be last.  Candidates are compared in fp64; each row's
 * log sum is within 2^-16 of the exact one (fp32 exponentials and sums) and the
 * same for equal rows of a call, so candidates of different beams may change places
 * where they are closer than 2^-15, a beam's own never do.
 * Logits must be finite or -inf (probability 0), scores too; continuations of score
 * -inf are listed only when the others are fewer than n_out.  1 <= beams <= 32,
 * 1 <= n_out <= 64, n_out <= vocab <= 2^20, groups * beams <= 65535; otherwise
 * LLAMA_ERR_INVALID_ARG. */
size_t llama_beam_select_workspace_bytes(int groups, int beams, int vocab, int n_out);
int llama_beam_select(const float* logits, int groups, int beams, int vocab, const float* scores,
                      const int32_t* last, int eos, int n_out, int32_t* parents, int32_t* tokens, float* out_scores,
                      void* workspace, size_t workspace_bytes, void* stream);

/* The beams' states follow the chosen parents, in place: row i of table [groups *
 * beams, table_stride] continues row parents[i] of the same group.  The beams of a
 * group have one length lens[i], i.e. c = lens / page_size full pages and r = lens %
 * page_size rows in the page after them.  Entries 0 .. c-1 of row i become those of
 * its parent (beams share full pages, which are not written again); if r > 0, rows
 * 0 .. r-1 of page table[i][c] become those of the parent's page, in the caches of
 * all n_layers (1 .. 128; distinct buffers of one n_pages and page_size).  Entries
 * from c on stay: they are the row's own pages.  No counts move: not for rows with pages
 * that llama_paged_fork shared.  A group whose parents lie outside
 * it, whose lengths differ or exceed the table, or whose rows share the page to be
 * filled is left as it was (LLAMA_ERR_INVALID_ARG in err_dev).  beams <= 32. */
int llama_beam_reorder(const int32_t* parents, int groups, int beams, const int32_t* lens, int32_t* table,
                       int table_stride, const llama_paged_cache* caches, int n_layers, int n_kv_heads, int head_dim,
                       int dtype, int32_t* err_dev, void* stream);

/* ---------------------------------------------------------------------------
 * Step-level entry points (the block's individual steps, for unit tests and
 * for callers that compose their own schedule).  Same conventions as above.
 * ------------------------------------------------------------------------- */

/* y = bf16(bf16(x * r) * g), r = 1/sqrt(mean(x^2) + eps) per row
 * ("Llama 3.1 70B", RMSNorm reference implementation).  rows x d. */
int llama_rmsnorm(const void* x, const void* g, void* y, int rows, int d, float eps, int dtype, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LLAMA_BLOCK_H_ */
