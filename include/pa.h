/*
 * pa.h -- C ABI of the paged-KV attention library (libpa.so), sm_103a.
 *
 * Three operations make up the path, in the order one model layer calls them
 * on a stream: pa_store_kvcache writes this step's new K/V rows into the
 * block pool, then pa_decode (one query token per sequence) or
 * pa_prefill_varlen (many query tokens per sequence, causal) reads K/V back
 * through the block tables.  Two helpers, pa_slot_mapping_decode and
 * pa_slot_mapping_prefill, build the slot_mapping the store consumes.
 *
 * Sources (web pages that define the operations):
 *   [NV12] "12. 推理加速(二):nano-vllm — 1200 行手写 vLLM" (chuoer47.github.io),
 *          §12.6 "Attention 层: Paged KV Cache", §12.7 "ModelRunner".
 *   [NV05] kyonqi.github.io "nano-vllm/05", ModelRunner: prepare_prefill,
 *          prepare_decode, prepare_block_tables, run_model.
 *   [VD]   "vLLM 深度解读" (luoboask.github.io), §3 "PagedAttention CUDA Kernel".
 *   [PA3]  "Nano-vLLM 源码解读 - 3. PagedAttention" (yeyulingfeng.com),
 *          §3 two-level mapping, §4 slot_mapping, §5 block size.
 *
 * Conventions shared by every entry point
 *   - Element type: bf16 for q, k, v, caches and outputs (passed as void*).
 *   - KV pool: one layer's k_cache and v_cache are each a contiguous
 *     [num_blocks, block_size, num_kv_heads, head_dim] array; slot s is the
 *     row k_cache + s*num_kv_heads*head_dim ([NV12 §12.7 allocate_kv_cache];
 *     [PA3 §3]).  The physical slot of logical position p of a sequence is
 *     block_table[p / block_size] * block_size + p % block_size.
 *   - block_tables: int32 [batch, max_blocks_per_seq], row-major; entries
 *     past a sequence's ceil(len/block_size) blocks are never read and may be
 *     -1 ([NV05 prepare_block_tables]).
 *   - head_dim must be 128 and num_q_heads a multiple of num_kv_heads with
 *     num_q_heads/num_kv_heads in {1, 2, 4, 8}; query head h reads kv head
 *     h / (num_q_heads/num_kv_heads).  Other shapes return PA_ERR_UNSUPPORTED.
 *   - block_size must be a positive multiple of 16 (256 is the tuned case).
 *   - Pointers are device pointers unless stated.  Base pointers of bf16
 *     arrays must be 16-byte aligned and row strides multiples of 8 elements.
 *   - Ownership: the caller owns every buffer and the stream.  No entry point
 *     allocates or frees device memory, and none synchronises the stream
 *     except pa_get_device_error.  Work is enqueued on `stream` in call order,
 *     so a store followed by an attention call on the same stream is ordered.
 *   - Errors: host-side argument checks return a status before anything is
 *     enqueued; pa_last_error_message() gives the detail (thread-local).  A
 *     launch failure returns PA_ERR_CUDA.  Problems only visible on the device
 *     (an out-of-range slot or block id, a context longer than its table, a
 *     wait that timed out) never fault: the kernel skips the access, records
 *     the first one in a device error word and carries on; read it with
 *     pa_get_device_error.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PA_API __attribute__((visibility("default")))
#else
#define PA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
struct CUstream_st;
typedef struct CUstream_st *pa_stream_t;

typedef enum {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misalignment, bad stride */
    PA_ERR_UNSUPPORTED = 2,   /* valid but not implemented (head_dim != 128, ...) */
    PA_ERR_WORKSPACE = 3,     /* workspace missing or smaller than required */
    PA_ERR_CUDA = 4,          /* a CUDA runtime/driver call or launch failed */
    PA_ERR_DEVICE_CHECK = 5   /* a kernel recorded a device-side error */
} pa_status;

/* Device-side error codes reported by pa_get_device_error. */
enum {
    PA_DEV_OK = 0,
    PA_DEV_TIMEOUT = 1,        /* a bounded wait gave up; where = kernel id */
    PA_DEV_BAD_SLOT = 2,       /* store: slot >= num_slots; where = token index */
    PA_DEV_BAD_CONTEXT = 3,    /* context length < 0 or > max_blocks_per_seq*block_size;
                                  where = sequence index */
    PA_DEV_BAD_BLOCK = 4,      /* checked mode: block id outside [0, num_blocks);
                                  where = sequence*max_blocks_per_seq + logical block */
    PA_DEV_BAD_SEQLENS = 5,    /* prefill: cu_seqlens not monotone or Lq > Lk;
                                  where = sequence index */
    PA_DEV_SMEM_ALIGN = 6,     /* a kernel could not align its shared-memory tiles
                                  (no work done); where = bytes of padding needed */
    PA_DEV_BAD_TEMPERATURE = 7, /* sampler, log probabilities: temperature not > 1e-10;
                                  where = row */
    PA_DEV_BAD_TOKEN = 8,      /* log probabilities: token >= vocab; where = row.
                                  verification: drafted token outside [0, vocab);
                                  where = sequence*num_nodes + node */
    PA_DEV_BAD_TREE = 9        /* drafts: a node's parent is not an earlier node, or a kept
                                  path does not ascend; where = sequence*num_nodes + node
                                  (place in the path) */
};

/* Scaling of rotary frequencies for long contexts (pa_rope_frequencies). */
enum {
    PA_ROPE_PLAIN = 0,
    PA_ROPE_LINEAR = 1,        /* positions divided by a factor */
    PA_ROPE_NTK = 2,           /* a larger base */
    PA_ROPE_YARN = 3           /* long wavelengths divided, short ones kept, a ramp between */
};

/* Code formats of an 8-bit KV pool (pa_store_kvcache_q8 and what reads it). */
enum {
    PA_Q8_E4M3 = 0,            /* OCP FP8 E4M3: 4 exponent and 3 mantissa bits */
    PA_Q8_INT8 = 1             /* two's-complement integers, -127..127 */
};

/* Library version (major*10000 + minor*100 + patch). */
PA_API int pa_version(void);

/* Static string for a status code. */
PA_API const char *pa_status_str(pa_status status);

/* Detail of the last non-OK status returned on the calling thread ("" if none). */
PA_API const char *pa_last_error_message(void);

/*
 * pa_store_kvcache -- scatter this step's K/V rows into the pool.
 * [NV12 §12.6 store_kvcache / store_kvcache_kernel; PA3 §4]
 *
 * For each token i in [0, num_tokens) with slot = slot_mapping[i] >= 0:
 *   k_cache[slot*Hkv*D + j] = key[i*key_row_stride + j]   for j < Hkv*D,
 * and the same for value -> v_cache.  Negative slots are padding (CUDA-graph
 * batches are padded with -1) and write nothing.  A slot >= num_slots is not
 * written and is recorded as PA_DEV_BAD_SLOT.
 *
 *   key, value           bf16 [num_tokens, *]: token i's Hkv*D values start at
 *                        key + i*key_row_stride (elements) and are contiguous
 *                        ([Hkv, D] row-major), so fused-QKV views are allowed.
 *   key_row_stride,
 *   value_row_stride     elements between tokens; >= Hkv*D, multiple of 8.
 *   k_cache, v_cache     bf16 pools [num_slots / block_size, block_size, Hkv, D].
 *   slot_mapping         int32 [num_tokens]; non-negative entries must be distinct.
 *   num_slots            num_blocks * block_size (bounds check only).
 * Copies are bit-exact.  num_tokens == 0 is a no-op.
 */
PA_API pa_status pa_store_kvcache(const void *key, int64_t key_row_stride, const void *value,
                           int64_t value_row_stride, void *k_cache, void *v_cache,
                           const int32_t *slot_mapping, int32_t num_tokens, int32_t num_kv_heads,
                           int32_t head_dim, int64_t num_slots, pa_stream_t stream);

/*
 * pa_slot_mapping_decode -- slot of each sequence's newest token.
 * [PA3 §4 "Decode 路径"; NV05 prepare_decode]
 *
 * slot_mapping[b] = block_tables[b][(ctx-1)/B]*B + (ctx-1)%B with
 * ctx = context_lens[b], i.e. last block * B + tokens in last block - 1;
 * context_lens[b] == 0 (a padded row) gives -1.
 *   slot_mapping   int32 [batch] (output, device).
 */
PA_API pa_status pa_slot_mapping_decode(int32_t *slot_mapping, const int32_t *block_tables,
                                 int32_t max_blocks_per_seq, const int32_t *context_lens,
                                 int32_t batch, int32_t block_size, pa_stream_t stream);

/*
 * pa_slot_mapping_prefill -- slots of the uncached suffix of every sequence.
 * [PA3 §4 "Prefill 路径"; NV12 §12.7 prepare_prefill]
 *
 * Sequence s computes positions [c, Lk) with Lk = cu_seqlens_k[s+1] -
 * cu_seqlens_k[s], Lq = cu_seqlens_q[s+1] - cu_seqlens_q[s], c = Lk - Lq (c
 * may sit mid-block: chunked prefill).  Query row cu_seqlens_q[s] + i gets
 * the slot of position c + i.
 *   slot_mapping   int32 [total_q] (output, device), total_q = cu_seqlens_q[num_seqs].
 */
PA_API pa_status pa_slot_mapping_prefill(int32_t *slot_mapping, const int32_t *block_tables,
                                  int32_t max_blocks_per_seq, const int32_t *cu_seqlens_q,
                                  const int32_t *cu_seqlens_k, int32_t num_seqs, int32_t total_q,
                                  int32_t block_size, pa_stream_t stream);

/*
 * pa_decode_workspace_size -- bytes of device workspace pa_decode needs.
 * It depends only on the GQA group (num_q_heads / num_kv_heads) and is at
 * most about 4.3 MB; 0 for shapes pa_decode does not support.
 */
PA_API size_t pa_decode_workspace_size(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim);

/*
 * pa_decode -- paged split-KV GQA decode attention, one query per sequence.
 * [NV12 §12.6 flash_attn_with_kvcache; VD §3 paged_attention_v1_kernel]
 *
 * For sequence b, query head h, kv head g = h / (Hq/Hkv), ctx = context_lens[b]:
 *   s_p = softmax_scale * <q[b,h,:], K[slot(b,p), g, :]>   for p < ctx,
 *   out[b,h,:] = sum_p softmax(s)_p * V[slot(b,p), g, :]    (bf16, RNE),
 * where slot(b,p) = block_tables[b][p/B]*B + p%B.  The query is the token at
 * position ctx-1 and sees all ctx keys, including its own (store it first).
 * ctx == 0 writes zeros and reads nothing.  The tiles of all (sequence, kv
 * head) pairs are cut into contiguous ranges (one per CTA, then small chunks
 * taken dynamically); a pair cut between ranges is combined in the same
 * kernel by the CTA that finishes its last part (log-sum-exp of the
 * online-softmax partials).  The kernel is launched as a programmatic
 * dependent launch and reads its inputs only after the preceding work on
 * the stream has completed.
 *
 *   out                bf16 [batch, Hq, D] contiguous.
 *   q                  bf16; row b (Hq*D contiguous values) at q + b*q_row_stride.
 *   k_cache, v_cache   the layer's pools (see conventions); num_blocks blocks.
 *   block_tables       int32 [batch, max_blocks_per_seq].
 *   context_lens       int32 [batch], each in [0, max_blocks_per_seq*block_size].
 *   softmax_scale      usually 1/sqrt(head_dim).
 *   workspace          device scratch of >= pa_decode_workspace_size(...)
 *                      bytes, 16-byte aligned, ZERO-FILLED before its first
 *                      use (fp32 split partials and work counters).  Every
 *                      call leaves it zero-filled again, so one memset at
 *                      allocation is enough; after a call that recorded a
 *                      device error, zero it again.  One workspace must not be
 *                      used by two calls that may run at the same time.
 * batch == 0 is a no-op; batch <= 2048.
 */
PA_API pa_status pa_decode(void *out, const void *q, int64_t q_row_stride, const void *k_cache,
                    const void *v_cache, const int32_t *block_tables, int32_t max_blocks_per_seq,
                    const int32_t *context_lens, int32_t batch, int32_t num_q_heads,
                    int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
                    float softmax_scale, void *workspace, size_t workspace_bytes,
                    pa_stream_t stream);

/*
 * pa_decode_store -- pa_decode that first stores the step's new token.
 * [NV12 §12.6: store_kvcache then attention, fused]
 *
 * For every sequence b with ctx = context_lens[b] > 0, the new token's K and
 * V rows (new_k[b], new_v[b]: Hkv*D bf16 each, row stride in elements) are
 * written to slot block_tables[b][(ctx-1)/B]*B + (ctx-1)%B of k_cache /
 * v_cache -- the token at position ctx-1, which the query is -- and the
 * attention then reads them like every other key.  The write is done inside
 * the decode kernel by the consumer warp that owns the token's key in the
 * sequence's last tile: it puts the row into that landed tile and into the
 * slot (one kv head's 256-byte row each), so the step needs neither a slot
 * mapping nor a separate store launch.  Afterwards the caches hold exactly what
 * pa_slot_mapping_decode + pa_store_kvcache would have written.  Other
 * arguments, the workspace contract and the outputs are those of pa_decode;
 * new_k / new_v 16-byte aligned.  The stored slots must be distinct, and none
 * may lie in the context of another row of the batch (rows that are one
 * sequence at lengths n and n+1, say): within the launch nothing orders one
 * row's store before another row's reads.  Use pa_store_kvcache and then
 * pa_decode there.
 */
PA_API pa_status pa_decode_store(void *out, const void *q, int64_t q_row_stride, const void *new_k,
                                 int64_t new_k_row_stride, const void *new_v, int64_t new_v_row_stride,
                                 void *k_cache, void *v_cache, const int32_t *block_tables,
                                 int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t batch,
                                 int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                 int32_t block_size, int32_t num_blocks, float softmax_scale, void *workspace,
                                 size_t workspace_bytes, pa_stream_t stream);

/*
 * pa_decode_shared_prefix -- pa_decode / pa_decode_store for batches in which
 * sequences share prefix-cache blocks.  [NV12 §12.8 BlockManager prefix
 * caching: sequences whose prompts begin with the same full blocks hold the
 * same physical blocks (ref_count > 1); NV12 §12.6 flash_attn_with_kvcache]
 *
 * Same result as pa_decode (new_k == new_v == NULL) or pa_decode_store (both
 * given, same layout and contract), within the attention tolerance: only the
 * summation order differs.  Sequences are grouped on the device by the id of
 * their first block; a group's shared prefix is the longest run of leading
 * block ids all its members agree on, limited for each member to the full
 * blocks before the one holding its newest token.  For groups of two or more
 * sequences a first kernel attends every member's query heads to the shared
 * prefix once per kv head (each of its K/V rows is read once, not once per
 * member) and leaves fp32 (m, l, o) partials in the workspace; the decode
 * kernel then streams only each member's own suffix and merges the prefix
 * partial into the member's result (log-sum-exp).  Batches without sharing
 * pay for the grouping pass and one extra launch; prefer pa_decode there.
 *
 *   workspace   >= pa_decode_shared_prefix_workspace_size(...) bytes (the
 *               pa_decode workspace plus the groups and the prefix partials
 *               of up to 8192 (member, q head) rows: ~8.6 MB more), same
 *               zero-filling contract as pa_decode.  Members beyond
 *               8192 / num_q_heads (in batch order) read the shared prefix
 *               themselves.
 *   batch       <= 1024.
 * Every other argument, the ordering and the error behaviour are those of
 * pa_decode / pa_decode_store.
 */
PA_API size_t pa_decode_shared_prefix_workspace_size(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim);
PA_API pa_status pa_decode_shared_prefix(void *out, const void *q, int64_t q_row_stride, const void *new_k,
                                         int64_t new_k_row_stride, const void *new_v, int64_t new_v_row_stride,
                                         void *k_cache, void *v_cache, const int32_t *block_tables,
                                         int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t batch,
                                         int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                         int32_t block_size, int32_t num_blocks, float softmax_scale, void *workspace,
                                         size_t workspace_bytes, pa_stream_t stream);

/*
 * pa_decode_static -- pa_decode for callers that cannot allocate device memory.
 * (An addition of this library: the source pages have no counterpart.)
 *
 * Same arguments and result as pa_decode, minus the workspace.  Some callers
 * cannot call cudaMalloc or an allocating library: code running inside
 * another framework's memory pool, plugins that must not touch the
 * allocator, or hosts that forbid device allocation after start-up.  This
 * entry point allocates nothing.  The split partials go to an 8 MiB scratch
 * array compiled into the library, which holds the workspace of every
 * supported shape (a shape needing more returns PA_ERR_UNSUPPORTED); every
 * GPU that loads the library holds those 8 MiB until the process exits.
 *   - The first call on a device (with that device current) looks up the
 *     array's device address; make that first call before any stream capture.
 *   - The partials need no initial value, but the work counters at the
 *     front of the array must be zero when the kernel starts.  Every call
 *     therefore clears them first (a cudaMemsetAsync of a few KiB on
 *     `stream`, which allocates nothing), so a call that stopped on a device
 *     error (PA_DEV_TIMEOUT) leaves nothing behind that a later call could
 *     trip on.
 *   - All calls share the one array and it keeps the last call's contents.
 *     Calls that may overlap on the GPU (other streams, other threads) race
 *     on it and must be serialised by the caller.
 */
PA_API pa_status pa_decode_static(void *out, const void *q, int64_t q_row_stride, const void *k_cache,
                                  const void *v_cache, const int32_t *block_tables,
                                  int32_t max_blocks_per_seq, const int32_t *context_lens, int32_t batch,
                                  int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                  int32_t block_size, int32_t num_blocks, float softmax_scale,
                                  pa_stream_t stream);

/*
 * pa_decode_static_scratch -- device address (on the current device) and size
 * in bytes of the scratch array pa_decode_static uses, for inspection and
 * tests.  Performs the same once-per-device look-up as pa_decode_static's
 * first call; allocates nothing.
 */
PA_API pa_status pa_decode_static_scratch(void **device_ptr, size_t *bytes);

/*
 * pa_prefill_varlen -- varlen causal attention for prompt (prefill) tokens.
 * [NV12 §12.6 flash_attn_varlen_func and its cu_seqlens example; NV05 prepare_prefill]
 *
 * Sequence s owns query rows [cu_seqlens_q[s], cu_seqlens_q[s+1]) (Lq rows)
 * and Lk = cu_seqlens_k[s+1] - cu_seqlens_k[s] >= Lq keys; the first
 * c = Lk - Lq keys were cached earlier (prefix-cache hits).  Query i sits at
 * position c + i and, with causal != 0, sees keys 0..c+i (bottom-right
 * alignment); with causal == 0 it sees all Lk keys.  Sequences never
 * interact.  Tensor cores (tcgen05, bf16 in, fp32 accumulate) compute
 * Q.K^T and P.V; the softmax runs in fp32 with P rounded to bf16.
 *   out            bf16 [total_q, Hq, D] contiguous.
 *   q              bf16; row t at q + t*q_row_stride, Hq*D contiguous values.
 *   total_q        rows of q (= cu_seqlens_q[num_seqs]); bounds the q reads.
 *   k, v           block_tables != NULL: the layer's caches (keys of sequence s
 *                  at slot(s, j)); the suffix must already be stored.
 *                  block_tables == NULL: contiguous rows, key j of sequence s
 *                  at k + (cu_seqlens_k[s] + j)*kv_row_stride, Hkv*D values.
 *   kv_row_stride  elements between rows in the contiguous case (ignored otherwise).
 *   total_k        rows of contiguous k/v (ignored when paged); bounds the reads.
 *   max_seqlen_q   an upper bound of Lq (sizes the grid); max_seqlen_k of Lk.
 *   num_blocks     pool size in blocks (paged case).
 */
PA_API pa_status pa_prefill_varlen(void *out, const void *q, int64_t q_row_stride, int32_t total_q,
                                   const void *k, const void *v, int64_t kv_row_stride, int32_t total_k,
                                   const int32_t *block_tables, int32_t max_blocks_per_seq,
                                   const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                   int32_t num_seqs, int32_t max_seqlen_q, int32_t max_seqlen_k,
                                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                   int32_t block_size, int32_t num_blocks, float softmax_scale,
                                   int32_t causal, pa_stream_t stream);

/*
 * pa_prefill_store_varlen -- pa_prefill_varlen (paged) that first stores the
 * uncached suffix.  [NV12 §12.6: store_kvcache then flash_attn_varlen_func,
 * fused; PA3 §4: the slot of position p is block_table[p/B]*B + p%B]
 *
 * new_k / new_v hold the suffix tokens' K and V rows in cu_seqlens_q order
 * ([total_q, Hkv, D] bf16, row strides in elements, multiples of 8, 16-byte
 * aligned): token t of sequence s sits at position (Lk - Lq) + (t -
 * cu_seqlens_q[s]), Lq / Lk its query / key lengths.  Each row is written to
 * that position's slot of k_cache / v_cache, exactly what
 * pa_slot_mapping_prefill + pa_store_kvcache would write (a block id outside
 * [0, num_blocks) is recorded as PA_DEV_BAD_SLOT with where = t, and that row
 * is not written); then the attention of pa_prefill_varlen runs over the
 * pool, with the same arguments and output.  block_tables is required.
 *
 * One launch: the CTAs copy the rows, meet at a grid barrier, then attend.
 * The launch is cooperative (its CTAs must be resident together, one per
 * SM); if the device cannot run it so, the call returns PA_ERR_CUDA.
 *
 * workspace: >= pa_prefill_store_workspace_size() bytes of device memory,
 * 8-byte aligned, zero-filled before first use; the call leaves it as it
 * found it, so it serves any number of calls on one stream (not concurrent
 * calls).  If the grid barrier gives up (PA_DEV_TIMEOUT, where = 440) no
 * attention runs in that CTA; zero the workspace again before the next call.
 */
PA_API size_t pa_prefill_store_workspace_size(void);
PA_API pa_status pa_prefill_store_varlen(void *out, const void *q, int64_t q_row_stride, int32_t total_q,
                                         const void *new_k, int64_t new_k_row_stride, const void *new_v,
                                         int64_t new_v_row_stride, void *k_cache, void *v_cache,
                                         const int32_t *block_tables, int32_t max_blocks_per_seq,
                                         const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                                         int32_t num_seqs, int32_t max_seqlen_q, int32_t max_seqlen_k,
                                         int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                         int32_t block_size, int32_t num_blocks, float softmax_scale,
                                         int32_t causal, void *workspace, size_t workspace_bytes,
                                         pa_stream_t stream);

/*
 * pa_sample_gumbel -- sample one token per row by the Gumbel-max trick.
 * [NV12 §12.2 "采样器": Sampler.forward and the Gumbel-max derivation]
 *
 *   token[b] = argmax_i softmax(float(logits[b]) / T_b)_i / max(E[b,i], 1e-10)
 *
 * computed in fp32; the lowest index wins among equal maxima.  E ~ Exp(1),
 * one independent draw per (row, vocabulary entry), is drawn by the caller
 * (e.g. torch.empty(...).exponential_(1)), which owns the random state.
 *   out_tokens        int32 [batch].
 *   logits            [batch, vocab] bf16 (logits_is_fp32 = 0) or fp32 (1);
 *                     row b at logits + b*logits_row_stride elements; the
 *                     stride is a multiple of 8 (bf16) or 4 (fp32) elements.
 *   temperatures      fp32 [batch], each > 1e-10; a row whose temperature is
 *                     not gets token -1 and PA_DEV_BAD_TEMPERATURE.
 *   exp_noise         fp32 [batch, vocab], row stride noise_row_stride (a
 *                     multiple of 4 elements).
 *   batch <= 65535.  A row with no finite candidate (all logits -inf or NaN)
 *   gets token 0.  Base pointers 16-byte aligned.  One kernel, a programmatic
 *   dependent launch; each row is read once (HBM-bound).
 */
PA_API pa_status pa_sample_gumbel(int32_t *out_tokens, const void *logits, int64_t logits_row_stride,
                                  int32_t logits_is_fp32, const float *temperatures, const float *exp_noise,
                                  int64_t noise_row_stride, int32_t batch, int32_t vocab, pa_stream_t stream);

/*
 * pa_logprobs -- log probabilities of given tokens, entropy, top alternatives:
 * what a server answers beside the tokens pa_sample_gumbel picks.  (An addition
 * of this library: the source pages stop at the token.)
 *
 * Per row, with z = float(logits) / T:
 *   logprobs[r]  = z_t - ln sum_i e^{z_i}   for t = tokens[r],
 *   entropy[r]   = -sum_i p_i ln p_i, p = softmax(z)   (0 ln 0 = 0),
 *   top_ids[r], top_logprobs[r]: the top_k largest logits in order (the lower
 *   index first among equals; NaN last) and their log probabilities.
 * All in fp32.  Logits of -inf have probability 0 and log probability -inf; a
 * row of nothing else has log probabilities -inf and entropy 0.  A NaN or
 * +inf logit makes its row's log probabilities and entropy NaN (top_ids still
 * follow the order).  A negative token (none given) has log probability -inf;
 * one >= vocab likewise, recorded as PA_DEV_BAD_TOKEN.
 *   logprobs, entropy      fp32 [rows].
 *   top_ids, top_logprobs  int32 / fp32 [rows, top_k]; unused for top_k == 0.
 *   logits                 [rows, vocab] bf16 (logits_is_fp32 = 0) or fp32 (1);
 *                          row stride in elements, >= vocab and a multiple of 8
 *                          (bf16) or 4 (fp32); 16-byte aligned.
 *   temperatures           fp32 [rows], each > 1e-10, or NULL (1).  Infinite
 *                          ones give equal probabilities to all logits but
 *                          -inf.  A row whose temperature is not > 1e-10 gets
 *                          NaN and ids -1 (PA_DEV_BAD_TEMPERATURE).
 *   tokens                 int32 [rows].
 *   top_k                  0..32, at most vocab; vocab at most 2^30.
 * The same call gives the same bits again; the order of a row's sums (so the
 * last bits) depends on rows and vocab.
 */
PA_API pa_status pa_logprobs(float *logprobs, float *entropy, int32_t *top_ids, float *top_logprobs,
                             const void *logits, int64_t logits_row_stride, int32_t logits_is_fp32,
                             const float *temperatures, const int32_t *tokens, int32_t rows, int32_t vocab,
                             int32_t top_k, pa_stream_t stream);

/* --------------------------------------------------------------------------
 * 8-bit KV pool.  (An addition of this library: the source pages keep the
 * pool in bf16.)  Decode is bound by the bytes of the cache; an 8-bit pool
 * halves them and doubles the tokens that fit.
 *
 * Layout (head-major, unlike the bf16 pool: the keys of one block and head are
 * contiguous, which 128-byte rows need to be streamed at full rate):
 *   k_cache, v_cache   1-byte codes [num_blocks, num_kv_heads, block_size, 128]
 *   k_scale, v_scale   1 byte       [num_blocks, num_kv_heads, block_size]
 * Slots, block tables and block_size are those of the bf16 pool: slot s is
 * token s % block_size of block s / block_size.
 *
 * A row (one token and head) stands for code * 2^(scale - 127), scale 0..254;
 * scale 255 marks a row that held a NaN or an infinity: it reads as NaN.  The
 * scale is the smallest power of two (at least 2^-126) with
 * max|x| <= 448 * 2^e (PA_Q8_E4M3) or 127 * 2^e (PA_Q8_INT8), and a code is
 * x * 2^-e rounded once, to nearest, ties to even, to a code whose value is
 * below 2^128 (bf16's last numbers would round up to it: finite rows read back
 * as finite numbers).  The result is a function of the row alone: it depends on
 * no other token, so appending a token never touches older ones.  An error of a
 * value is at most
 *   E4M3  the larger of 2^-4 of it and 2^-10 * 2^e (2^-4 of it from 2^-13 of the
 *         row's largest magnitude on, and anywhere in rows under 448 * 2^-126),
 *   INT8  1/126 of the row's largest magnitude (1/85 where that is the largest
 *         bf16 number; 2^-127 for rows under 127 * 2^-126).
 * Pointers 16-byte aligned; num_blocks * block_size * num_kv_heads < 2^31.
 * ------------------------------------------------------------------------ */

/*
 * pa_store_kvcache_q8 -- pa_store_kvcache into an 8-bit pool: each row is
 * quantised as it is written.  Arguments, padding (negative slots) and bad
 * slots (PA_DEV_BAD_SLOT) as there; non-negative slots must be distinct.
 *   format   PA_Q8_E4M3 or PA_Q8_INT8.
 */
PA_API pa_status pa_store_kvcache_q8(const void *key, int64_t key_row_stride, const void *value,
                                     int64_t value_row_stride, void *k_cache, void *v_cache, void *k_scale,
                                     void *v_scale, const int32_t *slot_mapping, int32_t num_tokens,
                                     int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                     int32_t num_blocks, int32_t format, pa_stream_t stream);

/*
 * pa_load_kvcache_q8 -- read rows of an 8-bit pool back as bf16, exactly.
 * Token i's rows are written to key + i*key_row_stride and value + i*
 * value_row_stride ([Hkv, 128] each, strides in elements, multiples of 8): the
 * rows of slot slot_mapping[i], zeros for a negative slot (and for a slot >=
 * num_blocks*block_size, recorded as PA_DEV_BAD_SLOT).  Slots may repeat.
 * With the slots of whole contexts (pa_slot_mapping_prefill with
 * cu_seqlens_q = cu_seqlens_k) the result is what pa_prefill_varlen takes as
 * contiguous k / v.
 */
PA_API pa_status pa_load_kvcache_q8(void *key, int64_t key_row_stride, void *value, int64_t value_row_stride,
                                    const void *k_cache, const void *v_cache, const void *k_scale,
                                    const void *v_scale, const int32_t *slot_mapping, int32_t num_tokens,
                                    int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                    int32_t num_blocks, int32_t format, pa_stream_t stream);

/*
 * pa_decode_q8 -- pa_decode over an 8-bit pool (one query token per sequence;
 * store its own key first).  Same definition, with K and V the values the
 * pool stands for; q and out bf16.  The scores use the codes exactly and q to
 * within 2^-39 of its head's largest element (elements from 2^-31 of it on are
 * exact), with fp32 accumulation; the softmax weights, each times its value
 * row's scale, are rounded to fp16.  A key or value row that reads as NaN makes its
 * sequence's outputs of that kv head NaN.
 *   workspace   device scratch of >= pa_decode_q8_workspace_size(...) bytes,
 *               16-byte aligned, ZERO-FILLED before its first use; contract as
 *               for pa_decode (every call leaves it ready for the next; zero it
 *               again after PA_DEV_TIMEOUT; not shared by calls that may run at
 *               the same time).  It serves pa_decode_q8 and
 *               pa_decode_store_q8 calls of any shape for which it is large
 *               enough, in turn, and no other entry point.
 * Other arguments and limits as pa_decode, and batch * num_kv_heads *
 * max_blocks_per_seq * block_size < 2^35.
 */
PA_API size_t pa_decode_q8_workspace_size(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim);
PA_API pa_status pa_decode_q8(void *out, const void *q, int64_t q_row_stride, const void *k_cache,
                              const void *v_cache, const void *k_scale, const void *v_scale,
                              const int32_t *block_tables, int32_t max_blocks_per_seq,
                              const int32_t *context_lens, int32_t batch, int32_t num_q_heads,
                              int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
                              int32_t format, float softmax_scale, void *workspace, size_t workspace_bytes,
                              pa_stream_t stream);

/*
 * pa_decode_store_q8 -- pa_decode_q8 that first stores the step's new token, as
 * pa_decode_store does for the bf16 pool: for every sequence with ctx =
 * context_lens[b] > 0 the rows new_k[b], new_v[b] ([Hkv, 128] bf16, row strides
 * in elements, multiples of 8; 16-byte aligned) are quantised into the slot of
 * position ctx-1 -- the same bytes pa_store_kvcache_q8 writes -- and attended to
 * like every other key, with the same outputs as that call followed by
 * pa_decode_q8, in one launch.  A block id outside [0, num_blocks) at that
 * position: the row is not stored and reads as zeros.  A context length out of
 * range (PA_DEV_BAD_CONTEXT): the row is not stored.  The stored slots must be
 * distinct, and none may lie in the context of another row of the batch: within
 * the launch nothing orders one row's store before another row's reads (rows
 * that are one sequence at lengths n and n+1, as when draft tokens are scored
 * together, need pa_store_kvcache_q8 and then pa_decode_q8).  Other arguments
 * and the workspace as pa_decode_q8.
 */
PA_API pa_status pa_decode_store_q8(void *out, const void *q, int64_t q_row_stride, const void *new_k,
                                    int64_t new_k_row_stride, const void *new_v, int64_t new_v_row_stride,
                                    void *k_cache, void *v_cache, void *k_scale, void *v_scale,
                                    const int32_t *block_tables, int32_t max_blocks_per_seq,
                                    const int32_t *context_lens, int32_t batch, int32_t num_q_heads,
                                    int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                    int32_t num_blocks, int32_t format, float softmax_scale, void *workspace,
                                    size_t workspace_bytes, pa_stream_t stream);

/* --------------------------------------------------------------------------
 * Speculative decoding over the pool.  (An addition of this library: the source
 * pages decode one token per sequence and step.)
 *
 * A step scores a small tree of drafted tokens per sequence in one pass of the
 * model: node 0 is the token that the drafts continue (the last one of the
 * sequence, whose K/V is not in the cache yet), node i > 0 a drafted token that
 * continues node parents[i] < i; a chain has parents[i] = i - 1.  At most 64
 * nodes.  The nodes' K/V rows take the positions that follow the context, in
 * the order of the nodes: context_lens[b] counts all keys, the n nodes of the
 * step the last of them (n = draft_lens[b], or num_drafts for every row with
 * context_lens[b] > 0 where draft_lens is NULL).  In the order of a step:
 *   pa_tree_metadata       masks, rotary positions and slots of the nodes
 *   pa_rope_store_kvcache  rotation of q and k, store of k and v   (per layer)
 *   pa_decode_tree         attention                               (per layer)
 *   pa_verify_drafts       which drafts the target keeps, and the next token
 *   pa_compact_kvcache     the kept nodes' rows moved next to the context
 * Nodes i >= n of a row are padding: no slot, zero outputs.
 * ------------------------------------------------------------------------ */

/*
 * pa_rope_frequencies -- rotary frequencies (host code; freqs and gain are host
 * pointers).  freqs[i], i < rotary_dim/2, are turns per position as fractions of
 * 2^64, rounded to the nearest, so that position * freqs[i] modulo 2^64 is the turn to
 * within 2^-34 at the farthest position: f_i = theta^(-2i/R) radians per position, and
 * with `factor` s:
 *   PA_ROPE_LINEAR  f_i / s
 *   PA_ROPE_NTK     theta * s^(R/(R-2)) in place of theta
 *   PA_ROPE_YARN    f_i (1 - r_i) + f_i / s * r_i, r_i = clamp((i - lo)/(hi - lo), 0, 1)
 *                   with lo, hi = floor, ceil of R ln(original_context / (2 pi beta))
 *                   / (2 ln theta) at beta_fast and beta_slow (usually 32 and 1),
 *                   clamped to [0, R-1]; *gain = 0.1 ln s + 1 (else 1)
 * rotary_dim: a multiple of 16 up to 128; theta > 1, factor >= 1.
 */
PA_API pa_status pa_rope_frequencies(uint64_t *freqs, float *gain, int32_t rotary_dim, double theta, int32_t scaling,
                                     double factor, double original_context, double beta_fast, double beta_slow);

/*
 * pa_rope -- per-head norm and rotation of q and k.  For each head x of 128 at
 * positions[t]: with a norm weight (q_norm / k_norm, bf16 [128], NULL: none)
 *   x <- x / sqrt(mean(x^2) + eps) * weight,
 * then the pairs (x[i], x[i + R/2]), or (x[2i], x[2i+1]) when interleaved, i < R/2,
 * R = rotary_dim, are rotated by positions[t] * f_i and multiplied by gain; the
 * values from R on are not rotated.  fp32 throughout, one rounding to bf16; the squares
 * too, so that a normed head holds values below 10^18, and above 10^-18 if eps is 0.
 *   out_q, out_k    bf16; token t's Hq*128 (Hkv*128) values at out + t*stride.
 *                   out_q may be q itself with its stride, out_k may be key.
 *   q, key          bf16, row strides in elements: >= a token's values, multiples
 *                   of 8 (fused-QKV views are allowed).
 *   positions       int32 [num_tokens].
 *   freqs           device copy of pa_rope_frequencies' [rotary_dim/2].
 * Pointers 16-byte aligned (freqs: 8).  num_tokens == 0 is a no-op.
 */
PA_API pa_status pa_rope(void *out_q, int64_t out_q_row_stride, void *out_k, int64_t out_k_row_stride, const void *q,
                         int64_t q_row_stride, const void *key, int64_t key_row_stride, const int32_t *positions,
                         const uint64_t *freqs, int32_t rotary_dim, int32_t interleaved, float gain,
                         const void *q_norm, const void *k_norm, float eps, int32_t num_tokens, int32_t num_q_heads,
                         int32_t num_kv_heads, int32_t head_dim, pa_stream_t stream);

/*
 * pa_rope_store_kvcache -- pa_rope, with the rotated keys and the values written
 * into the pool as pa_store_kvcache writes them: same slots, padding (negative
 * slots: neither K nor V is written, q is rotated all the same), bad slots
 * (PA_DEV_BAD_SLOT) and layout.  One launch; the caches hold exactly what pa_rope
 * and then pa_store_kvcache would have written.
 */
PA_API pa_status pa_rope_store_kvcache(void *out_q, int64_t out_q_row_stride, const void *q, int64_t q_row_stride,
                                       const void *key, int64_t key_row_stride, const void *value,
                                       int64_t value_row_stride, const int32_t *positions, const uint64_t *freqs,
                                       int32_t rotary_dim, int32_t interleaved, float gain, const void *q_norm,
                                       const void *k_norm, float eps, void *k_cache, void *v_cache,
                                       const int32_t *slot_mapping, int32_t num_tokens, int32_t num_q_heads,
                                       int32_t num_kv_heads, int32_t head_dim, int64_t num_slots, pa_stream_t stream);

/*
 * pa_tree_metadata -- what a step's kernels need of its trees.  For node i < n of
 * sequence b (outputs [batch, num_drafts]):
 *   tree_mask     bit j set where j is i or an ancestor of i
 *   positions     context_lens[b] - n + depth of i (the root's depth is 0)
 *   slot_mapping  slot of position context_lens[b] - n + i (-1 where the table
 *                 holds none, or one whose slots do not fit int32, recorded as
 *                 PA_DEV_BAD_BLOCK); padding: mask 0, position 0, slot -1
 * parents int32 [batch, num_drafts] (entry 0 of a row is not read), NULL: chains.
 * A parent that is not an earlier node ends the walk up (PA_DEV_BAD_TREE); lengths
 * that do not fit make the row padding (PA_DEV_BAD_CONTEXT).
 */
PA_API pa_status pa_tree_metadata(int64_t *tree_mask, int32_t *positions, int32_t *slot_mapping,
                                  const int32_t *parents, const int32_t *context_lens, const int32_t *draft_lens,
                                  const int32_t *block_tables, int32_t max_blocks_per_seq, int32_t batch,
                                  int32_t num_drafts, int32_t block_size, pa_stream_t stream);

/*
 * pa_decode_tree -- pa_decode for num_drafts query tokens per sequence, each with
 * its own set of the drafts' keys.  With n and ctx = context_lens[b] as above,
 * query i < n sees the keys at positions p < ctx - n, and that of draft j < n (at
 * position ctx - n + j) where bit j of tree_mask[b][i] is set; tree_mask NULL: the
 * drafts j <= i.  Any pattern is allowed; a query that sees nothing has output
 * zero.  num_drafts == 1 with bit 0 set is pa_decode.  What a mask hides does not
 * matter, NaN and infinities included.  The weights are rounded to bf16, and
 * normalised by the sum of the rounded ones.  The same call gives the same bits
 * again; a row's last bits depend on the batch, by which the keys are cut.
 *   out           bf16 [batch, num_drafts, Hq, 128] contiguous, overlaps no input;
 *                 zeros for i >= n.
 *   q             bf16; the Hq*128 values of (b, i) at q + (b*num_drafts + i)*q_row_stride.
 *   tree_mask     int64 [batch, num_drafts].
 *   draft_lens    int32 [batch] or NULL.  Lengths that do not fit (ctx < n among
 *                 them) are recorded as PA_DEV_BAD_CONTEXT and give zeros.
 *   workspace     >= pa_decode_tree_workspace_size(...) bytes, 32-byte aligned.  It
 *                 holds nothing between calls, and serves calls of any shape for
 *                 which it is large enough, one after the other.
 * num_drafts <= 64, batch <= 2048; other arguments and limits as pa_decode, and
 * batch * num_kv_heads * max_blocks_per_seq * block_size / 64 (twice that above 256
 * query heads times drafts per kv head) < 2^31.
 */
PA_API size_t pa_decode_tree_workspace_size(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                            int32_t num_drafts);
PA_API pa_status pa_decode_tree(void *out, const void *q, int64_t q_row_stride, const void *k_cache,
                                const void *v_cache, const int32_t *block_tables, int32_t max_blocks_per_seq,
                                const int32_t *context_lens, const int32_t *draft_lens, const int64_t *tree_mask,
                                int32_t batch, int32_t num_drafts, int32_t num_q_heads, int32_t num_kv_heads,
                                int32_t head_dim, int32_t block_size, int32_t num_blocks, float softmax_scale,
                                void *workspace, size_t workspace_bytes, pa_stream_t stream);

/*
 * pa_verify_drafts -- which drafted tokens the target model keeps, and the token
 * after them: speculative sampling from given random numbers.  Per sequence,
 * from node v = 0: p = softmax(float(logits[b][v]) / T_b), w = p, s = 1, and for
 * v's children in order, child c with token x:
 *   with draft_probs (q = draft_probs[b][v], the distribution that each of v's
 *   children was drawn from on its own):
 *     kept if uniforms[b][c] * q(x) * s < w(x), else w <- max(w - s q, 0), s <- sum w
 *   without (children are chosen candidates):
 *     kept if uniforms[b][c] * s < w(x), else s <- s - w(x), w(x) <- 0.
 * A kept child becomes v.  Where no child is kept, the sequence's next token is
 * argmax_i w_i / max(exp_noise[b][i], 1e-10), the lowest index among equals (with p
 * for w where nothing is left of w): tokens are distributed as the target's own.
 *   out_tokens   int32 [batch, num_nodes]: the kept tokens, then the next; -1 after.
 *   out_nodes    int32 [batch, num_nodes]: 0 and the kept nodes; -1 after.
 *   out_counts   int32 [batch]: entries of either.
 *   logits       bf16 or fp32, row (b*num_nodes + v); stride as pa_sample_gumbel.
 *   tokens       int32 [batch, num_nodes] (entry 0 of a row is not used).  One outside
 *                [0, vocab) is no child (PA_DEV_BAD_TOKEN).
 *   parents      int32 [batch, num_nodes] or NULL (chains).  A node whose parent is
 *                not an earlier node is no child (PA_DEV_BAD_TREE).
 *   uniforms     fp32 [batch, num_nodes] in [0, 1); exp_noise fp32 [batch, vocab], row
 *                stride a multiple of 4: the caller's random numbers.
 *   temperatures fp32 [batch], each > 1e-10; else count 0 (PA_DEV_BAD_TEMPERATURE).
 *   draft_probs  fp32, row (b*probs_rows + v), row stride a multiple of 4, or NULL;
 *                probs_rows >= num_nodes - 1 (the last node has no children).
 *   draft_lens   int32 [batch], nodes of each sequence (0: padding, count 0), or NULL.
 * NaN logits count as -inf, +inf as the largest number; a row of -inf alone keeps no
 * child and draws token 0, as pa_sample_gumbel does.  exp_noise holds no NaN (one
 * counts as 1e-10).  p, w and s are in fp32: a decision whose two sides differ by less
 * than 2^-14 of the larger (of p(x), where w is a difference) may go either way.
 * num_nodes <= 64, batch <= 65535, vocab <= 2^30; logits, exp_noise and draft_probs
 * 16-byte aligned.  A small temperature (1e-6) gives greedy verification.  The outputs
 * overlap no input.
 */
PA_API pa_status pa_verify_drafts(int32_t *out_tokens, int32_t *out_nodes, int32_t *out_counts, const void *logits,
                                  int64_t logits_row_stride, int32_t logits_is_fp32, const int32_t *tokens,
                                  const int32_t *parents, const float *uniforms, const float *exp_noise,
                                  int64_t noise_row_stride, const float *temperatures, const float *draft_probs,
                                  int64_t probs_row_stride, int32_t probs_rows, const int32_t *draft_lens,
                                  int32_t batch, int32_t num_nodes, int32_t vocab, pa_stream_t stream);

/*
 * pa_compact_kvcache -- after a verification: for j < counts[b] the K and V rows
 * of position base + nodes[b][j] are copied to position base + j, base =
 * context_lens[b] - n (n as above), in every layer, as if read before any is
 * written.  nodes / counts are pa_verify_drafts' out_nodes / out_counts: nodes[b][0]
 * = 0, ascending, below n; the first one that is not ends its row's moves
 * (PA_DEV_BAD_TREE).  The context is then base + counts[b] keys long.  Rows of other
 * positions stay as they are.  The rows from base on are the sequence's own: no other
 * sequence of the call holds their slots (a shared prefix lies before them).  A block
 * id outside [0, num_blocks): that row is not moved (PA_DEV_BAD_BLOCK).
 *   k_cache, v_cache  the first layer's pools; the next layer's follow
 *                     k_layer_stride / v_layer_stride elements on (multiples of 8).
 * Bit-exact.  num_nodes <= 64.
 */
PA_API pa_status pa_compact_kvcache(void *k_cache, int64_t k_layer_stride, void *v_cache, int64_t v_layer_stride,
                                    const int32_t *block_tables, int32_t max_blocks_per_seq,
                                    const int32_t *context_lens, const int32_t *draft_lens, const int32_t *nodes,
                                    const int32_t *counts, int32_t batch, int32_t num_nodes, int32_t num_layers,
                                    int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                    pa_stream_t stream);

/* --------------------------------------------------------------------------
 * Host block manager: the pool's allocator and prefix cache, whose block
 * tables the kernels above consume.  Host code only (no GPU, no CUDA calls).
 * [NV12 §12.8 "BlockManager: 分页 KV Cache + Prefix Caching";
 *  VS §1.1 (the four fields), §1.2.4 (a traced allocation), §1.2.5 (prefix hits)]
 *
 * State: num_blocks blocks of block_size tokens, each with a reference count,
 * the chained hash of its prefix (or none) and its token ids; a FIFO queue of
 * free block ids (taken from the front, returned to the back); the set of
 * used ids; a map from prefix hash to block id.  The chained hash of block i
 * of a sequence is XXH64 (seed 0) of [hash of block i-1 as 8 little-endian
 * bytes, omitted for i = 0] followed by the block's token ids as 64-bit
 * little-endian integers (pa_bm_block_hash).  Sequences are kept in the
 * manager and named by the id pa_bm_seq_add returns.
 *
 * pa_bm_can_allocate  number of leading full blocks (never the last block)
 *                     found in the prefix cache with identical tokens, or -1
 *                     if the free queue is shorter than the blocks still
 *                     needed (cached blocks in use need none); -2: bad args.
 * pa_bm_allocate      give the sequence its blocks: the first
 *                     num_cached_blocks from the cache (one more reference,
 *                     or taken back from the free queue), then fresh ones
 *                     from the front of the queue (a fresh block loses its
 *                     old map entry); num_cached_tokens = cached * block_size.
 * pa_bm_deallocate    drop one reference per block, last block first; blocks
 *                     at zero go to the back of the free queue keeping their
 *                     hash (so a later prefix hit can take them back).
 * pa_bm_can_append    1 if a decode step of the sequence can get the block it
 *                     needs (one exactly when len % block_size == 1), else 0.
 * pa_bm_may_append    take that block if needed.
 * pa_bm_hash_blocks   register the blocks filled by a step of
 *                     num_scheduled_tokens tokens after num_cached_tokens:
 *                     blocks [cached / B, (cached + scheduled) / B).  The
 *                     caller then advances num_cached_tokens
 *                     (pa_bm_seq_set_num_cached_tokens) and appends generated
 *                     tokens (pa_bm_seq_append_token).
 * pa_bm_block_tables  int32 [num_seqs, max_blocks_per_seq] block tables, -1
 *                     past each sequence's blocks (the kernels' format).
 * Queries return counts (or -2 for bad arguments); errors set
 * pa_last_error_message.  A manager is not thread-safe.
 */
typedef struct pa_block_manager pa_block_manager;
PA_API pa_status pa_bm_create(int32_t num_blocks, int32_t block_size, pa_block_manager **out);
PA_API void pa_bm_destroy(pa_block_manager *bm);
PA_API pa_status pa_bm_seq_add(pa_block_manager *bm, const int64_t *token_ids, int32_t num_tokens, int32_t *seq_id);
PA_API pa_status pa_bm_seq_append_token(pa_block_manager *bm, int32_t seq, int64_t token_id);
PA_API pa_status pa_bm_seq_set_num_cached_tokens(pa_block_manager *bm, int32_t seq, int32_t num_cached_tokens);
PA_API pa_status pa_bm_seq_info(const pa_block_manager *bm, int32_t seq, int32_t *num_tokens,
                                int32_t *num_cached_tokens, int32_t *num_table_blocks);
PA_API int32_t pa_bm_can_allocate(const pa_block_manager *bm, int32_t seq);
PA_API pa_status pa_bm_allocate(pa_block_manager *bm, int32_t seq, int32_t num_cached_blocks);
PA_API pa_status pa_bm_deallocate(pa_block_manager *bm, int32_t seq);
PA_API int32_t pa_bm_can_append(const pa_block_manager *bm, int32_t seq);
PA_API pa_status pa_bm_may_append(pa_block_manager *bm, int32_t seq);
PA_API pa_status pa_bm_hash_blocks(pa_block_manager *bm, int32_t seq, int32_t num_scheduled_tokens);
PA_API int32_t pa_bm_seq_block_table(const pa_block_manager *bm, int32_t seq, int32_t *out, int32_t capacity);
PA_API pa_status pa_bm_block_tables(const pa_block_manager *bm, const int32_t *seq_ids, int32_t num_seqs,
                                    int32_t *out, int32_t max_blocks_per_seq);
PA_API int32_t pa_bm_free_block_ids(const pa_block_manager *bm, int32_t *out, int32_t capacity);
PA_API pa_status pa_bm_block_info(const pa_block_manager *bm, int32_t block_id, int32_t *ref_count,
                                  int32_t *has_hash, uint64_t *hash, int32_t *num_token_ids);
PA_API int32_t pa_bm_lookup_hash(const pa_block_manager *bm, uint64_t hash);
PA_API int32_t pa_bm_num_hashes(const pa_block_manager *bm);
PA_API uint64_t pa_bm_block_hash(const int64_t *token_ids, int32_t num_tokens, int32_t has_prefix, uint64_t prefix);
PA_API uint64_t pa_bm_xxh64(const void *data, size_t len, uint64_t seed);

/*
 * pa_set_checked -- enable (1) or disable (0) extra device checks for calls
 * made after it on any thread: block ids outside [0, num_blocks) are then
 * recorded as PA_DEV_BAD_BLOCK (reads of them return zeros either way).
 */
PA_API pa_status pa_set_checked(int32_t enabled);

/*
 * pa_get_device_error -- synchronise `stream`, return the first device-side
 * error recorded on the current device since the last call (code 0 if none)
 * and clear it.  Returns PA_ERR_DEVICE_CHECK if an error was recorded.
 * code and where may be NULL.
 */
PA_API pa_status pa_get_device_error(pa_stream_t stream, int32_t *code, int64_t *where);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
