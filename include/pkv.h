/*
 * pkv.h — C ABI of the paged KV-cache attention library (libpagedkv.so).
 *
 * One engine step of PagedAttention over a block-table-indexed KV cache, as
 * the vLLM pages describe it: new K/V tokens are scattered into physical
 * cache slots given by slot_mapping, then every query token attends
 * causally over its own request's logical blocks, read through the
 * request's block table.
 *
 * Sources of the operations (page title, section):
 *  - "vLLM internals: managing the KV cache like an OS manages memory",
 *    section 2.1: the cache is cut into 16-token blocks, a per-request block
 *    table maps logical to physical blocks, and a fused cache-write op stores
 *    each new token's K/V in its physical slot.
 *  - "continuous batching and PagedAttention" tutorial (juhe.plus), section
 *    3.3 "Data structures" (logical token -> block, offset -> physical block)
 *    and section 3.6 "PagedAttention kernel" (loop over the request's
 *    blocks, look up the physical block, load K/V, accumulate softmax(QK^T)V).
 *  - "Inside vLLM: Anatomy of a High-Throughput LLM Inference System",
 *    "Executing the forward pass": slot_mapping is built when inputs are
 *    prepared, and all sequences are flattened into one super-sequence whose
 *    positions keep each sequence attending only to its own tokens.
 *  - "vLLM source reading", section 5.1: the kernel scatters new K/V by
 *    slot_mapping and gathers cached K/V by block table.
 *
 * Conventions shared by every call
 *  - All tensor pointers are DEVICE pointers owned by the caller.  The
 *    library allocates nothing, keeps no state between calls, and enqueues
 *    its kernels on `stream` (a cudaStream_t; NULL is the legacy default
 *    stream) in call order.  Calls return after enqueueing, not after the
 *    GPU has finished.
 *  - bf16 means IEEE bfloat16 (16-bit) values; int32/int64 are little-endian
 *    two's complement.
 *  - Host-side argument errors are returned BEFORE anything is enqueued.
 *    Errors the GPU finds (a slot or block id outside the cache, inconsistent
 *    lengths, a bounded wait that ran out) are written to a device status
 *    word (see each call); the host reads it after synchronising.
 *  - Block size is fixed at 16 tokens.  Head size is 64 or 128.
 *  - The attention calls launch their first kernel with programmatic
 *    dependent launch: it may start while the kernel just before it on the
 *    stream (normally pkv_kv_write) is still running, and it reads
 *    seq_lens, query_start_loc, key_start_loc and block_tables at once
 *    (pkv_latent_attn_expanded may store an error in its device_status
 *    then, too).  Work of any ordinary kind before the call (copies,
 *    memsets, kernels launched without programmatic dependent launch) is
 *    complete by then.  A caller's own kernel that releases its dependents
 *    early (griddepcontrol.launch_dependents) must write that metadata,
 *    and clear that status word, first.
 *
 * KV cache layout (this library's own, not the one printed on the pages):
 *     bf16 kv_cache[num_blocks][num_kv_heads][2][16][head_size]
 *  index 0 of the third axis holds K, index 1 holds V.  A slot number is
 *  block * 16 + offset.  One block of one kv head is 2*16*head_size*2 bytes
 *  (8 KiB at head_size 128), contiguous; the whole cache is the pages'
 *  per-block formula 2 * block_size * num_kv_heads * head_size * 2 bytes
 *  times num_blocks.
 */
#ifndef PKV_H
#define PKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PKV_BLOCK_SIZE 16

typedef enum pkv_status {
    PKV_OK = 0,
    PKV_ERR_NULL = 1,            /* a required pointer is NULL                        */
    PKV_ERR_SHAPE = 2,           /* sizes negative or inconsistent with each other    */
    PKV_ERR_UNSUPPORTED = 3,     /* head_size not 64/128, block_size not 16, ...      */
    PKV_ERR_ALIGNMENT = 4,       /* a pointer or stride breaks the stated alignment   */
    PKV_ERR_WORKSPACE = 5,       /* workspace missing or too small (size reported)    */
    PKV_ERR_CUDA = 6,            /* a CUDA runtime call or kernel launch failed       */
    /* written by the GPU into a device status word: */
    PKV_ERR_DEVICE_INDEX = 7,    /* a slot or block id outside the cache was skipped  */
    PKV_ERR_DEVICE_METADATA = 8, /* seq_len < query_len, query_start_loc not ordered, */
                                 /* a sequence longer than its table or the hints     */
    PKV_ERR_DEVICE_TIMEOUT = 9,  /* a bounded wait on an asynchronous copy ran out    */
    PKV_ERR_PROTOCOL = 10        /* combine given a workspace paged_attn did not fill */
                                 /* for the same num_tokens/num_q_heads/head_size     */
} pkv_status;

/*
 * pkv_kv_write — the cache write ("reshape_and_cache").
 *
 * For every token t in [0, num_tokens) with slot_mapping[t] >= 0:
 *     b = slot_mapping[t] / 16, o = slot_mapping[t] % 16, and for every kv head h
 *     kv_cache[b][h][0][o][:] = key  [t][h][:]   (bit copy)
 *     kv_cache[b][h][1][o][:] = value[t][h][:]
 * Tokens with a negative slot are padding and are skipped.  Nothing else in
 * the cache changes.  Two tokens with the same slot in one call leave that
 * slot holding one of them (which one is unspecified).
 *
 *  kv_cache            bf16, layout above; 16-byte aligned.
 *  num_blocks          blocks in the cache (>= 1).
 *  key, value          bf16; token t, head h starts at ptr + t*token_stride + h*head_size;
 *                      heads of one token are contiguous.  16-byte aligned.
 *  *_token_stride      elements between consecutive tokens (a multiple of 8,
 *                      >= num_kv_heads*head_size); lets K/V be views of a fused QKV.
 *  slot_mapping        int64 [num_tokens].
 *  device_status       optional int32 device word (may be NULL).  If a slot is
 *                      >= num_blocks*16, that token is skipped and
 *                      PKV_ERR_DEVICE_INDEX is stored there.  The library never
 *                      clears it: the caller zeroes it beforehand.
 * Returns PKV_OK or a host-side error code; num_tokens == 0 enqueues nothing.
 */
int pkv_kv_write(void *kv_cache, int64_t num_blocks, int32_t num_kv_heads,
                 int32_t head_size, int32_t block_size,
                 const void *key, int64_t key_token_stride,
                 const void *value, int64_t value_token_stride,
                 const int64_t *slot_mapping, int32_t num_tokens,
                 int32_t *device_status, void *stream);

/*
 * pkv_paged_attn — causal paged attention for one flattened batch.
 *
 * Request r owns query tokens [query_start_loc[r], query_start_loc[r+1]);
 * with q_r of them and seq_lens[r] = L_r, its context is c_r = L_r - q_r and
 * its i-th query token sits at position c_r + i.  That token's row for q
 * head h is
 *     out[t][h][:] = sum_j softmax_j(scale * <query[t][h], K_j>) * V_j,
 *     j = 0 .. c_r + i,
 * where K_j, V_j are read from block block_tables[r][j / 16], offset j % 16,
 * kv head h / (num_q_heads / num_kv_heads) (grouped-query attention).  The
 * request's new tokens must already be in the cache (call pkv_kv_write
 * first, on the same stream).  Scores and the softmax are fp32; out is bf16
 * rounded to nearest even.
 *
 * Long rows of short requests are split along their keys (split-K
 * flash-decoding): this call writes `out` directly for rows that were not
 * split and leaves per-split partial results in the workspace for the rest.
 * pkv_paged_attn_combine MUST follow on the same stream to finish those rows.
 *
 *  out               bf16 [num_tokens][num_q_heads][head_size], contiguous, 16-byte aligned.
 *  query             bf16; token t, head h at query + t*query_token_stride + h*head_size;
 *                    16-byte aligned, stride a multiple of 8.
 *  kv_cache          bf16, layout above, 16-byte aligned; num_blocks in [1, 2^31) and
 *                    num_blocks * num_kv_heads < 2^31 (PKV_ERR_SHAPE otherwise; such a
 *                    cache is terabytes).
 *  block_tables      int32 [num_seqs][max_blocks_per_seq]; entries past
 *                    ceil(L_r/16) are never read.
 *  seq_lens          int32 [num_seqs].
 *  query_start_loc   int32 [num_seqs+1], non-decreasing, [0] = 0, [num_seqs] <= num_tokens.
 *  max_query_len,
 *  max_seq_len       host-side upper bounds of q_r and L_r; they size the
 *                    workspace.  A device value above its bound is an error
 *                    (PKV_ERR_DEVICE_METADATA) and that request's rows are
 *                    left unwritten.
 *  scale             softmax scale, e.g. 1/sqrt(head_size).
 *  num_splits        0 = automatic; k > 0 splits each splittable row's keys
 *                    into min(k, 32, pages) parts (testing and tuning).
 *  workspace         device scratch of workspace_bytes (256-byte aligned).
 *                    Its first int32 is the device status word: this call
 *                    resets it to PKV_OK and the GPU stores an error code there.
 *  workspace_needed  if not NULL, receives the bytes this call needs.  With
 *                    workspace == NULL or too small, nothing is enqueued and
 *                    PKV_ERR_WORKSPACE is returned (the size query).
 * The workspace depends only on num_seqs, num_tokens, max_query_len,
 * max_seq_len, the head counts and head_size; one workspace serves any number
 * of calls in stream order.
 */
int pkv_paged_attn(void *out, const void *query, int64_t query_token_stride,
                   const void *kv_cache, int64_t num_blocks,
                   const int32_t *block_tables, int32_t max_blocks_per_seq,
                   const int32_t *seq_lens, const int32_t *query_start_loc,
                   int32_t num_seqs, int32_t num_tokens,
                   int32_t max_query_len, int32_t max_seq_len,
                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_size,
                   int32_t block_size, float scale, int32_t num_splits,
                   void *workspace, size_t workspace_bytes, size_t *workspace_needed,
                   void *stream);

/*
 * pkv_paged_attn_shared_prefix — pkv_paged_attn for a batch whose requests
 * share a prefix of their block tables (cascade attention).
 *
 * Requests that share a prefix keep one physical copy of its blocks, each
 * block referenced from every sharer's table ("vLLM internals: managing the
 * KV cache like an OS manages memory", section 2.2: shared blocks with
 * reference counts; "continuous batching and PagedAttention" tutorial,
 * sections 3.5 and 5.2: parallel sampling, beam search and prefix caching
 * share the prompt's blocks).  This call computes exactly the result of
 * pkv_paged_attn (same arguments, same formula, same combine afterwards),
 * but reads the shared blocks once per kv head for all sharers: the keys of
 * the first `shared_prefix_blocks` table entries are attended by every
 * sharing row together on tensor-core tiles, cut into a few key ranges that
 * become splits of that row, and merged with the row's own keys by the
 * log-sum-exp combine (at most 32 splits per row in all).
 *
 * A request takes this path when its first shared_prefix_blocks table entries
 * equal request 0's, its query rows fit one decode tile (q_r * G <= 16) and
 * its context covers the prefix (L_r - q_r >= 16 * shared_prefix_blocks;
 * request 0's must too).  Other requests are computed as by pkv_paged_attn.
 * shared_prefix_blocks = 0 is pkv_paged_attn.  The workspace size also
 * depends on shared_prefix_blocks.
 */
int pkv_paged_attn_shared_prefix(void *out, const void *query, int64_t query_token_stride,
                                 const void *kv_cache, int64_t num_blocks,
                                 const int32_t *block_tables, int32_t max_blocks_per_seq,
                                 const int32_t *seq_lens, const int32_t *query_start_loc,
                                 int32_t num_seqs, int32_t num_tokens,
                                 int32_t max_query_len, int32_t max_seq_len,
                                 int32_t num_q_heads, int32_t num_kv_heads, int32_t head_size,
                                 int32_t block_size, float scale, int32_t num_splits,
                                 int32_t shared_prefix_blocks,
                                 void *workspace, size_t workspace_bytes, size_t *workspace_needed,
                                 void *stream);

/*
 * FP8 KV cache ("vLLM internals: managing the KV cache like an OS manages
 * memory", section 7.2: the KV cache itself can be kept in FP8; "continuous
 * batching and PagedAttention" tutorial, sections 8.8 and 10.3 and the FAQ
 * of 10.8: an FP8 KV cache halves its memory at almost no loss).
 *
 * The cache has the bf16 layout with one byte per element:
 *     uint8 [num_blocks][num_kv_heads][2][16][head_size]
 * each byte an E4M3 code (OCP FP8: sign, 4 exponent bits with bias 7, 3
 * mantissa bits; exponent 0 subnormal; 0x7F and 0xFF NaN; largest finite
 * 448).  One fp32 scale covers all K (k_scale) and one all V (v_scale); a
 * stored code c stands for value(c) * scale.
 *
 * pkv_kv_write_fp8 — pkv_kv_write into an E4M3 cache.  Element x (bf16) of
 * a new K (V) row is stored as the E4M3 code nearest to the fp32 quotient
 * x / k_scale (x / v_scale), computed with IEEE division rounded to nearest;
 * ties go to the even code and magnitudes beyond 448 are held at 448, with
 * the sign kept (a result that rounds to zero keeps its sign).  Arguments
 * as pkv_kv_write; k_scale and v_scale must be positive and finite
 * (PKV_ERR_SHAPE otherwise).
 */
int pkv_kv_write_fp8(void *kv_cache, int64_t num_blocks, int32_t num_kv_heads,
                     int32_t head_size, int32_t block_size,
                     const void *key, int64_t key_token_stride,
                     const void *value, int64_t value_token_stride,
                     const int64_t *slot_mapping, int32_t num_tokens,
                     float k_scale, float v_scale,
                     int32_t *device_status, void *stream);

/*
 * pkv_paged_attn_fp8 — pkv_paged_attn over an E4M3 cache, with K_j and V_j
 * taken as value(code) * k_scale and value(code) * v_scale; arguments,
 * workspace and protocol (pkv_paged_attn_combine after it) as
 * pkv_paged_attn.  Decode rows run on the streaming decode kernel, long
 * chunks on the tensor-core kernel with K and V widened to f16 in shared
 * memory.  Scores, softmax and accumulation are fp32; the query enters the
 * products as f16 after a per-row power-of-two scaling (exact for every
 * query element not below 2^-24 of its row's largest).
 */
int pkv_paged_attn_fp8(void *out, const void *query, int64_t query_token_stride,
                       const void *kv_cache, int64_t num_blocks,
                       const int32_t *block_tables, int32_t max_blocks_per_seq,
                       const int32_t *seq_lens, const int32_t *query_start_loc,
                       int32_t num_seqs, int32_t num_tokens,
                       int32_t max_query_len, int32_t max_seq_len,
                       int32_t num_q_heads, int32_t num_kv_heads, int32_t head_size,
                       int32_t block_size, float scale, float k_scale, float v_scale,
                       int32_t num_splits,
                       void *workspace, size_t workspace_bytes, size_t *workspace_needed,
                       void *stream);

/*
 * pkv_paged_attn_shared_prefix_fp8 — pkv_paged_attn_shared_prefix over an
 * E4M3 cache, with K_j and V_j taken as value(code) * k_scale and
 * value(code) * v_scale (as pkv_paged_attn_fp8): the shared prefix's keys are
 * read once per kv head for all sharers, widened to f16 in shared memory.
 * Arguments, workspace (sized as for pkv_paged_attn_shared_prefix) and
 * protocol (pkv_paged_attn_combine after it) as pkv_paged_attn_shared_prefix.
 */
int pkv_paged_attn_shared_prefix_fp8(void *out, const void *query, int64_t query_token_stride,
                                     const void *kv_cache, int64_t num_blocks,
                                     const int32_t *block_tables, int32_t max_blocks_per_seq,
                                     const int32_t *seq_lens, const int32_t *query_start_loc,
                                     int32_t num_seqs, int32_t num_tokens,
                                     int32_t max_query_len, int32_t max_seq_len,
                                     int32_t num_q_heads, int32_t num_kv_heads, int32_t head_size,
                                     int32_t block_size, float scale, float k_scale, float v_scale,
                                     int32_t num_splits, int32_t shared_prefix_blocks,
                                     void *workspace, size_t workspace_bytes, size_t *workspace_needed,
                                     void *stream);

/*
 * pkv_paged_attn_combine — the log-sum-exp merge of split rows.
 *
 * For every row (t, h) that pkv_paged_attn split into n parts with partial
 * outputs o_s (each normalised over its own keys) and lse_s = log of the sum
 * of exp(score) over that part's keys:
 *     M = max_s lse_s,  w_s = exp(lse_s - M),
 *     out[t][h][:] = sum_s w_s o_s / sum_s w_s      (bf16, nearest even);
 * a part with no visible key has lse_s = -inf and weight 0.  Rows that were
 * not split are left untouched.
 *
 *  out, workspace    the same buffers given to the preceding pkv_paged_attn;
 *  num_tokens, num_q_heads, head_size
 *                    the same values; a mismatch with what that call recorded
 *                    in the workspace stores PKV_ERR_PROTOCOL in the status
 *                    word and writes nothing.
 */
int pkv_paged_attn_combine(void *out, const void *workspace, size_t workspace_bytes,
                           int32_t num_tokens, int32_t num_q_heads, int32_t head_size,
                           void *stream);

/*
 * pkv_copy_blocks — copy-on-write of shared blocks.
 *
 * "continuous batching and PagedAttention" tutorial, section 3.8 "COW and
 * reference counting" (and "vLLM internals: managing the KV cache like an OS
 * manages memory", section 2.2): a request about to write into a block that
 * other requests still share gets a fresh block holding a copy of the
 * shared one; its block table then points at the copy.  This call makes the
 * copies: for every pair p,
 *     kv_cache[block_mapping[2p+1]][h][k_or_v][:][:] =
 *         kv_cache[block_mapping[2p]][h][k_or_v][:][:]     for every kv head h,
 * a bit copy of all 2*16*head_size*2 bytes per kv head.  Pairs with a source
 * or destination outside [0, num_blocks) are skipped and PKV_ERR_DEVICE_INDEX
 * is stored in *device_status (when not NULL; never cleared by the library).
 * A block that is the destination of one pair and the source of another in
 * the same call has no defined result.
 *
 *  block_mapping   int64 [num_pairs][2]: {source block, destination block}.
 */
int pkv_copy_blocks(void *kv_cache, int64_t num_blocks, int32_t num_kv_heads,
                    int32_t head_size, int32_t block_size,
                    const int64_t *block_mapping, int32_t num_pairs,
                    int32_t *device_status, void *stream);

/*
 * pkv_paged_attn_noalloc — paged attention that allocates nothing.
 *
 * The pages have no counterpart to this call; it exists for callers that
 * cannot allocate GPU memory where they run attention (for example code
 * in a serving loop under a strict no-allocation policy, or a plugin whose
 * host engine owns all device memory and passes in only inputs and
 * outputs).  It computes exactly what pkv_paged_attn followed by
 * pkv_paged_attn_combine computes, with the same arguments except the
 * workspace: the scratch lives in a fixed array of this library's own device
 * memory, PKV_NOALLOC_SCRATCH_BYTES (256 MiB) on every GPU where the call's
 * code is loaded, held until the process exits.  It calls no cudaMalloc,
 * cudaFree or other allocating routine.
 *
 *  - Sizes whose scratch (the workspace size pkv_paged_attn would report)
 *    exceeds PKV_NOALLOC_SCRATCH_BYTES are refused with PKV_ERR_WORKSPACE
 *    before anything is enqueued; argument errors return the same codes as
 *    pkv_paged_attn.
 *  - Every call looks up the array's device address on the current device
 *    (a host-side query that enqueues nothing).  Under lazy module loading
 *    the first call on each device also loads this code onto the device;
 *    make that first call before any stream capture.
 *  - Every call on a device shares the one array and leaves its contents
 *    behind; each call rewrites all of the scratch it later reads, so nothing
 *    needs clearing between calls.  Calls that overlap on the GPU (other
 *    streams, other threads' streams) race on the array: keep them ordered,
 *    e.g. on one stream.
 *  - device_status: optional int32 device word.  After the call's kernels,
 *    an error the GPU found (a PKV_ERR_DEVICE_* code, or PKV_ERR_PROTOCOL)
 *    is stored there unless the word already holds an error: as for the
 *    other calls' status words, the first error stays and the library never
 *    clears the word, so the caller zeroes it beforehand.  A call that finds
 *    no error, or that has no requests (num_seqs == 0, nothing enqueued),
 *    leaves the word as it was.
 */
#define PKV_NOALLOC_SCRATCH_BYTES (256u << 20)

int pkv_paged_attn_noalloc(void *out, const void *query, int64_t query_token_stride,
                           const void *kv_cache, int64_t num_blocks,
                           const int32_t *block_tables, int32_t max_blocks_per_seq,
                           const int32_t *seq_lens, const int32_t *query_start_loc,
                           int32_t num_seqs, int32_t num_tokens,
                           int32_t max_query_len, int32_t max_seq_len,
                           int32_t num_q_heads, int32_t num_kv_heads, int32_t head_size,
                           int32_t block_size, float scale, int32_t num_splits,
                           int32_t *device_status, void *stream);

/*
 * The step before the cache write, in the same pass as the write: the norm of
 * each query and key head, and their rotation to the tokens' positions.
 *
 * pkv_qk_norm_rope_kv_write — for every token t with position p = positions[t]
 * and slot s = slot_mapping[t] (block b = s / 16, offset o = s % 16):
 *     query_out[t][h]         = R_p(norm(query[t][h], q_weight))
 *     kv_cache[b][h][0][o][:] = R_p(norm(key[t][h], k_weight))
 *     kv_cache[b][h][1][o][:] = value[t][h]                        (bit copy)
 * with, per head of d = head_size dims, in fp32 and rounded once at the end
 * (to nearest even):
 *     norm(x, w)_i = x_i / sqrt(sum_j x_j^2 / d + eps) * w_i       (x itself if w is NULL)
 *     R_p          turns plane f = 0 .. rotary_dim / 2 - 1, the dims
 *                  (f, rotary_dim / 2 + f), or (2 f, 2 f + 1) if interleaved != 0,
 *                  from (x, y) to (x c - y s, y c + x s) with
 *                  c = cos_sin[p][f], s = cos_sin[p][rotary_dim / 2 + f];
 *                  dims from rotary_dim on stay as they are.
 * It replaces pkv_kv_write in a step; pkv_paged_attn follows on query_out.
 *
 *  query_out         bf16; token t, head h at ptr + t*token_stride + h*head_size.  May be
 *                    query itself (same pointer and stride); must not overlap the
 *                    inputs in any other way.
 *  query, key, value bf16, token strides as in pkv_kv_write (views of a fused QKV).
 *  kv_cache, slot_mapping, num_blocks, device_status
 *                    as pkv_kv_write.  A token with a negative slot is padding: its
 *                    query row is still written if its position is in the table.
 *                    Two tokens with one slot leave no defined K/V there.
 *  q_weight, k_weight bf16 [head_size], or NULL for no norm.
 *  eps               >= 0.
 *  cos_sin           fp32 [max_position][rotary_dim]: rotary_dim / 2 cosines, then as
 *                    many sines.  rotary_dim is a multiple of 16 in [16, head_size].
 *  positions         int64 [num_tokens].  A token whose position is outside
 *                    [0, max_position) is skipped, query row and slot, and
 *                    PKV_ERR_DEVICE_INDEX stored in device_status unless its slot is
 *                    negative; one with a slot past the cache has its query row
 *                    written, its K/V skipped and the same code stored.
 * Pointers are 16-byte aligned (positions, slot_mapping 8), strides multiples
 * of 8.  num_tokens == 0 enqueues nothing.
 */
int pkv_qk_norm_rope_kv_write(void *query_out, int64_t query_out_token_stride,
                              void *kv_cache, int64_t num_blocks,
                              int32_t num_q_heads, int32_t num_kv_heads,
                              int32_t head_size, int32_t block_size,
                              const void *query, int64_t query_token_stride,
                              const void *key, int64_t key_token_stride,
                              const void *value, int64_t value_token_stride,
                              const void *q_weight, const void *k_weight, float eps,
                              const float *cos_sin, int64_t max_position,
                              int32_t rotary_dim, int32_t interleaved,
                              const int64_t *positions, const int64_t *slot_mapping,
                              int32_t num_tokens, int32_t *device_status, void *stream);

/*
 * pkv_qk_norm_rope_kv_write_fp8 — the same into an E4M3 cache: the K row's fp32
 * values and the V row are stored as the codes of their quotients by k_scale
 * and v_scale (rounding as pkv_kv_write_fp8; K is not rounded to bf16 on the way).
 */
int pkv_qk_norm_rope_kv_write_fp8(void *query_out, int64_t query_out_token_stride,
                                  void *kv_cache, int64_t num_blocks,
                                  int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_size, int32_t block_size,
                                  const void *query, int64_t query_token_stride,
                                  const void *key, int64_t key_token_stride,
                                  const void *value, int64_t value_token_stride,
                                  const void *q_weight, const void *k_weight, float eps,
                                  const float *cos_sin, int64_t max_position,
                                  int32_t rotary_dim, int32_t interleaved,
                                  const int64_t *positions, const int64_t *slot_mapping,
                                  int32_t num_tokens, float k_scale, float v_scale,
                                  int32_t *device_status, void *stream);

/*
 * The latent cache (latent attention): one row a token instead of keys and
 * values per head,
 *     bf16 latent_cache[num_blocks][16][576]
 * of 512 latent dims (keys and values of every head are made from them) and 64
 * rotated key dims that all heads share.  Blocks, slots and block tables as
 * for the K/V cache; pkv_copy_blocks does not apply to it.
 */
#define PKV_LATENT_DIM 512
#define PKV_LATENT_ROPE_DIM 64

/*
 * pkv_latent_kv_write — for every token t with position p and slot s:
 *     latent_cache[s][0 .. 511]   = norm(latent[t], weight)
 *     latent_cache[s][512 .. 575] = R_p(key_rope[t])
 *     query_rope_out[t][h]        = R_p(query_rope[t][h])   for h < num_heads
 * with norm (over 512 dims) and R_p (rotary_dim 64) as in
 * pkv_qk_norm_rope_kv_write: fp32, rounded once.
 *
 *  latent            bf16, 512 dims at ptr + t*token_stride.
 *  key_rope          bf16, 64 dims at ptr + t*token_stride (both may be views of one
 *                    projection's output).
 *  weight            bf16 [512], or NULL for no norm.
 *  cos_sin           fp32 [max_position][64].
 *  query_rope(_out)  bf16, 64 dims at ptr + t*token_stride + h*head_stride; the output
 *                    may be the input itself, or the last 64 dims of the 576-wide rows
 *                    that pkv_latent_paged_attn takes.  num_heads == 0: no query.
 *  slot_mapping, positions, device_status
 *                    as pkv_qk_norm_rope_kv_write; padding tokens' query rows are
 *                    written if their positions are in the table.
 * Pointers are 16-byte aligned (positions, slot_mapping 8), strides multiples of 8.
 */
int pkv_latent_kv_write(void *latent_cache, int64_t num_blocks, int32_t block_size,
                        const void *latent, int64_t latent_token_stride,
                        const void *key_rope, int64_t key_rope_token_stride,
                        const void *weight, float eps,
                        const float *cos_sin, int64_t max_position, int32_t interleaved,
                        const int64_t *positions, const int64_t *slot_mapping, int32_t num_tokens,
                        void *query_rope_out, int64_t query_rope_out_token_stride,
                        int64_t query_rope_out_head_stride,
                        const void *query_rope, int64_t query_rope_token_stride,
                        int64_t query_rope_head_stride, int32_t num_heads,
                        int32_t *device_status, void *stream);

/*
 * pkv_latent_gather — the cached rows of every request, in order, into one
 * contiguous array: out[key_start_loc[r] + j] = row j of request r (bit copy),
 * j < seq_lens[r].  The per-head keys and values of the expanded form
 * (pkv_latent_attn_expanded) are a linear map of these rows.
 *
 *  out             bf16 [out_rows][576]; rows no request covers are left as they were.
 *                  May be NULL if out_rows == 0 (a batch of empty requests).
 *  block_tables    int32 [num_seqs][max_blocks_per_seq].
 *  seq_lens, key_start_loc
 *                  int32 [num_seqs] (key_start_loc may be longer).
 *  max_seq_len     host-side bound of seq_lens; at most 16 * max_blocks_per_seq.
 *  device_status   optional int32 device word, never cleared by the library.  A
 *                  request with a negative length, one past max_seq_len, or rows
 *                  outside `out` is skipped (PKV_ERR_DEVICE_METADATA); the rows of a
 *                  block id outside the cache are skipped (PKV_ERR_DEVICE_INDEX).
 * num_seqs is at most 65535.
 */
int pkv_latent_gather(void *out, int64_t out_rows, const void *latent_cache, int64_t num_blocks,
                      int32_t block_size, const int32_t *block_tables, int32_t max_blocks_per_seq,
                      const int32_t *seq_lens, const int32_t *key_start_loc, int32_t num_seqs,
                      int32_t max_seq_len, int32_t *device_status, void *stream);

/*
 * pkv_latent_paged_attn — causal attention over a latent cache, in the latent
 * space (the absorbed form of latent attention).  Requests, lengths and tables
 * as pkv_paged_attn; every head reads the same cached rows C_j of 576 dims:
 *     out[t][h][:] = sum_j softmax_j(scale * <query[t][h], C_j>) * C_j[0 .. 511],
 *     j = 0 .. c_r + i.
 * A query row holds the head's query in the latent space (its 128 or so plain
 * dims times the key up-projection: 512) and its rotated part (64, as
 * pkv_latent_kv_write leaves it); `out` times the value up-projection is the
 * head's output.  The request's new rows must already be in the cache.  Scores,
 * softmax and sums are fp32; the weights enter the product with the values as
 * bf16 (an error of at most 2^-8 of each weight); out is bf16, nearest even.
 * One call: no combine follows it.
 *
 *  out               bf16 [num_tokens][num_heads][512], contiguous.  Rows that no
 *                    request owns are left as they were.
 *  query             bf16; token t, head h at query + t*query_token_stride + h*576.
 *  latent_cache      bf16 [num_blocks][16][576]; num_blocks < 2^31.  Unwritten slots may
 *                    hold anything.  An infinity or NaN in a key row reaches no token
 *                    that does not see the row; one that sees a NaN is NaN, and what one
 *                    that sees an infinity gets is not defined.
 *  num_heads         1 .. 1024; num_tokens * num_heads < 2^31.
 *  max_query_len, max_seq_len, block_tables, seq_lens, query_start_loc
 *                    as pkv_paged_attn (a request whose values break them is left
 *                    unwritten, PKV_ERR_DEVICE_METADATA).  A block id outside the cache
 *                    reads as zeros (PKV_ERR_DEVICE_INDEX).
 *  workspace         device scratch, 256-byte aligned, of a fixed size (40 MB) whatever
 *                    the batch.  Its first int32 is the device status word: the call
 *                    stores PKV_OK or an error code there (PKV_OK, and nothing else, if
 *                    num_seqs == 0).  One workspace serves any
 *                    number of calls in stream order; calls that may overlap (other
 *                    streams, graphs replayed side by side) need one each.
 *  workspace_needed  if not NULL, receives that size; with workspace == NULL or
 *                    workspace_bytes too small nothing is enqueued and
 *                    PKV_ERR_WORKSPACE is returned (the size query).
 * Like the attention calls above, the first kernel may start while the kernel
 * before it (normally pkv_latent_kv_write) still runs, and reads the lengths
 * (seq_lens, query_start_loc) at once.
 */
int pkv_latent_paged_attn(void *out, const void *query, int64_t query_token_stride,
                          const void *latent_cache, int64_t num_blocks,
                          const int32_t *block_tables, int32_t max_blocks_per_seq,
                          const int32_t *seq_lens, const int32_t *query_start_loc,
                          int32_t num_seqs, int32_t num_tokens,
                          int32_t max_query_len, int32_t max_seq_len,
                          int32_t num_heads, int32_t block_size, float scale,
                          void *workspace, size_t workspace_bytes, size_t *workspace_needed,
                          void *stream);

/*
 * pkv_latent_attn_expanded — causal attention over per-head keys and values
 * made of latent rows (the expanded form of latent attention), for long
 * chunks.  Request r owns query tokens [query_start_loc[r], query_start_loc[r+1])
 * (q_r of them) and keys [key_start_loc[r], key_start_loc[r+1]) (L_r >= q_r: its
 * cached context, then the chunk); its i-th query sees the keys j <= L_r - q_r + i:
 *     s_j          = scale * (<query[t][h][0 .. 127], key[j][h]>
 *                             + <query[t][h][128 .. 191], key_rope[j]>)
 *     out[t][h][:] = sum_j softmax_j(s_j) * value[j][h][:]
 * pkv_latent_gather gives the rows of cached requests in this order: key and
 * value are their first 512 dims times the up-projection, key_rope is the last
 * 64 (a view of the gathered rows).  Arithmetic as pkv_latent_paged_attn.
 *
 *  out               bf16 [num_tokens][num_heads][128], contiguous; rows that no request
 *                    owns are left as they were.
 *  query             bf16; token t, head h at ptr + t*token_stride + h*192 (128 plain
 *                    dims, then 64 rotated ones).
 *  key, value        bf16; key row j, head h at ptr + j*token_stride + h*head_stride, 128
 *                    dims (views of one projection's output, or head-major).
 *  key_rope          bf16; 64 dims at ptr + j*token_stride, shared by the heads.
 *  query_start_loc, key_start_loc
 *                    int32 [num_seqs + 1], non-decreasing, the last at most num_tokens
 *                    and num_keys.
 *  max_query_len, max_key_len
 *                    host-side bounds of q_r and L_r.  A request that breaks them, or
 *                    has fewer keys than queries, is left unwritten.
 *  device_status     optional int32 device word, never cleared by the library:
 *                    PKV_ERR_DEVICE_METADATA for such a request (also where no token can
 *                    be answered: num_tokens, num_keys or max_query_len of 0).
 * What lies between or behind the requests' rows may be anything.  An infinity or
 * NaN in a key or value row reaches no token that does not see the row; one that
 * sees a NaN in a key is NaN, and what one that sees another such value gets (NaN
 * in all its dims, or in those) is not defined.  Pointers are 16-byte aligned, strides
 * multiples of 8.  No workspace.
 * Like the attention calls above, the kernel may start while the kernel before it
 * (normally the up-projection that makes key and value) still runs.  It reads
 * query_start_loc and key_start_loc, and reports requests that break their
 * bounds, at once; the tensors only when that kernel has ended.
 */
int pkv_latent_attn_expanded(void *out, const void *query, int64_t query_token_stride,
                             const void *key, int64_t key_token_stride, int64_t key_head_stride,
                             const void *key_rope, int64_t key_rope_token_stride,
                             const void *value, int64_t value_token_stride, int64_t value_head_stride,
                             const int32_t *query_start_loc, const int32_t *key_start_loc,
                             int32_t num_seqs, int32_t num_tokens, int32_t num_keys,
                             int32_t max_query_len, int32_t max_key_len,
                             int32_t num_heads, float scale, int32_t *device_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H */
