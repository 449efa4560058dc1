/*
 * pa.h -- C ABI of the GB300 (sm_103a) PagedAttention decode library.
 *
 * The library implements the data-parallel hot path of a paged KV cache as
 * described in "vLLM: Architecture, PagedAttention & Internals" (LLM stack
 * book 7.3) and "vLLM: High-Throughput Serving with PagedAttention" (lesson 13.15):
 *
 *   pa_reshape_and_cache   scatter each step's new K/V rows into their slots
 *   pa_decode              one query token per sequence attends over its
 *                          paged context, walking the block table
 *   pa_decode_partitioned  the same attention split into fixed token
 *                          partitions whose results are merged by
 *                          log-sum-exp (for long contexts)
 *   pa_decode_multi        several new query tokens per sequence (a
 *                          prompt chunk or speculative positions), causal
 *                          among themselves, over the same paged cache
 *   pa_decode_cascade      decode of a batch sharing a prompt prefix: the
 *                          shared blocks read once per KV head
 *   pa_copy_blocks         block copies of copy-on-write, all layers at once
 *   pa_rope_and_cache      the cache write with per-head norms of the new
 *                          queries and keys and their rotation by position
 *   pa_verify_drafts       drafted tokens accepted or rejected against the
 *                          target's probabilities, and the token after them
 *   *_fp8                  the cache writes, decode, split-KV decode and
 *                          multi-token attention over an FP8 (E4M3) cache
 *                          with per-KV-head scales
 *   *_fp4                  the cache write, its reading, decode, split-KV decode
 *                          and multi-token attention over a cache of 4-bit
 *                          (E2M1) codes with a scale for every 16 of them
 *   pa_build_step          block tables, lengths, positions and slots of a step
 *   pa_trim_blocks         from lengths on the device; blocks given back
 *   pa_process_logits      penalties, biases, masks, temperature and softmax
 *                          between the model's logits and pa_verify_drafts
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Memory.  Every pointer argument except `workspace_bytes`-style sizes is a
 * DEVICE pointer on the current CUDA device.  The caller owns all memory,
 * including the workspace of pa_decode_partitioned; the library allocates
 * nothing and frees nothing.
 *
 * Layouts (elements, row-major):
 *   k_cache, v_cache : [num_blocks, num_kv_heads, block_size, head_dim],
 *                      contiguous; a (physical block, KV head) tile is one
 *                      contiguous run of block_size * head_dim elements.
 *   q                : [num_seqs, num_heads, head_dim]; heads contiguous,
 *                      sequence stride q_seq_stride (>= num_heads*head_dim).
 *   out              : [num_seqs, num_heads, head_dim], contiguous.
 *   k, v (new rows)  : [num_tokens, num_kv_heads, head_dim]; heads
 *                      contiguous, token stride k_token_stride /
 *                      v_token_stride.
 *   block_tables     : int32 [num_seqs, max_blocks_per_seq]; entry
 *                      [s][i] is the physical block holding tokens
 *                      16*i .. 16*i+15 of sequence s.  Entries at and past
 *                      ceil(seq_lens[s] / block_size) are never read.
 *   seq_lens         : int32 [num_seqs], tokens each sequence attends over.
 *   slot_mapping     : int64 [num_tokens]; slot = block * block_size + row;
 *                      a negative slot marks a padding token (skipped).
 *
 * Query head h reads KV head h / (num_heads / num_kv_heads) (grouped-query
 * attention with consecutive query heads sharing a KV head).  A sequence
 * with seq_len 0 produces zeros.
 *
 * dtype (pa_dtype) is the storage type of q, out, k, v and both caches (all
 * the same).  Arithmetic is fp32; out is rounded to nearest-even.
 *
 * Streams.  `stream` is a cudaStream_t (NULL = the legacy default stream).
 * Every call only enqueues kernels on it and never synchronises, except
 * pa_device_error, which reads device memory synchronously.  The decode
 * kernels are launched with programmatic stream serialization: when the
 * kernel before them in the stream is a cache write of this library
 * (pa_reshape_and_cache and its _fp8 and _fp4 forms, or pa_rope_and_cache and its
 * _fp8 form without queries), they start while it finishes and read seq_lens,
 * block_tables and query_start meanwhile -- the cache writes never touch those --
 * and touch the caches, q and out only after it has completed.  After any other
 * kernel they start as usual.
 *
 * Errors.  Calls return PA_OK (0) or a negative pa_status; nothing is
 * launched when the host-side checks fail.  Contents of device arrays are not
 * inspected on the host.  Instead the kernels range-check every block id,
 * slot and sequence length they read, skip the offending access and set a bit
 * in a sticky device-side error word (PA_DEVERR_*), read and cleared with
 * pa_device_error.  No input can make a kernel read or write outside the
 * buffers described by the arguments.
 *
 * Thread safety.  Calls may be made from any host thread; the only shared
 * state is the device error word.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    PA_F32 = 0,
    PA_BF16 = 1,
    PA_F16 = 2,
    PA_E4M3 = 3,     /* FP8 E4M3 cache storage (the *_fp8 entry points only) */
    PA_E2M1 = 4      /* FP4 E2M1 cache storage (the *_fp4 entry points only) */
} pa_dtype;

typedef enum {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = -1,   /* NULL pointer, bad size, misaligned pointer */
    PA_ERR_UNSUPPORTED = -2,   /* head_dim, GQA group, block_size or dtype not built */
    PA_ERR_WORKSPACE = -3,     /* workspace missing or too small */
    PA_ERR_CUDA = -4           /* a CUDA runtime call or launch failed */
} pa_status;

/* bits of the device error word */
#define PA_DEVERR_BLOCK_ID   0x1u  /* a block-table entry outside [0, num_blocks) was skipped */
#define PA_DEVERR_SEQ_LEN    0x2u  /* a seq_len < 0 or > max_blocks_per_seq*block_size (or past
                                      max_seq_len in the partitioned call) was clamped, or
                                      a query row range of pa_decode_multi was invalid */
#define PA_DEVERR_SLOT       0x4u  /* a slot >= num_blocks*block_size was skipped */
#define PA_DEVERR_TIMEOUT    0x8u  /* a wait on an asynchronous copy exceeded its limit */
#define PA_DEVERR_POSITION   0x10u /* a position outside the rotation table: its token was skipped */
#define PA_DEVERR_TOKEN      0x20u /* a drafted token outside the vocabulary was rejected, or a
                                      token of pa_process_logits outside it was left out */
#define PA_DEVERR_NO_BLOCKS  0x40u /* pa_build_step: the free list ran out, sequences were refused */

/*
 * pa_reshape_and_cache -- write the step's new keys and values into the cache.
 *
 * Defined in "vLLM: Architecture, PagedAttention & Internals", *The forward
 * step in detail*: the runner computes, for each token being written, the
 * physical slot (block * block_size + offset) and the attention layer first
 * scatters the fresh K and V there.  For every token t with slot_mapping[t]
 * >= 0, the rows k[t][j][:] and v[t][j][:] of every KV head j are copied bit
 * for bit to k_cache[slot/bs][j][slot%bs][:] and v_cache[...]; nothing else
 * in the caches changes.  Two tokens with the same slot race (last writer
 * wins, per element).
 *
 * Requirements: num_tokens >= 0 (0 launches nothing); block_size == 16;
 * head_dim * element size a multiple of 16 bytes; the token strides >=
 * num_kv_heads*head_dim.
 */
int pa_reshape_and_cache(const void *k, const void *v, void *k_cache,
                         void *v_cache, const int64_t *slot_mapping,
                         int64_t num_tokens, int32_t num_kv_heads,
                         int32_t head_dim, int64_t k_token_stride,
                         int64_t v_token_stride, int64_t num_blocks,
                         int32_t block_size, int32_t dtype, void *stream);

/*
 * pa_rope_and_cache -- the step's cache write with what precedes it in the
 * attention layer, in one pass: norms of the new queries and keys for each
 * head, their rotation by position, q to q_out and k and v to their slots.
 *
 * For every token t, query head h and KV head j, with x one head's head_dim
 * elements of q or k:
 *   norm      with a weight row (q_weight for q, k_weight for k; [head_dim] of
 *             `dtype`; NULL: no norm):  x <- x / sqrt(mean(x^2) + eps) * weight
 *   rotation  of the first rot_dim elements (0: none), as rot_dim / 2 pairs:
 *             (x[i], x[i + rot_dim/2]), or (x[2i], x[2i+1]) when interleaved
 *             is not 0.  Pair i becomes (a cos - b sin, b cos + a sin) with
 *             cos = rope_table[p][i], sin = rope_table[p][rot_dim/2 + i] and
 *             p = positions[t].  Elements past rot_dim pass.
 * q_out[t][h] is the result for q, and the slot of t receives the result for
 * k in k_cache and v[t][j] bit for bit in v_cache.  Arithmetic is fp32 with one
 * rounding at the end (squares have to stay inside the binary32 range).
 *
 * rope_table is float32 [num_positions][rot_dim], contiguous.  q and q_out are
 * [num_tokens][num_heads][head_dim] with heads contiguous and token strides of
 * their own; q_out may be q itself with the same stride (in place), and may not
 * overlap q, k or v otherwise.  num_heads == 0 writes keys and values only
 * (q, q_out and q_weight are not looked at then).
 *
 * A token with a negative slot (padding) has its q_out row written and nothing
 * in the caches; a slot past the pool likewise, with PA_DEVERR_SLOT.  A position
 * outside [0, num_positions) skips the token altogether, with
 * PA_DEVERR_POSITION unless it is a padding token.
 *
 * Requirements: block_size == 16; head_dim a multiple of 16, at most 256;
 * rot_dim a multiple of 16, at most head_dim; num_heads, num_kv_heads <= 65535;
 * eps >= 0 and finite if there is a weight; all pointers but positions and
 * slot_mapping 16-byte aligned, token strides >= one token's heads with a byte
 * size that is a multiple of 16.  Two tokens with the same slot race.
 */
int pa_rope_and_cache(void *q_out, const void *q, const void *k, const void *v,
                      void *k_cache, void *v_cache, const void *q_weight,
                      const void *k_weight, float eps, const float *rope_table,
                      int64_t num_positions, int32_t rot_dim, int32_t interleaved,
                      const int64_t *positions, const int64_t *slot_mapping,
                      int64_t num_tokens, int32_t num_heads, int32_t num_kv_heads,
                      int32_t head_dim, int64_t q_token_stride,
                      int64_t q_out_token_stride, int64_t k_token_stride,
                      int64_t v_token_stride, int64_t num_blocks,
                      int32_t block_size, int32_t dtype, void *stream);

/*
 * pa_decode -- decode-step paged attention.
 *
 * Defined in "vLLM: Architecture, PagedAttention & Internals", *PagedAttention
 * in one paragraph* (the kernel gathers K and V block by block through the
 * block table; the arithmetic of attention is unchanged) and "vLLM:
 * High-Throughput Serving with PagedAttention", *PagedAttention, the core
 * idea* (step 4, attend through the table).
 * For every sequence s and query head h:
 *     out[s][h] = sum_t softmax_t(scale * q[s][h] . K_s[t]) * V_s[t],
 *     t = 0 .. seq_lens[s]-1, K_s[t] = k_cache[bt[s][t/16]][h/G][t%16].
 * The softmax is evaluated online (running maximum and sum in fp32), which is
 * exact up to rounding.
 *
 * Requirements: block_size == 16; head_dim in {64, 128}; num_heads a
 * multiple of num_kv_heads with G = num_heads/num_kv_heads in {1, 2, 4, 8};
 * num_seqs <= 65535 (batches larger than one thread block orders in shared
 * memory -- 4096 sequences at head_dim 128 -- run as consecutive slices);
 * num_kv_heads <= 65535; k_cache and v_cache 16-byte
 * aligned.  num_seqs == 0 launches nothing.
 */
int pa_decode(void *out, const void *q, const void *k_cache,
              const void *v_cache, const int32_t *block_tables,
              const int32_t *seq_lens, int32_t num_seqs, int32_t num_heads,
              int32_t num_kv_heads, int32_t head_dim, int64_t num_blocks,
              int32_t block_size, int32_t max_blocks_per_seq,
              int64_t q_seq_stride, float scale, int32_t dtype, void *stream);

/*
 * pa_decode_split -- pa_decode with an explicit work split: each (sequence,
 * KV head) is processed by a cluster of `splits` thread blocks (1, 2, 4 or 8)
 * whose partial results are merged on chip.  splits == 0 picks the split from
 * the problem shape (what pa_decode does).  The result does not depend on the
 * thread count within a block, but its rounding may differ between split
 * counts.
 */
int pa_decode_split(void *out, const void *q, const void *k_cache,
                    const void *v_cache, const int32_t *block_tables,
                    const int32_t *seq_lens, int32_t num_seqs,
                    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                    int64_t num_blocks, int32_t block_size,
                    int32_t max_blocks_per_seq, int64_t q_seq_stride,
                    float scale, int32_t dtype, int32_t splits, void *stream);

/*
 * pa_decode_partitioned_workspace_size -- bytes of workspace that
 * pa_decode_partitioned needs for these sizes.  Returns 0 on invalid sizes.
 *
 * Workspace layout (fp32, documented so that callers and tests can read the
 * per-partition results; P = ceil(max_seq_len / partition_size)):
 *   o_part [num_seqs][num_heads][P][head_dim]   normalised partial outputs
 *   m_part [num_seqs][num_heads][P]             max of scale*q.k in the
 *                                               partition (natural units)
 *   l_part [num_seqs][num_heads][P]             sum of exp(scale*q.k - m)
 * each array starting on a 256-byte boundary in that order.  Entries of
 * partitions past a sequence's last one are not written.
 */
size_t pa_decode_partitioned_workspace_size(int32_t num_seqs,
                                            int32_t num_heads,
                                            int32_t head_dim,
                                            int32_t max_seq_len,
                                            int32_t partition_size);

/*
 * pa_decode_partitioned -- split-KV decode for long contexts.
 *
 * Same result as pa_decode.  The tokens of each sequence are cut into
 * partitions of partition_size tokens (a multiple of 16); one thread block
 * per (sequence, KV head, partition) writes that partition's softmax
 * statistics (m_p, l_p) and normalised output o_p to the workspace, and a
 * second kernel merges them:  M = max_p m_p,  c_p = l_p exp(m_p - M),
 * out = sum_p c_p o_p / sum_p c_p.  The streaming softmax this rests on is
 * named in "vLLM" (stanleyjacob.dev), Part IV, *Stage 6: The forward pass*
 * (the kernel streams through a sequence it never holds in one piece).
 *
 * max_seq_len bounds seq_lens (it sizes the grid and the workspace); a
 * larger seq_len is clamped and flagged PA_DEVERR_SEQ_LEN.
 * Requirements as pa_decode, plus partition_size a positive multiple of 16
 * and workspace_bytes >= pa_decode_partitioned_workspace_size(...); the
 * workspace must be 256-byte aligned.
 *
 * If pa_device_error reports PA_DEVERR_TIMEOUT after a call, that call's
 * output is undefined: a partition whose bounded wait ran out is not written,
 * and the merge then reads whatever the workspace held before the call.
 */
int pa_decode_partitioned(void *out, const void *q, const void *k_cache,
                          const void *v_cache, const int32_t *block_tables,
                          const int32_t *seq_lens, int32_t num_seqs,
                          int32_t num_heads, int32_t num_kv_heads,
                          int32_t head_dim, int64_t num_blocks,
                          int32_t block_size, int32_t max_blocks_per_seq,
                          int64_t q_seq_stride, float scale, int32_t dtype,
                          int32_t partition_size, int32_t max_seq_len,
                          void *workspace, size_t workspace_bytes,
                          void *stream);

/*
 * pa_decode_multi -- paged attention for several new query tokens per
 * sequence: a chunk of a long prompt (chunked prefill) or the k+1 positions
 * a target model verifies in one pass of speculative decoding.
 *
 * Defined in "vLLM: Architecture, PagedAttention & Internals", *Prefill,
 * decode, and chunked prefill* (one forward pass mixes a slice of a prompt's
 * tokens with one-token decodes, each attending over its sequence's cache)
 * and *Speculative decoding* (the target model scores the k drafted tokens
 * and the one after them in a single pass).  The new tokens' keys and values
 * are in the cache already (pa_reshape_and_cache of the same step), and new
 * token i of a sequence sees the cache up to and including itself.
 *
 * Sequence s owns query rows r = query_start[s] .. query_start[s+1]-1
 * (n_s = query_start[s+1] - query_start[s] of them, 0 <= n_s <= seq_lens[s]);
 * row r = query_start[s] + i is the token at position seq_lens[s] - n_s + i.
 * For every such row and query head h:
 *     out[r][h] = sum_t softmax_t(scale * q[r][h] . K_s[t]) * V_s[t],
 *     t = 0 .. seq_lens[s] - n_s + i,
 * with K_s, V_s and the GQA mapping as in pa_decode.  A sequence with n_s = 0
 * (a request that runs no token this step) has no rows.
 *
 * Layouts: q is [num_q_rows][num_heads][head_dim] with row stride
 * q_row_stride (>= num_heads*head_dim, a multiple of 8 elements); out is
 * [num_q_rows][num_heads][head_dim], contiguous; query_start is int32
 * [num_seqs + 1], non-decreasing, query_start[num_seqs] <= num_q_rows.
 *
 * Requirements: as pa_decode, and dtype PA_BF16 or PA_F16 (PA_F32 gives
 * PA_ERR_UNSUPPORTED); max_query_len >= every n_s (it sizes the launch);
 * q, out 16-byte aligned.  A sequence whose row range is out of bounds,
 * decreasing, longer than max_query_len or longer than seq_lens[s] sets
 * PA_DEVERR_SEQ_LEN and its rows are not written.  num_seqs == 0 or
 * num_q_rows == 0 launches nothing.
 */
int pa_decode_multi(void *out, const void *q, const void *k_cache,
                    const void *v_cache, const int32_t *block_tables,
                    const int32_t *seq_lens, const int32_t *query_start,
                    int32_t num_seqs, int32_t num_q_rows, int32_t max_query_len,
                    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                    int64_t num_blocks, int32_t block_size,
                    int32_t max_blocks_per_seq, int64_t q_row_stride,
                    float scale, int32_t dtype, void *stream);

/*
 * pa_verify_drafts -- verification of drafted tokens, the step after
 * pa_decode_multi in speculative decoding: "vLLM: Architecture, PagedAttention &
 * Internals", *Speculative decoding* (the target scores the drafted tokens and
 * the one after them in a single pass; drafts are kept up to the first one the
 * target rejects).
 *
 * The rows are those of pa_decode_multi: sequence s owns rows query_start[s] ..
 * query_start[s+1]-1, n of them; tokens[r] is row r's input token, so row
 * query_start[s] is the token accepted last and row query_start[s] + i, i = 1 ..
 * n-1, is draft i.  target_probs row r is the target's distribution of the
 * token that follows row r; draft_probs row r is the distribution that draft
 * tokens[r] was drawn from (rows query_start[s] are not read).  With
 * draft_probs NULL the drafts come without probabilities (copied from the
 * prompt, or greedy) and their probability is 1.
 *
 * Draft i at row r is accepted while accept_uniform[r] * draft_probs[r][x] <
 * target_probs[r-1][x], x = tokens[r] (the product is exact).  With a the number
 * accepted, the next token is drawn from the weights
 *   w_v = max(target_probs[r-1][v] - draft_probs[r][v], 0)   a rejected draft r
 *         (or target_probs[r-1] with w_x = 0 without draft probabilities; if
 *         nothing is left, target_probs[r-1] itself);
 *   w_v = target_probs[last row][v]                          if all are accepted.
 * The difference is rounded to binary32; a sum is a pair of binary32 numbers,
 * itself and what its roundings lost (about 46 bits together).  The token is the
 * first v with w_0 + .. + w_v > u * sum(w), u = sample_uniform[s] clamped to
 * [0, 1] and NaN as 0 (at u = 1 the last v with a weight).  Entries
 * that are negative or NaN count as 0, and an infinite entry leaves weight 0;
 * a row without any weight gives token -1.  Sums must stay inside the binary32
 * range.
 *
 * out_tokens, int32 [num_seqs][max_query_len], receives the a accepted drafts,
 * the token drawn, then -1; num_accepted[s] receives a.  A sequence without
 * rows gets -1 throughout and 0; one whose row range is out of bounds,
 * decreasing or longer than max_query_len likewise, with PA_DEVERR_SEQ_LEN.  A
 * drafted token outside [0, vocab_size) is rejected, with PA_DEVERR_TOKEN if it
 * is the first one rejected.
 *
 * accept_uniform is float32 [num_rows] (rows query_start[s] are not read),
 * sample_uniform float32 [num_seqs].  target_probs and draft_probs are of
 * `dtype`, rows contiguous with strides >= vocab_size of any alignment.
 * num_seqs == 0 launches nothing.
 */
int pa_verify_drafts(int32_t *out_tokens, int32_t *num_accepted,
                     const void *target_probs, const void *draft_probs,
                     const int32_t *tokens, const float *accept_uniform,
                     const float *sample_uniform, const int32_t *query_start,
                     int32_t num_seqs, int32_t num_rows, int32_t max_query_len,
                     int32_t vocab_size, int64_t target_row_stride,
                     int64_t draft_row_stride, int32_t dtype, void *stream);

/*
 * pa_copy_blocks -- the GPU half of copy-on-write.
 *
 * Defined in "vLLM: Architecture, PagedAttention & Internals", *Copy-on-write
 * for shared blocks* (a writer about to append into a block whose refcount is
 * above one gets a fresh block holding a copy of the shared one; the
 * scheduler emits the copy) and "vLLM: High-Throughput Serving with
 * PagedAttention", *PagedAttention, the core idea* (parallel sampling, beam
 * search and prefix caching share blocks until one writer diverges).
 * For every pair i and every cache c, bytes
 * [src_i * block_bytes, (src_i + 1) * block_bytes) of caches[c] are copied to
 * the same range at dst_i.  One launch covers K and V of every layer.
 *
 * caches        HOST array of num_caches (0..256) DEVICE pointers, each the
 *               base of a cache of num_blocks blocks of block_bytes bytes
 *               (any storage type: K, V, of any layer, 16-bit or E4M3), each
 *               16-byte aligned.
 * block_mapping DEVICE int64 [num_pairs][2]: (src, dst) block ids.
 * block_bytes   bytes of one block of one cache, a positive multiple of 16
 *               (num_kv_heads * block_size * head_dim * element size).
 * Pairs run in parallel: no dst may appear twice or also be a src (what
 * copy-on-write produces: fresh destinations, shared sources, possibly one
 * source copied several times).  A pair with src or dst outside
 * [0, num_blocks) is skipped and sets PA_DEVERR_BLOCK_ID.  num_pairs == 0 or
 * num_caches == 0 launches nothing.
 */
int pa_copy_blocks(void *const *caches, int32_t num_caches,
                   const int64_t *block_mapping, int64_t num_pairs,
                   int64_t num_blocks, int64_t block_bytes, void *stream);

/*
 * FP8 KV cache.
 *
 * Defined in "vLLM: Architecture, PagedAttention & Internals", *The knobs
 * that actually matter*, item 5 (an FP8 KV cache enlarges the effective pool)
 * and "vLLM: High-Throughput Serving with PagedAttention", *The benefits of
 * vLLM* (quantized KV cache); the pages fix no format.  This library stores
 * OCP FP8 E4M3 codes (1 sign, 4 exponent bits with bias 7, 3 fraction bits;
 * largest finite 448; S.1111.111 is NaN) in the same layout
 * [num_blocks, num_kv_heads, 16, head_dim] (one byte per element), with one
 * float scale per KV head for K and one for V: code c of KV head j stands for
 * value(c) * k_scale[j] (or v_scale[j]).  Scales are device arrays float32
 * [num_kv_heads] owned by the caller; a per-tensor scale is the case where
 * all entries are equal.  Scales must be positive and finite (others are
 * not checked; they make the results meaningless, never unsafe).
 *
 * pa_reshape_and_cache_fp8 -- the cache write of pa_reshape_and_cache, with
 * each element x of KV head j stored as E4M3(x / scale_j): the quotient is
 * rounded to binary32 (IEEE division), then to E4M3 with round to nearest,
 * ties to even; finite magnitudes above 448 and infinities saturate to
 * +-448, NaN stays NaN.  k and v are in `dtype` (PA_F32, PA_BF16, PA_F16),
 * 16-byte aligned with token strides whose byte size is a multiple of 16;
 * head_dim a multiple of 16; k_cache and v_cache 16-byte aligned.
 */
int pa_reshape_and_cache_fp8(const void *k, const void *v, void *k_cache,
                             void *v_cache, const float *k_scale,
                             const float *v_scale, const int64_t *slot_mapping,
                             int64_t num_tokens, int32_t num_kv_heads,
                             int32_t head_dim, int64_t k_token_stride,
                             int64_t v_token_stride, int64_t num_blocks,
                             int32_t block_size, int32_t dtype, void *stream);

/*
 * pa_rope_and_cache_fp8 -- pa_rope_and_cache into E4M3 caches: the result x for
 * k, and v itself, of KV head j are stored as E4M3(x / scale_j), rounded as in
 * pa_reshape_and_cache_fp8 (the quotient of the fp32 result).  q_out stays in
 * `dtype`.
 */
int pa_rope_and_cache_fp8(void *q_out, const void *q, const void *k, const void *v,
                          void *k_cache, void *v_cache, const float *k_scale,
                          const float *v_scale, const void *q_weight,
                          const void *k_weight, float eps, const float *rope_table,
                          int64_t num_positions, int32_t rot_dim,
                          int32_t interleaved, const int64_t *positions,
                          const int64_t *slot_mapping, int64_t num_tokens,
                          int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                          int64_t q_token_stride, int64_t q_out_token_stride,
                          int64_t k_token_stride, int64_t v_token_stride,
                          int64_t num_blocks, int32_t block_size, int32_t dtype,
                          void *stream);

/*
 * pa_decode_fp8 / pa_decode_partitioned_fp8 -- pa_decode and
 * pa_decode_partitioned over E4M3 caches: K_s[t] = value(code) * k_scale[j]
 * and V_s[t] = value(code) * v_scale[j] for KV head j, the attention itself
 * unchanged.  `dtype` is the type of q and out: PA_BF16 or PA_F16 (q is
 * rounded to f16 for the tensor cores, so its entries must lie within the
 * f16 range, |q| < 65504).  The partitioned form takes the workspace of
 * pa_decode_partitioned_workspace_size and writes the same statistics.
 * Other requirements as pa_decode, plus q and out 16-byte aligned with a q
 * stride whose byte size is a multiple of 16.
 */
int pa_decode_fp8(void *out, const void *q, const void *k_cache,
                  const void *v_cache, const float *k_scale, const float *v_scale,
                  const int32_t *block_tables, const int32_t *seq_lens,
                  int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                  int32_t head_dim, int64_t num_blocks, int32_t block_size,
                  int32_t max_blocks_per_seq, int64_t q_seq_stride, float scale,
                  int32_t dtype, void *stream);

int pa_decode_partitioned_fp8(void *out, const void *q, const void *k_cache,
                              const void *v_cache, const float *k_scale,
                              const float *v_scale, const int32_t *block_tables,
                              const int32_t *seq_lens, int32_t num_seqs,
                              int32_t num_heads, int32_t num_kv_heads,
                              int32_t head_dim, int64_t num_blocks,
                              int32_t block_size, int32_t max_blocks_per_seq,
                              int64_t q_seq_stride, float scale, int32_t dtype,
                              int32_t partition_size, int32_t max_seq_len,
                              void *workspace, size_t workspace_bytes,
                              void *stream);

/*
 * pa_decode_multi_fp8 -- pa_decode_multi over E4M3 caches: several new tokens
 * per sequence (drafts to verify, or a chunk of a prompt), causal among
 * themselves, K_s[t] and V_s[t] dequantised as in pa_decode_fp8.  `dtype` is the
 * type of q and out, PA_BF16 or PA_F16.  q is rounded to f16: |q| < 65504, in
 * steps of 2^-24 below 2^-14 (a bf16 query under 2^-25 counts as 0).  Weights are
 * rounded to f16 relative to the row's largest (half a step 2^-11; the sum that
 * divides is of the rounded ones) and sums are fp32: keys each below 2^-25 of
 * what a row has summed so far may add nothing, n of them up to n 2^-25 of the
 * row.  A block id outside the pool is left out of every row that would see it.
 * Rows, query_start, errors and requirements as pa_decode_multi.  As there, a
 * NaN among the values of a run's new tokens may also reach rows of the run that
 * stand before it (the product with a weight of 0); every other row past a
 * row's limit, and past the sequence, may hold anything.  The result of a row
 * is the same for every physical placement of the blocks; its rounding depends
 * on the sizes of the call (how its keys are split).
 */
int pa_decode_multi_fp8(void *out, const void *q, const void *k_cache,
                        const void *v_cache, const float *k_scale,
                        const float *v_scale, const int32_t *block_tables,
                        const int32_t *seq_lens, const int32_t *query_start,
                        int32_t num_seqs, int32_t num_q_rows, int32_t max_query_len,
                        int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                        int64_t num_blocks, int32_t block_size,
                        int32_t max_blocks_per_seq, int64_t q_row_stride,
                        float scale, int32_t dtype, void *stream);

/*
 * FP4 KV cache.
 *
 * What the FP8 cache is to the 16-bit one ("vLLM: Architecture, PagedAttention &
 * Internals", *The knobs that actually matter*, item 5: a smaller cache entry
 * enlarges the effective pool), once more.  An element is an OCP E2M1 code (1 sign,
 * 2 exponent bits with bias 1, 1 fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
 * negatives); every 16 neighbouring elements of a row share an E4M3 scale (its NaN
 * makes all 16 NaN), and a KV head a float scale as in the FP8 cache:
 *     value = E2M1(code) * E4M3(scale of the group) * k_scale[j]   (or v_scale[j]).
 * A tile, the 16 rows of a (block, KV head), is 9 * head_dim contiguous bytes: the
 * codes of row 0, head_dim / 2 bytes with element 2i in the low half of byte i, of
 * row 1 and so on; then the scales of row 0, head_dim / 16 bytes, and so on.
 * k_cache and v_cache are [num_blocks, num_kv_heads, 9, head_dim] bytes.
 *
 * pa_reshape_and_cache_fp4 -- the cache write.  For the 16 elements x of a group of
 * KV head j: y = x / k_scale[j] (rounded to binary32); scale = E4M3(max |y| / 6), the
 * quotient rounded to binary32 and then to nearest, ties to even, saturating at 448;
 * code = E2M1(y / scale), likewise, saturating at 6.  A scale of 0 (max |y| at most
 * 6 * 2^-10) has codes of 0; an infinite y is 6 * 448; a NaN makes its group NaN.
 * Requirements as pa_reshape_and_cache_fp8, and head_dim <= 1024; of two tokens with
 * the same slot a group may get the codes of one and the scale of the other.
 *
 * pa_gather_cache_fp4 -- the rows at the given slots as values: k_out[t] and
 * v_out[t] ([num_tokens, num_kv_heads, head_dim] of `dtype`, strides as for k and
 * v) receive what the cache holds at slot_mapping[t], rounded to binary32 and then
 * to `dtype`.  A negative slot leaves its row as it is, and so does one past the
 * pool, with PA_DEVERR_SLOT.  Requirements as the write.
 */
int pa_reshape_and_cache_fp4(const void *k, const void *v, void *k_cache,
                             void *v_cache, const float *k_scale,
                             const float *v_scale, const int64_t *slot_mapping,
                             int64_t num_tokens, int32_t num_kv_heads,
                             int32_t head_dim, int64_t k_token_stride,
                             int64_t v_token_stride, int64_t num_blocks,
                             int32_t block_size, int32_t dtype, void *stream);

int pa_gather_cache_fp4(void *k_out, void *v_out, const void *k_cache,
                        const void *v_cache, const float *k_scale,
                        const float *v_scale, const int64_t *slot_mapping,
                        int64_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                        int64_t k_token_stride, int64_t v_token_stride,
                        int64_t num_blocks, int32_t block_size, int32_t dtype,
                        void *stream);

/*
 * pa_decode_fp4, pa_decode_partitioned_fp4, pa_decode_multi_fp4 -- pa_decode_fp8,
 * pa_decode_partitioned_fp8 and pa_decode_multi_fp8 over E2M1 caches: arguments,
 * requirements, errors and the rounding of q and of the weights as there (an
 * element's code times its group's scale is exact).  In the workspace of the
 * partitioned form m_part is the level that a partition's weights are relative to,
 * 7 ln 2 to 15 ln 2 below the largest scale * q.k of the partition, and l_part
 * their sum to that level.  Tokens past a sequence's
 * end, NaN scales among them, change nothing; a NaN scale of a value reaches the
 * rows that see its token, and rows of the same run that stand before it.
 */
int pa_decode_fp4(void *out, const void *q, const void *k_cache,
                  const void *v_cache, const float *k_scale, const float *v_scale,
                  const int32_t *block_tables, const int32_t *seq_lens,
                  int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                  int32_t head_dim, int64_t num_blocks, int32_t block_size,
                  int32_t max_blocks_per_seq, int64_t q_seq_stride, float scale,
                  int32_t dtype, void *stream);

int pa_decode_partitioned_fp4(void *out, const void *q, const void *k_cache,
                              const void *v_cache, const float *k_scale,
                              const float *v_scale, const int32_t *block_tables,
                              const int32_t *seq_lens, int32_t num_seqs,
                              int32_t num_heads, int32_t num_kv_heads,
                              int32_t head_dim, int64_t num_blocks,
                              int32_t block_size, int32_t max_blocks_per_seq,
                              int64_t q_seq_stride, float scale, int32_t dtype,
                              int32_t partition_size, int32_t max_seq_len,
                              void *workspace, size_t workspace_bytes,
                              void *stream);

int pa_decode_multi_fp4(void *out, const void *q, const void *k_cache,
                        const void *v_cache, const float *k_scale,
                        const float *v_scale, const int32_t *block_tables,
                        const int32_t *seq_lens, const int32_t *query_start,
                        int32_t num_seqs, int32_t num_q_rows, int32_t max_query_len,
                        int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                        int64_t num_blocks, int32_t block_size,
                        int32_t max_blocks_per_seq, int64_t q_row_stride,
                        float scale, int32_t dtype, void *stream);

/*
 * pa_build_step -- what the other calls of a step read, built on the device from
 * the requests' lengths: "vLLM: Architecture, PagedAttention & Internals", *The free
 * list and the block table* (ceil(n / block_size) blocks a request, a new one only
 * when the next token starts it) and *The forward step in detail* (slot = block *
 * block_size + offset).  For steps whose lengths are on the device, as behind
 * pa_verify_drafts; blocks that requests share are the host block manager's
 * (pa_blocks.h), which gives tables that are complete (no free list here).
 *
 * State, updated in place:
 *   request_tables  int32 [num_requests][request_width], the blocks of each request
 *   request_blocks  int32 [num_requests], how many of them it holds
 *   free_blocks     int32 [free_capacity], free block ids, taken from the end of the
 *                   first free_count[0] (its entries are not changed); both NULL:
 *                   there is nothing to take
 * The step: request_ids int32 [num_seqs], the request that sequence s runs (distinct;
 * NULL: request s); context_lens[s], its tokens in the cache; new_lens[s], its new
 * rows (NULL: one each).  With want = ceil((context + new) / 16), sequence s needs
 * max(want - request_blocks, 0) blocks; sequences are served in order, each if the
 * list still holds what it and those before it need.  Then, for a sequence served,
 *   request_tables[id][held ..] and request_blocks[id] receive its new blocks,
 *   block_tables[s][0 .. want) its blocks (entries behind stay as they are),
 *   seq_lens[s] context + new;
 * and always query_start (int32 [num_seqs + 1], the sums of new_lens), and for row r
 * = query_start[s] + i positions[r] = context + i and slot_mapping[r] (both int64
 * [num_rows]); rows behind the last one get position 0 and slot -1.
 *
 * A sequence not served has seq_lens 0, slots -1 and its request unchanged: the list
 * holds too little (PA_DEVERR_NO_BLOCKS; sequences behind it that need blocks are
 * not served either), or its request id, a length or its rows' place is out of
 * bounds -- context + new past 16 * the narrower table, rows past num_rows -- with
 * PA_DEVERR_SEQ_LEN (query_start stays within num_rows).  A table entry outside
 * [0, num_blocks) gives slot -1 and PA_DEVERR_BLOCK_ID, a free_count outside [0,
 * free_capacity] the latter too.  A request id of -1 pads the batch: it is not served,
 * and nothing is flagged.  With a request named twice no sequence is served
 * (PA_DEVERR_SEQ_LEN).  num_seqs <= 65535, and num_requests <= 2^19 with request_ids.
 * Calls on one state must be ordered by the caller.
 */
int pa_build_step(int32_t *block_tables, int32_t *seq_lens, int32_t *query_start,
                  int64_t *positions, int64_t *slot_mapping,
                  int32_t *request_tables, int32_t *request_blocks,
                  const int32_t *request_ids, const int32_t *context_lens,
                  const int32_t *new_lens, const int32_t *free_blocks,
                  int32_t *free_count, int32_t num_seqs, int32_t num_requests,
                  int32_t max_blocks_per_seq, int32_t request_width,
                  int64_t num_rows, int64_t free_capacity, int64_t num_blocks,
                  int32_t block_size, void *stream);

/*
 * pa_trim_blocks -- blocks past a length go back to the free list: after rejected
 * drafts (keep_lens = the accepted length) or when a request ends (0).  For each
 * named request (request_ids as above) the blocks past ceil(keep_lens[s] / 16) are
 * put behind the first free_count[0] entries of free_blocks so that the first
 * sequence's first one is taken next -- a step built and trimmed to its context
 * leaves the list as it was -- and request_blocks and free_count follow.  A bad id or
 * length changes nothing of its request (PA_DEVERR_SEQ_LEN; an id of -1 pads, without
 * it); if a request is named twice (PA_DEVERR_SEQ_LEN) or the blocks do not fit into
 * free_capacity (PA_DEVERR_BLOCK_ID) nothing changes at all.
 */
int pa_trim_blocks(const int32_t *request_tables, int32_t *request_blocks,
                   const int32_t *request_ids, const int32_t *keep_lens,
                   int32_t *free_blocks, int32_t *free_count, int32_t num_seqs,
                   int32_t num_requests, int32_t request_width,
                   int64_t free_capacity, int32_t block_size, void *stream);

/*
 * pa_process_logits -- logits made ready for sampling, or the target_probs of
 * pa_verify_drafts.  Rows as there: sequence s owns rows query_start[s] ..
 * query_start[s+1]-1 of logits ([num_rows][vocab_size] of `dtype`) and out (of `dtype`
 * or PA_F32), rows contiguous with strides of any alignment.
 *
 * For token v of row i of sequence s, with x its logit, c the times v occurs in the
 * output so far -- history[s][prompt_lens[s] .. history_lens[s]), which ends with the
 * token of the sequence's first row, and tokens[query_start[s] + 1 .. + i], the drafts
 * before the row's prediction -- and seen if c > 0 or v is among history[s][0 ..
 * prompt_lens[s]):
 *   x <- x / repetition[s] if x > 0, else x * repetition[s]        (seen only)
 *   x <- x - frequency[s] * c - presence[s] * [c > 0]
 *   x <- x + the values of every entry e of bias_start[s] .. bias_start[s+1]-1 with
 *        bias_tokens[e] = v
 *   x <- -inf if bit v % 32 of allowed[row][v / 32] is 0 (whatever x was)
 *   x <- x / temperature[s] if that is above 0
 * out receives x, or with probs != 0 softmax(x) over the row; with a temperature
 * not above 0 then a 1 at the first largest x and 0 elsewhere.  A row that allows
 * nothing is 0 throughout (-inf without probs); a NaN or an infinity of the largest
 * x makes a row of probabilities NaN.  Arithmetic is fp32, rounded once at the end
 * (divisions as products with the fp32 reciprocal).
 *
 * NULL for repetition, frequency, presence or temperature is 1, 0, 0 or 1; history,
 * tokens, bias_start and allowed may be NULL (nothing there); prompt_lens NULL is 0.
 * history is int32 [num_seqs][history_stride], bias_start int32 [num_seqs + 1] into
 * num_bias entries, allowed int32 rows of allowed_stride words.  Token ids outside
 * the vocabulary are left out, with PA_DEVERR_TOKEN; lengths or bias ranges out of
 * bounds are clamped or left out, with PA_DEVERR_SEQ_LEN.  Rows of no sequence stay as
 * they are.  out may be logits itself with the same type and stride, and may not
 * overlap it otherwise.  vocab_size <= 2^30.
 */
int pa_process_logits(void *out, const void *logits, const int32_t *query_start,
                      const int32_t *tokens, const int32_t *history,
                      const int32_t *prompt_lens, const int32_t *history_lens,
                      const float *repetition, const float *frequency,
                      const float *presence, const int32_t *bias_start,
                      const int32_t *bias_tokens, const float *bias_values,
                      const int32_t *allowed, const float *temperature,
                      int32_t num_seqs, int32_t num_rows, int32_t vocab_size,
                      int64_t logits_row_stride, int64_t out_row_stride,
                      int64_t history_stride, int64_t allowed_stride,
                      int64_t num_bias, int32_t probs, int32_t dtype,
                      int32_t out_dtype, void *stream);

/*
 * pa_decode_cascade_workspace_size -- bytes of workspace pa_decode_cascade
 * needs for these sizes (fp32 partial results in the layout documented at
 * pa_decode_partitioned_workspace_size, with one partition per prefix chunk
 * followed by 512-token partitions of each sequence's own blocks).  Returns
 * 0 on invalid sizes (num_prefix_blocks must be positive).
 */
size_t pa_decode_cascade_workspace_size(int32_t num_seqs, int32_t num_heads,
                                        int32_t head_dim,
                                        int32_t num_prefix_blocks,
                                        int32_t max_blocks_per_seq);

/*
 * pa_decode_cascade -- decode for a batch whose sequences all begin with
 * the same physical blocks (a shared prompt: "vLLM: High-Throughput Serving
 * with PagedAttention", *How PagedAttention shares memory*; "vLLM:
 * Architecture, PagedAttention & Internals", *Prefix caching: reuse KV
 * across requests*), reading the shared blocks once per KV head instead of
 * once per sequence.
 *
 * Sequence s attends over 16 * num_prefix_blocks prefix tokens, held in the
 * physical blocks prefix_blocks[0 .. num_prefix_blocks) (int32, device),
 * followed by seq_lens[s] tokens of its own, held in block_tables[s][0 ..].
 * The result equals pa_decode over the concatenated table
 * (prefix_blocks ++ block_tables[s]) with seq_len 16 * num_prefix_blocks +
 * seq_lens[s].  The caller states the sharing (the block manager knows which
 * leading blocks a batch shares); nothing here compares tables.
 *
 * Work: the prefix is cut into chunks; per (chunk, KV head) the query heads
 * of all sequences, 128 (sequence, head) rows at a time, are multiplied
 * against the chunk's keys and values on the tensor cores (tcgen05); each
 * sequence's own blocks are decoded as 512-token split-KV partitions; a last
 * kernel merges every (sequence, head)'s partials by log-sum-exp.  Three
 * launches on `stream`.
 *
 * Requirements as pa_decode, plus: dtype PA_BF16 or PA_F16 (PA_F32:
 * PA_ERR_UNSUPPORTED when num_prefix_blocks > 0), q rows and out 16-byte
 * aligned, workspace_bytes >= pa_decode_cascade_workspace_size(...) with a
 * 256-byte aligned workspace.  num_prefix_blocks == 0 is pa_decode (no
 * workspace needed).  A prefix block id outside the pool is skipped and
 * flagged PA_DEVERR_BLOCK_ID; a seq_len past max_blocks_per_seq * 16 is
 * clamped and flagged PA_DEVERR_SEQ_LEN.
 */
int pa_decode_cascade(void *out, const void *q, const void *k_cache,
                      const void *v_cache, const int32_t *prefix_blocks,
                      int32_t num_prefix_blocks, const int32_t *block_tables,
                      const int32_t *seq_lens, int32_t num_seqs,
                      int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                      int64_t num_blocks, int32_t block_size,
                      int32_t max_blocks_per_seq, int64_t q_seq_stride,
                      float scale, int32_t dtype, void *workspace,
                      size_t workspace_bytes, void *stream);

/*
 * pa_decode_partitioned_noalloc -- pa_decode_partitioned without a caller
 * workspace, for callers that cannot allocate device memory where they
 * decode (for example while another stream is being captured into a CUDA
 * graph, under an allocator that forbids allocation after start-up, or in a
 * plug-in whose host program owns all device memory).  It is an addition of
 * this library with no counterpart on the reference pages.
 *
 * Same arguments, result and requirements as pa_decode_partitioned, minus
 * `workspace` and `workspace_bytes`: the partition workspace is a fixed
 * array of PA_NOALLOC_SCRATCH_BYTES compiled into the library, which every
 * GPU that loads the library holds until the process exits.  Problems whose
 * pa_decode_partitioned_workspace_size(...) exceeds that size are rejected
 * with PA_ERR_WORKSPACE before anything is launched.  Nothing is allocated
 * or freed (no cudaMalloc, cudaFree or allocating library routine).
 *
 * The arguments are checked in the same order, and bad ones refused with
 * the same status, as by pa_decode_partitioned.
 *
 * The first call on a device looks up the array's device address (with that
 * device current) and caches it; make that first call before any stream
 * capture.  The cached address belongs to the CUDA context it was looked up
 * in: after cudaDeviceReset (or anything else that destroys the device's
 * primary context) it is stale, and this entry point must not be called
 * again on that device in the same process.  All calls on a device share the
 * one array, which keeps whatever the last call left in it.  Every entry a
 * call reads is first written by the same call, so nothing needs clearing --
 * except after PA_DEVERR_TIMEOUT, when the output is undefined and may mix in
 * an earlier call's partials (see pa_decode_partitioned).  Calls whose
 * kernels may overlap on the GPU -- on different streams, or from several
 * host threads -- race on the array and must be serialised by the caller.
 */
#define PA_NOALLOC_SCRATCH_BYTES (32u << 20)

int pa_decode_partitioned_noalloc(void *out, const void *q, const void *k_cache,
                                  const void *v_cache, const int32_t *block_tables,
                                  const int32_t *seq_lens, int32_t num_seqs,
                                  int32_t num_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int64_t num_blocks,
                                  int32_t block_size, int32_t max_blocks_per_seq,
                                  int64_t q_seq_stride, float scale, int32_t dtype,
                                  int32_t partition_size, int32_t max_seq_len,
                                  void *stream);

/* Human-readable text of a pa_status (static storage). */
const char *pa_status_string(int status);

/*
 * pa_device_error -- read the sticky device error word of the current device
 * into *flags (PA_DEVERR_* bits) and clear it when `clear` is non-zero.
 * Synchronises the device first.  Returns PA_OK or PA_ERR_CUDA.
 */
int pa_device_error(uint32_t *flags, int clear);

/*
 * pa_test_stall_next_decode -- test hook for the kernels' bounded waits.  The
 * next decode call (any pa_decode* entry point, from any host thread) makes
 * the first copy of every warp of its persistent kernel expect 16 bytes more
 * than it delivers -- in the long runs of pa_decode_multi_fp8 and _fp4, the first keys of
 * every thread block never count as arrived -- so the wait for it runs out at its
 * 1 s limit: the kernel sets PA_DEVERR_TIMEOUT, waits (bounded) for its copies in
 * flight and returns, leaving that call's output incomplete (the call takes ~2 s).
 * The context stays usable.  For tests of the error path only.  Returns PA_OK.
 */
int pa_test_stall_next_decode(void);

/* ABI version of this header (increments when the signature or the meaning of a
 * declared function changes).  Additions raised it up to 4, and no longer do:
 * pa_rope_and_cache, pa_rope_and_cache_fp8, pa_decode_multi_fp8,
 * pa_verify_drafts, the *_fp4 functions, pa_build_step, pa_trim_blocks and
 * pa_process_logits came to version 4, so a loader that may meet an older library
 * looks these up by name. */
int pa_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
