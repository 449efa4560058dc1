// pa_internal.h -- declarations shared by the translation units of the
// library (not part of the public ABI).
#pragma once

#include <cuda.h>   // CUtensorMap (a plain 128-byte descriptor)
#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

// Kernels that let a following decode start early (they call
// launch_dependents()) keep the shared-memory carveout the decode needs:
// an SM cannot change its L1 / shared split while one of their blocks is
// resident, and a decode block that cannot be placed would wait for that.
// Set once per kernel (and per process: the attribute is the function's).
template <auto Kernel>
inline void prefer_shared_carveout() {
    static const bool done = [] {
        cudaFuncSetAttribute(Kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             (int)cudaSharedmemCarveoutMaxShared);
        return true;
    }();
    (void)done;
}

struct DecodeParams;
struct MergeParams;

// per storage type: cluster-split decode, persistent decode (whole sequences
// or partitions) and the partition merge; D in {64,128}, G in {1,2,4,8}.
// cudaErrorNotSupported: shape not built (or too many sequences for the
// persistent kernel's in-block sort).
cudaError_t decode_split_f32(const DecodeParams &p, int D, int G, dim3 grid, int splits,
                             cudaStream_t st);
cudaError_t decode_split_bf16(const DecodeParams &p, int D, int G, dim3 grid, int splits,
                              cudaStream_t st);
cudaError_t decode_split_f16(const DecodeParams &p, int D, int G, dim3 grid, int splits,
                             cudaStream_t st);
cudaError_t decode_persistent_f32(const DecodeParams &p, int D, int G, bool partial,
                                  long long unit_bound, int cluster, cudaStream_t st);
cudaError_t decode_persistent_bf16(const DecodeParams &p, int D, int G, bool partial,
                                   long long unit_bound, int cluster, cudaStream_t st);
cudaError_t decode_persistent_f16(const DecodeParams &p, int D, int G, bool partial,
                                  long long unit_bound, int cluster, cudaStream_t st);
// multi-token queries (16-bit storage only)
cudaError_t decode_multi_bf16(const DecodeParams &p, int D, int G, long long unit_bound,
                              int cluster, cudaStream_t st);
cudaError_t decode_multi_f16(const DecodeParams &p, int D, int G, long long unit_bound,
                             int cluster, cudaStream_t st);
// the rows of sequences with many (token, head) rows: groups of 64 rows per block
cudaError_t prefill_bf16(const DecodeParams &p, int D, int G, int groups, cudaStream_t st);
cudaError_t prefill_f16(const DecodeParams &p, int D, int G, int groups, cudaStream_t st);
constexpr int PREFILL_GROUP_ROWS = 64;     // rows of one prefill block (= its minimum)
constexpr int PREFILL_TC_ROWS = 128;      // rows of one item of the tcgen05 prefill kernel
// tmap_q: q [num_q_rows][H][D] as the 3-D tensor (D, H, rows) in boxes of
// 64 elements x G heads x 128 / G tokens with the 128-byte swizzle
cudaError_t prefill_tc_bf16(const DecodeParams &p, const CUtensorMap &tmap_q, int D, int G,
                            int groups, cudaStream_t st);
cudaError_t prefill_tc_f16(const DecodeParams &p, const CUtensorMap &tmap_q, int D, int G,
                           int groups, cudaStream_t st);
cudaError_t merge_f32(const MergeParams &p, int num_seqs, cudaStream_t st);
cudaError_t merge_bf16(const MergeParams &p, int num_seqs, cudaStream_t st);
cudaError_t merge_f16(const MergeParams &p, int num_seqs, cudaStream_t st);

// cache write
cudaError_t reshape_and_cache(const void *k, const void *v, void *k_cache, void *v_cache,
                              const int64_t *slot_mapping, int64_t num_tokens,
                              int num_kv_heads, int row_bytes, int64_t k_tok_stride_bytes,
                              int64_t v_tok_stride_bytes, int64_t num_slots,
                              cudaStream_t st);

// FP8 (E4M3) cache write; src_dtype 0 f32, 1 bf16, 2 f16; strides in elements
cudaError_t reshape_and_cache_fp8(const void *k, const void *v, void *k_cache, void *v_cache,
                                  const int64_t *slot_mapping, int64_t num_tokens,
                                  int num_kv_heads, int head_dim, int64_t k_tok_stride,
                                  int64_t v_tok_stride, int64_t num_slots, int src_dtype,
                                  const float *k_scale, const float *v_scale,
                                  cudaStream_t st);

// the cache write with per-head norms and the rotation by position in front
// (pa_rope.cu); k_scale set: E4M3 caches.  Strides in elements.
struct RopeParams {
    void *q_out;
    const void *q, *k, *v;
    void *k_cache, *v_cache;
    const float *k_scale, *v_scale;           // [num_kv_heads], or nullptr
    const void *q_weight, *k_weight;          // [head_dim], or nullptr: no norm
    const float *rope_table;                  // [num_positions][rot_dim]: cos, then sin
    const int64_t *positions, *slot_mapping;  // [num_tokens]
    int64_t num_tokens, num_positions, num_slots;
    int64_t q_stride, q_out_stride, k_stride, v_stride;
    float eps;
    int num_heads, num_kv_heads, head_dim, rot_dim, interleaved;
    int parts, part_iters;                    // warps per token, iterations of each
    unsigned int *err;
};
cudaError_t rope_and_cache(const RopeParams &p, int dtype, cudaStream_t st);

// rows written into E2M1 caches, or read back (pa_fp4.cu); strides in elements, of
// k and v or of k_out and v_out
struct Fp4RowsParams {
    const void *k, *v;
    void *k_out, *v_out;
    void *k_cache, *v_cache;
    const float *k_scale, *v_scale;           // [num_kv_heads]
    const int64_t *slot_mapping;              // [num_tokens]
    int64_t num_tokens, num_slots, k_stride, v_stride;
    int num_kv_heads, head_dim;
    unsigned num_items;                       // of a launch: groups of 16 of its tokens' rows
    unsigned int *err;
};
cudaError_t reshape_and_cache_fp4(const Fp4RowsParams &p, int dtype, cudaStream_t st);
cudaError_t gather_cache_fp4(const Fp4RowsParams &p, int dtype, cudaStream_t st);

// block tables and maps of a step, and blocks given back (pa_step.cu)
struct StepParams {
    int32_t *block_tables, *seq_lens, *query_start;   // [num_seqs][max_blocks], [num_seqs], [num_seqs + 1]
    int64_t *positions, *slot_mapping;        // [num_rows]
    int32_t *request_tables, *request_blocks; // [num_requests][request_width], [num_requests]
    const int32_t *request_ids;               // [num_seqs], or nullptr: s
    const int32_t *context_lens, *new_lens;   // [num_seqs]; new_lens nullptr: one each
    int32_t *free_blocks, *free_count;        // [free_capacity], [1]; nullptr: nothing to take
    int64_t num_blocks, num_rows, free_capacity;
    int num_seqs, num_requests, max_blocks, request_width;
    unsigned int *err;
};
cudaError_t build_step(const StepParams &p, cudaStream_t st);
cudaError_t trim_blocks(const StepParams &p, cudaStream_t st);

// logits made ready for sampling or verification (pa_logits.cu); strides in elements
struct LogitsParams {
    void *out;
    const void *logits;
    const int32_t *query_start, *tokens;      // [num_seqs + 1], [num_rows] or nullptr
    const int32_t *history, *prompt_lens, *history_lens;
    const float *repetition, *frequency, *presence;   // [num_seqs], nullptr: neutral
    const int32_t *bias_start, *bias_tokens;  // [num_seqs + 1], [num_bias]
    const float *bias_values;
    const uint32_t *allowed;                  // [num_rows] rows of bits, or nullptr
    const float *temperature;                 // [num_seqs], nullptr: 1
    int64_t logits_stride, out_stride, history_stride, allowed_stride, num_bias;
    int num_seqs, num_rows, vocab, probs;
    int run;                                  // elements of a block's run, at most
    unsigned int *err;
};
cudaError_t process_logits_f32(const LogitsParams &p, int out_dtype, cudaStream_t st);
cudaError_t process_logits_bf16(const LogitsParams &p, int out_dtype, cudaStream_t st);
cudaError_t process_logits_f16(const LogitsParams &p, int out_dtype, cudaStream_t st);

// verification of drafted tokens (pa_verify.cu); strides in elements
struct VerifyParams {
    int32_t *out_tokens, *num_accepted;       // [num_seqs][max_query_len], [num_seqs]
    const void *target, *draft;               // rows of the vocabulary; draft may be nullptr
    const int32_t *tokens;                    // [num_rows]
    const float *accept_u, *sample_u;         // [num_rows], [num_seqs]
    const int32_t *query_start;               // [num_seqs + 1]
    int64_t target_stride, draft_stride;
    int num_seqs, num_rows, max_query_len, vocab;
    unsigned int *err;
};
cudaError_t verify_drafts(const VerifyParams &p, int dtype, cudaStream_t st);

// the rows of long multi-token runs over E4M3 caches (pa_prefill_f8.cuh)
constexpr int PREFILL_F8_ROWS = 256;       // rows of one item
// Runs of at least so many rows go there.  Two 16-row tiles (20 rows, 4 heads a
// group) read their keys twice on the persistent kernel and are still faster
// there in a batch (32 sequences x 6000 keys 184 us against 245, 128 x 500: 81
// against 112); with three tiles (36 rows) it is 268 against 246 over 6000 keys
// and 111 against 114 over 500, and a single sequence is even (36.6 against 35).  The kernel looks its
// items up by walking the sequences when there are more than 256.
constexpr int prefill_f8_min_rows(int num_seqs) { return num_seqs <= 256 ? 33 : PREFILL_GROUP_ROWS; }
cudaError_t prefill_f8_bf16(const DecodeParams &p, int D, int G, int groups, cudaStream_t st);
cudaError_t prefill_f8_f16(const DecodeParams &p, int D, int G, int groups, cudaStream_t st);

// multi-token queries over E4M3 caches (q and out bf16 / f16)
cudaError_t decode_multi_fp8_bf16(const DecodeParams &p, int D, int G, long long unit_bound,
                                  int cluster, cudaStream_t st);
cudaError_t decode_multi_fp8_f16(const DecodeParams &p, int D, int G, long long unit_bound,
                                 int cluster, cudaStream_t st);

// persistent decode over E4M3 caches (q and out bf16 / f16); partial as above
cudaError_t decode_fp8_bf16(const DecodeParams &p, int D, int G, bool partial,
                            long long unit_bound, int cluster, cudaStream_t st);
cudaError_t decode_fp8_f16(const DecodeParams &p, int D, int G, bool partial,
                           long long unit_bound, int cluster, cudaStream_t st);

// the same over E2M1 caches with a scale for every 16 elements (pa_fp4.cuh)
cudaError_t decode_fp4_bf16(const DecodeParams &p, int D, int G, bool partial,
                            long long unit_bound, int cluster, cudaStream_t st);
cudaError_t decode_fp4_f16(const DecodeParams &p, int D, int G, bool partial,
                           long long unit_bound, int cluster, cudaStream_t st);
cudaError_t decode_multi_fp4_bf16(const DecodeParams &p, int D, int G, long long unit_bound,
                                  int cluster, cudaStream_t st);
cudaError_t decode_multi_fp4_f16(const DecodeParams &p, int D, int G, long long unit_bound,
                                 int cluster, cudaStream_t st);
cudaError_t prefill_f4_bf16(const DecodeParams &p, int D, int G, int groups, cudaStream_t st);
cudaError_t prefill_f4_f16(const DecodeParams &p, int D, int G, int groups, cudaStream_t st);

// block copies for copy-on-write: every (src, dst) pair of `mapping`, in every cache
constexpr int COPY_MAX_CACHES = 256;
struct CopyParams {
    unsigned char *caches[COPY_MAX_CACHES];   // device bases, 16-byte aligned
    const int64_t *mapping;                   // device [num_pairs][2]
    int64_t num_pairs, num_blocks, block_bytes;
    int num_caches;
    unsigned int *err;
};
cudaError_t copy_blocks(const CopyParams &p, cudaStream_t st);

// device error word
cudaError_t device_error_ptr(unsigned int **out);
cudaError_t read_device_error(unsigned int *flags, bool clear);
int sm_count_of_current_device();

}  // namespace pa
