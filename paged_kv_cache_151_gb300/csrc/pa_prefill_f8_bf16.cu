// pa_prefill_f8_bf16.cu -- prefill kernel for multi-token queries with many rows per
// sequence over E4M3 caches, bf16 queries and outputs.
#include "pa_internal.h"
#include "pa_prefill_f8.cuh"

namespace pa {

cudaError_t prefill_f8_bf16(const DecodeParams &p, int D, int G, int groups, cudaStream_t st) {
    return dispatch_prefill_f8<__nv_bfloat16>(p, D, G, groups, st);
}

}  // namespace pa
