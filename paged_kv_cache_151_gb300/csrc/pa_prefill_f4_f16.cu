// pa_prefill_f4_f16.cu -- prefill kernel for multi-token queries with many rows per
// sequence over E2M1 caches, f16 queries and outputs.
#include "pa_internal.h"
#include "pa_prefill_f8.cuh"

namespace pa {

cudaError_t prefill_f4_f16(const DecodeParams &p, int D, int G, int groups, cudaStream_t st) {
    return dispatch_prefill_f8<__half, e2m1>(p, D, G, groups, st);
}

}  // namespace pa
