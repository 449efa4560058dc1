// pa_fp4_multi_bf16.cu -- persistent kernel for multi-token queries over E2M1 caches,
// bf16 queries and outputs.
#include "pa_internal.h"
#include "pa_persistent.cuh"

namespace pa {

cudaError_t decode_multi_fp4_bf16(const DecodeParams &p, int D, int G, long long unit_bound,
                                  int cluster, cudaStream_t st) {
    return dispatch_persistent<__nv_bfloat16, MODE_MULTI, e2m1>(p, D, G, unit_bound, cluster, st);
}

}  // namespace pa
