// pa_fp8_multi_f16.cu -- persistent kernel for multi-token queries over E4M3
// caches, f16 queries and outputs.
#include "pa_internal.h"
#include "pa_persistent.cuh"

namespace pa {

cudaError_t decode_multi_fp8_f16(const DecodeParams &p, int D, int G, long long unit_bound,
                                 int cluster, cudaStream_t st) {
    return dispatch_persistent<__half, MODE_MULTI, e4m3>(p, D, G, unit_bound, cluster, st);
}

}  // namespace pa
