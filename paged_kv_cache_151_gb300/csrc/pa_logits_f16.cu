// pa_logits_f16.cu -- f16 logits (pa_logits.cuh)
#include "pa_logits.cuh"

namespace pa {

cudaError_t process_logits_f16(const LogitsParams &p, int out_dtype, cudaStream_t st) {
    return out_dtype == 0 ? launch_logits<__half, float>(p, st) : launch_logits<__half, __half>(p, st);
}

}  // namespace pa
