// pa_logits_bf16.cu -- bf16 logits (pa_logits.cuh)
#include "pa_logits.cuh"

namespace pa {

cudaError_t process_logits_bf16(const LogitsParams &p, int out_dtype, cudaStream_t st) {
    return out_dtype == 0 ? launch_logits<__nv_bfloat16, float>(p, st) : launch_logits<__nv_bfloat16, __nv_bfloat16>(p, st);
}

}  // namespace pa
