// pa_logits_f32.cu -- f32 logits (pa_logits.cuh)
#include "pa_logits.cuh"

namespace pa {

cudaError_t process_logits_f32(const LogitsParams &p, int, cudaStream_t st) {
    return launch_logits<float, float>(p, st);
}

}  // namespace pa
