// layernorm_f32.cu -- the layer norm of 32-bit rows (layernorm.cuh).
#include "layernorm.cuh"

namespace bigemm {

cudaError_t launch_layernorm_f32(const LayerNormArgs &a, int form, bool vec, int sms, cudaStream_t s)
{
    return launch_layernorm_type<float>(a, form, vec, sms, s);
}

}  // namespace bigemm
