// layernorm_bf16.cu -- the layer norm of bf16 rows (layernorm.cuh).
#include "layernorm.cuh"

namespace bigemm {

cudaError_t launch_layernorm_bf16(const LayerNormArgs &a, int form, bool vec, int sms, cudaStream_t s)
{
    return launch_layernorm_type<__nv_bfloat16>(a, form, vec, sms, s);
}

}  // namespace bigemm
