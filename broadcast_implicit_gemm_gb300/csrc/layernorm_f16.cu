// layernorm_f16.cu -- the layer norm of f16 rows (layernorm.cuh).
#include "layernorm.cuh"

namespace bigemm {

cudaError_t launch_layernorm_f16(const LayerNormArgs &a, int form, bool vec, int sms, cudaStream_t s)
{
    return launch_layernorm_type<__half>(a, form, vec, sms, s);
}

}  // namespace bigemm
