// norm_back_bf16.cu -- the norms' gradients of bf16 rows (norm_back.cuh).
#include "norm_back.cuh"

namespace bigemm {

cudaError_t launch_norm_back_bf16(const NormBackArgs &a, bool layer, bool vec, float *rstds, int parts, cudaStream_t s)
{
    return launch_norm_back_type<__nv_bfloat16>(a, layer, vec, rstds, parts, s);
}

}  // namespace bigemm
