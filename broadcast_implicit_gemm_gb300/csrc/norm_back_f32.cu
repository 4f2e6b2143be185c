// norm_back_f32.cu -- the norms' gradients of 32-bit rows (norm_back.cuh).
#include "norm_back.cuh"

namespace bigemm {

cudaError_t launch_norm_back_f32(const NormBackArgs &a, bool layer, bool vec, float *rstds, int parts, cudaStream_t s)
{
    return launch_norm_back_type<float>(a, layer, vec, rstds, parts, s);
}

}  // namespace bigemm
