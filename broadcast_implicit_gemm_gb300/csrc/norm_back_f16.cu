// norm_back_f16.cu -- the norms' gradients of f16 rows (norm_back.cuh).
#include "norm_back.cuh"

namespace bigemm {

cudaError_t launch_norm_back_f16(const NormBackArgs &a, bool layer, bool vec, float *rstds, int parts, cudaStream_t s)
{
    return launch_norm_back_type<__half>(a, layer, vec, rstds, parts, s);
}

}  // namespace bigemm
