// norm_f32.cu -- the root-mean-square norm of 32-bit rows (norm.cuh).
#include "norm.cuh"

namespace bigemm {

cudaError_t launch_norm_f32(const NormArgs &a, int form, bool vec, int sms, cudaStream_t s)
{
    return launch_norm_type<float>(a, form, vec, sms, s);
}

}  // namespace bigemm
