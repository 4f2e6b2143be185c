// norm_bf16.cu -- the root-mean-square norm of bf16 rows (norm.cuh).
#include "norm.cuh"

namespace bigemm {

cudaError_t launch_norm_bf16(const NormArgs &a, int form, bool vec, int sms, cudaStream_t s)
{
    return launch_norm_type<__nv_bfloat16>(a, form, vec, sms, s);
}

}  // namespace bigemm
