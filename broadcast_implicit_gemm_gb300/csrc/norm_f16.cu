// norm_f16.cu -- the root-mean-square norm of fp16 rows (norm.cuh).
#include "norm.cuh"

namespace bigemm {

cudaError_t launch_norm_f16(const NormArgs &a, int form, bool vec, int sms, cudaStream_t s)
{
    return launch_norm_type<__half>(a, form, vec, sms, s);
}

}  // namespace bigemm
