// matmul_gated.cuh -- a gated layer's two products as their kernels see them:
//
//   g = x w_gate^T + bias_gate;  u = x w_up^T + bias_up;  out = act(g) u
//
// The sums are fp32 and out is rounded once: g and u are not rounded on the way to
// it, and once each where they are kept for the gradients.
#pragma once
#include "matmul.cuh"

namespace bigemm {

// N: of each product.  The base's w, ldw and bias are the gate's.
struct GatedArgs : MatmulArgs {
    const void *w_up;
    long long ldw_up;
    const float *bias_up;
    bool vec_bias_up;
    void *gate, *up;                 // [M,N] each or null: g and u
    long long ldgate, ldup;
    bool vec_gate, vec_up;           // rows start on 16-byte boundaries
};

// Many tokens (matmul_gated.cu): 256 tokens by 128 channels of each product.
struct GatedMaps {
    CUtensorMap x, w[2], out, kept[2];
};
cudaError_t launch_gated_many(const GatedArgs &a, const GatedMaps &maps, int sms, cudaStream_t stream);

// Few tokens (matmul_few.cu): 64 channels of each product by cut.bn tokens.
cudaError_t launch_gated_few(const GatedArgs &a, FewCut cut, const CUtensorMap &map_w, const CUtensorMap &map_up,
                             const CUtensorMap &map_x, cudaStream_t stream);

}  // namespace bigemm
