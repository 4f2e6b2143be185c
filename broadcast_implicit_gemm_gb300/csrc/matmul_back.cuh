// matmul_back.cuh -- gradients of a product, and of a gated layer's two, as their
// kernels see them:
//
//   out = x w^T:          dx = d w,                 dw = d^T x
//   out = act(g) u:       d_g = dout u act'(g),     d_u = dout act(g)
//                         dx = d_g w_gate + d_u w_up,  dw_gate = d_g^T x,  dw_up = d_u^T x
//
// with one d for a plain product and two for a gated one.
#pragma once
#include "back_walk.h"
#include "matmul.cuh"

namespace bigemm {

// Units of 256 x 256 sums; of the products' summed axis, blocks of 64.
struct BackArgs {
    int M, N, K;                     // tokens, output channels (of each product), input channels
    int dt;                          // bigemm_dtype of everything
    int count;                       // products: 1 or 2
    int n_blocks, m_blocks;          // of one d's channels, of the tokens
    int dx_m, dx_n, split;           // dx: tiles, and shares of the summed axis that a tile is cut into
    int dw_m, dw_n;                  // dw: tiles of one of them
    BackWalk walk;
    void *dx, *dw[2];
    long long lddx, lddw[2];
    bool dx_rows, dw_rows[2];        // by TMA
    unsigned long long timeout_ns;
    int *err;
};

// Operands as boxes of 64 x 64, outputs of 32 rows by 64; part: dx's shares, [split][M][K]
// fp32, 32 by 32.
struct BackMaps {
    CUtensorMap d[2], w[2], x, dx, dw[2], part;
};
cudaError_t launch_matmul_back(const BackArgs &a, const BackMaps &maps, int pairs, cudaStream_t stream);

// dx from its shares (rows of `pitch` elements), added in their order.
cudaError_t launch_back_join(const float *part, int split, int M, int K, long long pitch, void *dx, long long lddx, int dt,
                             cudaStream_t stream);

// Before the products (gate_back.cu): d_g and d_u, rounded to the operands' type, and
// sums over runs of rows where `sums` is not null: [runs][sum_pitch(N)] of d_g, the
// same of d_u.
// Or, for a plain product, the sums of d alone.
struct GateBackArgs {
    int M, N, runs;
    int act;                         // -1: sums of dout alone
    const void *dout, *gate, *up;
    long long ldd, ldg, ldu, pitch;
    void *dg, *du;                   // rows of `pitch` elements, on the 16-byte grid
    float *sums[2];
};
constexpr int kGateColumns = 256;    // of a block
constexpr int kGateBeside(bool vec) { return vec ? 2 : 3; }      // blocks that an SM's registers hold
cudaError_t launch_gate_back(const GateBackArgs &a, int dt, bool vec, cudaStream_t stream);

}  // namespace bigemm
