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
#include "fastdiv.h"
#include "matmul.cuh"

namespace bigemm {

// A result's units: tiles of 256 x 256 sums, each in `split` shares of its summed axis of
// `blocks` blocks of 64.  Divisors are the launch's: a unit of one block (few tokens) is
// done in less time than divisions take (64 x 8192 x 8192: 60 us with some, 73 with more).
struct UnitGrid {
    int m, n, split, blocks;
    int whole, rest;                 // blocks by split
    FastDiv tiles, group, shares;    // by m * n, 8 * n and split
};
constexpr int kMostShares = 32768;   // rest times a share's number has 31 bits
inline UnitGrid make_unit_grid(int m, int n, int split, int blocks)
{
    return {m, n, split, blocks, blocks / split, blocks % split, make_fastdiv((uint32_t)(m * n)), make_fastdiv(8u * (uint32_t)n),
            make_fastdiv((uint32_t)split)};
}
// A share's first block (the number of blocks for share `split`).
BIGEMM_FD_HD int share_start(const UnitGrid &g, int share)
{
    return g.whole * share + (int)fd_div((uint32_t)(g.rest * share), g.shares);
}

struct BackArgs {
    int M, N, K;                     // tokens, output channels (of each product), input channels
    int dt;                          // bigemm_dtype of everything
    int count;                       // products: 1 or 2
    int n_blocks;                    // blocks of one d's channels
    UnitGrid to_dx, to_dw;           // dw: of both products, one below the other
    int dw_m;                        // tiles of one
    bool dw_first;                   // the walk's first units are dw's (the longer ones)
    BackWalk walk;
    void *dx, *dw[2];
    long long lddx, lddw[2];
    bool dx_rows, dw_rows[2];        // by TMA
    const void *dout;                // sums of its columns go to `sums`, if that is not null
    long long ldd;
    float *sums;
    unsigned long long timeout_ns;
    int *err;
};

// Operands as boxes of 64 x 64, outputs of 32 rows by 64; part: shares of dx, [split][M][K]
// fp32, and of dw, [count * dw_split][N][K], 32 by 32.
struct BackMaps {
    CUtensorMap d[2], w[2], x, dx, dw[2], part[2];
};
cudaError_t launch_matmul_back(const BackArgs &a, const BackMaps &maps, int pairs, cudaStream_t stream);

// Results from their shares, [split][rows][pitch] fp32 each, added in their order: up to
// three in a launch.
struct JoinResult {
    const float *part;
    void *out;
    long long ld;
    int rows, split;
    bool vec;                        // rows start on 8-byte boundaries
};
constexpr int kJoinMost = 3;
struct JoinArgs {
    JoinResult result[kJoinMost];
    int count, cols;
    long long pitch, runs;           // of 128 columns: of a row
    long long items[kJoinMost];      // runs up to the end of each result
};
cudaError_t launch_back_join(JoinArgs &a, int dt, cudaStream_t stream);

// Before the products (gate_back.cu): d_g and d_u, rounded to the operands' type, and
// sums over runs of rows where `sums` is not null: [runs][sum_pitch(N)] of d_g, the
// same of d_u.
// Or, for a plain product of more than kSumsBeside tokens, the sums of d alone.  Those of
// fewer are taken by two warps of each block that the products leave idle, a column a lane
// (100 x 4096 x 4096 f16 21.4 us, 21.3 without sums, 6 more with a launch for them;
// 64 x 4096 x 256 8.0, 7.9 and 9.7; 128 x 4096 x 256 9.5, 9.1 and 11.6; more rows take
// those warps longer than the launch: 256 x 4096 x 256 12.8 in a launch, 24 beside).
struct GateBackArgs {
    int M, N, runs;
    int act;                         // -1: sums of dout alone
    const void *dout, *gate, *up;
    long long ldd, ldg, ldu, pitch;
    void *dg, *du;                   // rows of `pitch` elements, on the 16-byte grid
    float *sums[2];
};
constexpr int kSumsBeside = 128;
constexpr int kGateColumns = 256;    // of a block
constexpr int kGateBeside(bool vec) { return vec ? 2 : 3; }      // blocks that an SM's registers hold
cudaError_t launch_gate_back(const GateBackArgs &a, int dt, bool vec, cudaStream_t stream);

}  // namespace bigemm
