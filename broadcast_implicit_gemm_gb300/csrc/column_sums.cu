// column_sums.cu -- the last step of sums over all rows (column_sums.cuh).  A block
// has 32 columns, whose rows its eight warps share; the rows lie in L2, where the
// kernel before left them.
#include "column_sums.cuh"

#include "internal.h"
#include "ptx.cuh"

namespace bigemm {

namespace {

__global__ void __launch_bounds__(256) column_sums_kernel(const ColumnSums a)
{
    griddep_enter();
    __shared__ float total[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long c = (long long)blockIdx.x * 32 + lane;
    const float *from = a.from[blockIdx.y] + c;
    float v = 0.f;
    if (c < a.cols) {
#pragma unroll 4
        for (int p = warp; p < a.parts; p += 8) v += from[p * a.cols];
    }
    total[warp][lane] = v;
    __syncthreads();
    if (warp > 0 || c >= a.cols) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) v += total[w][lane];
    a.out[blockIdx.y][c] = v;
}

}  // namespace

cudaError_t launch_column_sums(const ColumnSums &a, cudaStream_t stream)
{
    ProfScope prof("column_sums", stream);
    return launch_pdl(column_sums_kernel, dim3((unsigned)((a.cols + 31) / 32), (unsigned)a.count), dim3(256), 0, stream, a);
}

}  // namespace bigemm
