// column_sums.cu -- the last step of sums over all rows (column_sums.cuh).  A block has
// 32 columns, four a lane, and takes 64 rows at once, eight such turns' loads in flight:
// the rows lie in L2, where the kernel before left them, and latency and an even share
// for all SMs are what counts (456 rows of 2 x 2049 columns: 128 columns a block 5 us).
#include "column_sums.cuh"

#include "internal.h"
#include "ptx.cuh"

namespace bigemm {

namespace {

constexpr int kSumWarps = 16;

__global__ void __launch_bounds__(kSumWarps * 32) column_sums_kernel(const ColumnSums a)
{
    griddep_enter();
    __shared__ float4 total[kSumWarps][8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long c = (long long)blockIdx.x * 32 + (lane & 7) * 4, pitch = sum_pitch(a.cols) / 4;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (c < a.cols) {
        const float4 *from = reinterpret_cast<const float4 *>(a.from[blockIdx.y] + c);
#pragma unroll 8
        for (int p = warp * 4 + (lane >> 3); p < a.parts; p += kSumWarps * 4) {
            const float4 w = from[p * pitch];
            v[0] += w.x, v[1] += w.y, v[2] += w.z, v[3] += w.w;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] += __shfl_xor_sync(0xffffffffu, v[i], 8);
        v[i] += __shfl_xor_sync(0xffffffffu, v[i], 16);
    }
    if (lane < 8) total[warp][lane] = make_float4(v[0], v[1], v[2], v[3]);
    __syncthreads();
    // a thread a column
    const long long col = (long long)blockIdx.x * 32 + threadIdx.x;
    if (threadIdx.x >= 32 || col >= a.cols) return;
    const float *of = reinterpret_cast<const float *>(total) + threadIdx.x;
    float sum = of[0];
#pragma unroll
    for (int w = 1; w < kSumWarps; ++w) sum += of[w * 32];
    a.out[blockIdx.y][col] = sum;
}

}  // namespace

cudaError_t launch_column_sums(const ColumnSums &a, cudaStream_t stream)
{
    ProfScope prof("column_sums", stream);
    const dim3 grid((unsigned)((a.cols + 31) / 32), (unsigned)a.count);
    return launch_pdl(column_sums_kernel, grid, dim3(kSumWarps * 32), 0, stream, a);
}

}  // namespace bigemm
