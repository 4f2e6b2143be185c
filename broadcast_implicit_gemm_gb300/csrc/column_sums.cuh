// column_sums.cuh -- the last step of sums over all rows (gradients of weights and
// biases): rows of partial sums, added in their order.
#pragma once
#include <cuda_runtime.h>

namespace bigemm {

// Rows of partial sums are so many elements apart, each on a 16-byte boundary.
__host__ __device__ constexpr long long sum_pitch(long long cols) { return (cols + 3) / 4 * 4; }

// out[i][c] = sum over p < parts of from[i][p * sum_pitch(cols) + c], i < count; zeros where parts = 0.
struct ColumnSums {
    const float *from[2];
    float *out[2];
    int count, parts;
    long long cols;
};
cudaError_t launch_column_sums(const ColumnSums &a, cudaStream_t stream);

}  // namespace bigemm
