// norm_back_bf16.cu -- the norms' gradients of bf16 rows (norm_back.cuh).
#include "norm_back.cuh"

namespace bigemm {

cudaError_t launch_norm_back_bf16(const NormBackArgs &a, bool layer, bool vec, float *rstds, int parts, cudaStream_t s)
{
    return launch_norm_back_type<__nv_bfloat16>(a, layer, vec, rstds, parts, s);
}

// (of 544 to 1024 threads of 64 registers an SM holds one block, so one form stands for all)
int back_clusters(int cluster)
{
    static std::atomic<int> known[64][4];    // by device and the cluster's logarithm
    int dev = 0, log = 0;
    while (log < 3 && 1 << log < cluster) ++log;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 0;
    int most = known[dev][log];
    if (most > 0) return most;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)cluster);
    cfg.blockDim = dim3(kBackCtaCols / kPiece);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto kern = norm_back_kernel<__nv_bfloat16, true, true, kBackCtaCols / kPiece, true, true>;
    if (cudaOccupancyMaxActiveClusters(&most, kern, &cfg) != cudaSuccess) return 0;
    known[dev][log] = most;
    return most;
}

}  // namespace bigemm
