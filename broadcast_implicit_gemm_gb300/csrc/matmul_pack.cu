// matmul_pack.cu -- a matrix product's operands whose rows are off the 16-byte
// grid, copied to rows that are on it, both in one launch.  Bound by memory: a
// warp takes a run of 128 pieces of 16 bytes of a row, four per lane in flight.
#include "matmul.cuh"
#include "unaligned.cuh"

namespace bigemm {

namespace {

__global__ void __launch_bounds__(256) matmul_pack_kernel(const PackArgs a)
{
    griddep_enter();
    constexpr int U = 4;
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    const bool second = item >= a.items0;
    const PackOperand &o = second ? a.op[1] : a.op[0];
    const long long i = second ? item - a.items0 : item;
    const long long row = i / o.runs;
    if (row >= o.rows) return;
    const long long p0 = (i - row * o.runs) * 32 * U + lane;
    const Span span = {o.src, o.src + (o.rows - 1) * o.src_pitch + o.bytes};
    const uint8_t *from = o.src + row * o.src_pitch;
    uint8_t *to = o.dst + row * o.dst_pitch;
    Wide w[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long at = (p0 + 32ll * u) * 16;
        w[u] = wide_load(from + at, 0, (int)max(0ll, min(16ll, o.bytes - at)), span);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const long long at = (p0 + 32ll * u) * 16;
        if (at < o.bytes)
            *reinterpret_cast<uint4 *>(to + at) = wide_take(w[u], 0, (int)min(16ll, o.bytes - at));
    }
}

}  // namespace

cudaError_t launch_matmul_pack(PackArgs &a, cudaStream_t stream)
{
    ProfScope prof("matmul_pack", stream);
    for (PackOperand &o : a.op) o.runs = o.bytes > 2048 ? (o.bytes + 2047) / 2048 : 1;
    a.items0 = a.op[0].rows * a.op[0].runs;
    const long long blocks = (a.items0 + a.op[1].rows * a.op[1].runs + 7) / 8;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_pdl(matmul_pack_kernel, dim3((unsigned)blocks), dim3(256), 0, stream, a);
}

}  // namespace bigemm
