// matmul_host.cuh -- what the matrix products' entry points share on the host: which
// operands TMA can address, tensor maps, and copies of the others.
#pragma once
#include "matmul.cuh"

namespace bigemm {

namespace {

inline long long up(long long a, long long b) { return (a + b - 1) / b; }

inline bool on_grid(const void *p, long long ld, long long size, long long to)
{
    return reinterpret_cast<uintptr_t>(p) % (uintptr_t)to == 0 && (ld * size) % to == 0;
}

constexpr int kMaxSize = 1 << 30;   // indices within a row are in 32 bits, byte offsets in 64

constexpr long long kFar = 1ll << 40;           // TMA: strides below 2^40 bytes

// Whether TMA can address an operand's rows.
inline bool addressable(const void *p, long long ld, long long es) { return on_grid(p, ld, es, 16) && ld * es < kFar; }

inline long long packed_bytes(long long rows, long long cols, long long es) { return up(rows * up(cols * es, 16) * 16, 256) * 256; }

// A row-major matrix as boxes of box_rows rows by box_cols columns.
inline bool box_map(CUtensorMap *map, const void *p, int dt, long long rows, long long cols, long long ld, int box_rows,
                    int box_cols, CUtensorMapSwizzle swizzle)
{
    const uint64_t es = dt == BIGEMM_MXF8 ? 1 : dtype_size(dt);
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
    const uint64_t strides[1] = {(uint64_t)ld * es};
    const uint32_t box[2] = {(uint32_t)box_cols, (uint32_t)box_rows};
    const uint32_t ones[2] = {1, 1};
    const CUtensorMapDataType t = dt == BIGEMM_MXF8  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                  : dt == BIGEMM_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                  : dt == BIGEMM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encode_tiled(map, t, 2, p, dims, strides, box, ones, swizzle);
}

// A row-major operand as boxes of box_rows rows by 128 bytes, 128-byte swizzle.
inline bool operand_map(CUtensorMap *map, const void *p, int dt, long long rows, long long cols, long long ld, int box_rows)
{
    return box_map(map, p, dt, rows, cols, ld, box_rows, dt == BIGEMM_MXF8 ? kRow : kRow / 2, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Operands that TMA cannot address, at most kPackMost, copied to `space` one after the
// other.
struct PackList {
    uint8_t *space;
    PackArgs args = {};
    int count = 0;

    explicit PackList(uint8_t *to) : space(to) {}
    // The copy takes the operand's place.
    void add(const void *&p, long long &ld, long long rows, long long cols, long long es)
    {
        if (addressable(p, ld, es)) return;
        const long long pitch = up(cols * es, 16) * 16;
        args.op[count++] = {static_cast<const uint8_t *>(p), space, rows, ld * es, pitch, cols * es, 0};
        p = space, ld = pitch / es;
        space += packed_bytes(rows, cols, es);
    }
    cudaError_t run(cudaStream_t stream) { return count > 0 ? launch_matmul_pack(args, stream) : cudaSuccess; }
};

}  // namespace

}  // namespace bigemm
