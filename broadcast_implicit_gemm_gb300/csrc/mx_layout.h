// mx_layout.h -- where the scale of an MXFP8 matrix's element lies.
//
// Scales are kept in blocks of 128 rows by 128 columns, 512 bytes each, the
// blocks of one block row next to each other.  Within a block, the byte of row
// r and group g is (r % 32) * 16 + (r / 32) * 4 + g: the order in which tensor
// memory takes a block's scales from shared memory in one copy.
//
// Offsets are in 64 bits: four bytes of scales per column of a block row pass
// 2^31 at 2^29 columns.
//
// No CUDA dependency on the host side, so that a plain C++ test can check it.
#pragma once
#include <stdint.h>

#if defined(__CUDACC__)
#define BIGEMM_MX_HD __host__ __device__ __forceinline__
#else
#define BIGEMM_MX_HD inline
#endif

namespace bigemm {

constexpr int kMxGroup = 32;        // elements per scale
constexpr int kMxBlock = 128;       // rows, and columns, per block of scales
constexpr int kMxBlockBytes = 512;

// Byte offset of a row's first scale in a matrix with col_blocks blocks per
// block row.
BIGEMM_MX_HD long long mx_scale_row(long long row, int col_blocks)
{
    const int r = (int)row;
    return (row >> 7) * col_blocks * kMxBlockBytes + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// Byte offset of a group's scale from its row's first one.
BIGEMM_MX_HD long long mx_scale_group(int group) { return (long long)(group >> 2) * kMxBlockBytes + (group & 3); }

BIGEMM_MX_HD long long mx_scale_offset(long long row, int group, int col_blocks)
{
    return mx_scale_row(row, col_blocks) + mx_scale_group(group);
}

}  // namespace bigemm
