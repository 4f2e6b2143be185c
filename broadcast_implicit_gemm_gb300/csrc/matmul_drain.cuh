// matmul_drain.cuh -- what the pair kernels (matmul_many.cu, matmul_pair.cuh) share: the
// walk over their tiles, and the way of 32 x 32 sums from registers to memory.
#pragma once
#include "matmul.cuh"

namespace bigemm {

namespace {

struct Tile {
    int m, n;
};

// Eight tiles along m share a sweep over the tiles along n.
__device__ __forceinline__ Tile tile_in(int m_tiles, int n_tiles, int t)
{
    constexpr int kGroup = 8;
    const int per = kGroup * n_tiles;
    const int g = t / per, r = t - g * per;
    const int rows = min(kGroup, m_tiles - g * kGroup);
    return {g * kGroup + r % rows, r / rows};
}

// 32 rows of WORDS 32-bit words, a lane's row in w, to the warp's staging (two
// buffers of it, where two fit), swizzled as the output's map is: ready for a TMA
// store by lane 0, which commits it as a bulk group.
template <int PER_WARP, int WORDS>
__device__ __forceinline__ const uint8_t *stage_words(uint8_t *stage, int &piece, int lane, const uint32_t (&w)[WORDS])
{
    constexpr int bytes = WORDS * 128;
    static_assert(bytes <= PER_WARP, "the next warp's staging follows");
    constexpr bool two = 2 * bytes <= PER_WARP;
    uint8_t *buf = stage + (two ? (piece & 1) * bytes : 0);
    if (lane == 0) bulk_wait_read<two ? 1 : 0>();
    __syncwarp();
    // rows of 128, 64 or 32 bytes
    const int key = WORDS == 32 ? lane & 7 : WORDS == 16 ? (lane >> 1) & 3 : (lane >> 2) & 1;
#pragma unroll
    for (int c = 0; c < WORDS / 4; ++c)
        *reinterpret_cast<uint4 *>(buf + lane * WORDS * 4 + ((c ^ key) << 4)) =
            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    ++piece;
    return buf;
}

// 16 values, a row each, to element 0 of rows ld bytes apart; `rows` of them.
template <typename T>
__device__ __forceinline__ void store_down(uint8_t *at, long long ld, int rows, const float (&v)[16])
{
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        if (r < rows) {
            if constexpr (sizeof(T) == 4) *reinterpret_cast<float *>(at) = v[r];
            else *reinterpret_cast<T *>(at) = T(v[r]);
        }
        at += ld;
    }
}

}  // namespace

}  // namespace bigemm
