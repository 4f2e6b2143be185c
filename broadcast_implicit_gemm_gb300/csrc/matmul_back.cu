// matmul_back.cu -- the products of the gradients (matmul_back.cuh), dx and dw in one
// launch.
//
// Neither reads a transposed copy: d [tokens, channels], w [channels, in] and x
// [tokens, in] are loaded as they lie, in boxes of 64 x 64, and what the summed axis is
// not contiguous in is an MN-major operand of the MMA.  dx sums over channels (d
// K-major, w MN-major; of both products one after the other, in one accumulator), dw
// over tokens (d^T and x MN-major).
//
// A dx unit is long (4096 tokens, 2 x 16384 channels: 512 blocks) and a dw unit short
// (64): the pairs share them as back_walk.h says (4096 x 4096 x 16384 gated: 3449
// blocks' time per pair, 3776 in two launches).  Few tokens leave too few dx units, and
// few channels too few dw units: each is cut along the summed axis then, the shares go to
// a workspace in fp32, and launch_back_join adds them in their order.  So is a sum that is
// longer than one accumulator takes (kLongestSum).
#include "matmul_back.cuh"

#include "matmul_pair.cuh"

namespace bigemm {

namespace {

struct BackJob {
    // 64 columns of a warp's rows leave at once, which takes a stage's worth of staging (with 32 at a time and six
    // stages 1 x 4096 x 4096 26.1 us, 24.4 so; 8192 x 16384 x 4096 1170 and 1193)
    static constexpr int stages = 5, per_warp = 4096;
    using Args = BackArgs;
    using Maps = BackMaps;
    struct Unit {
        int what;                    // 0: dx, 1 and 2: dw of a product
        int m0, n0;                  // rows and columns of the result
        int k0, k1, part;
    };

    static __device__ __forceinline__ bool unit(const Args &p, int turn, int pair, int pairs, Unit &u)
    {
        int i = back_unit(p.walk, turn, pair, pairs);
        if (i < 0) return false;
        const bool first = i < p.walk.dx;
        if (!first) i -= p.walk.dx;
        if (first != p.dw_first) {
            const Tile t = place(p.to_dx, i, u);
            u.what = 0, u.m0 = t.m * 256, u.n0 = t.n * 256;
        } else {
            const Tile t = place(p.to_dw, i, u);
            const int which = t.m >= p.dw_m ? 1 : 0;
            u.what = 1 + which, u.m0 = (t.m - which * p.dw_m) * 256, u.n0 = t.n * 256;
        }
        return true;
    }

    // Sums of dout's columns over a few tokens, 32 columns a turn, sixteen rows in flight.
    static __device__ __forceinline__ void beside(const Args &p, int i, int count, int lane)
    {
        if (!p.sums) return;
        if (p.dt == BIGEMM_F16) sums_of<__half>(p, i, count, lane);
        else sums_of<__nv_bfloat16>(p, i, count, lane);
    }

    template <typename T>
    static __device__ __forceinline__ void sums_of(const Args &p, int i, int count, int lane)
    {
        for (long long c = i * 32ll + lane; c < p.N; c += count * 32ll) {
            const T *at = static_cast<const T *>(p.dout) + c;
            float v = 0.f;
            for (int r = 0; r < p.M; r += 16, at += 16 * p.ldd) {
                T row[16];
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (r + k < p.M) row[k] = at[k * p.ldd];
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    if (r + k < p.M) v += (float)row[k];
            }
            p.sums[c] = v;
        }
    }

    // Tile and share of a result's unit, in tile_in's order.
    static __device__ __forceinline__ Tile place(const UnitGrid &g, int i, Unit &u)
    {
        uint32_t t;
        u.part = (int)fd_divmod((uint32_t)i, g.tiles, &t);
        u.k0 = share_start(g, u.part);
        u.k1 = share_start(g, u.part + 1);
        uint32_t r;
        const int m = (int)fd_divmod(t, g.group, &r) * 8, rows = min(8, g.m - m);
        if (rows == 8) return {m + (int)(r & 7), (int)(r >> 3)};
        return {m + (int)r % rows, (int)r / rows};
    }

    // a box's coordinates: column, row
    static __device__ __forceinline__ void load(const Maps &maps, const Args &p, const Unit &u, int kb, int rank, uint8_t *sa,
                                                uint8_t *sb, uint32_t bar)
    {
        const int m = u.m0 + rank * 128, n = u.n0 + rank * 128;
        if (u.what == 0) {
            const int which = kb >= p.n_blocks ? 1 : 0, k = (kb - which * p.n_blocks) * 64;
            tma_load_2d_pair(sa, &maps.d[which], bar, k, m);
            tma_load_2d_pair(sa + PairCfg::box, &maps.d[which], bar, k, m + 64);
            tma_load_2d_pair(sb, &maps.w[which], bar, n, k);
            tma_load_2d_pair(sb + PairCfg::box, &maps.w[which], bar, n + 64, k);
        } else {
            const CUtensorMap *d = &maps.d[u.what - 1];
            tma_load_2d_pair(sa, d, bar, m, kb * 64);
            tma_load_2d_pair(sa + PairCfg::box, d, bar, m + 64, kb * 64);
            tma_load_2d_pair(sb, &maps.x, bar, n, kb * 64);
            tma_load_2d_pair(sb + PairCfg::box, &maps.x, bar, n + 64, kb * 64);
        }
    }

    static __device__ __forceinline__ void mma(const Args &p, const Unit &u, uint32_t d, uint32_t a, uint32_t b, uint32_t accum)
    {
        const uint32_t fmt = p.dt == BIGEMM_BF16 ? 1u : 0u, hi = desc_hi(1024u, 2u), b_lo = operand_lo(b, true);
        if (u.what == 0)
            umma4_pair<2, 128>(d, operand_lo(a, false), b_lo, hi, make_idesc(fmt, 0u, 1u, 256, 256), accum);
        else
            umma4_pair<128, 128>(d, operand_lo(a, true), b_lo, hi, make_idesc(fmt, 1u, 1u, 256, 256), accum);
    }

    static __device__ __forceinline__ void drain(const Maps &maps, const Args &p, const Unit &u, int rank, int q, int h,
                                                 uint32_t tmem, uint8_t *stage, int &piece, int lane)
    {
        const long long m_warp = u.m0 + rank * 128 + q * 32, rows = u.what == 0 ? p.M : p.N;
        const int n = u.n0 + h * 64;
        if (m_warp >= rows || n >= p.K) return;
        const uint32_t from = tmem + (uint32_t)(h * 64);
        const bool dx = u.what == 0;
        const int w = max(0, u.what - 1);
        if ((dx ? p.to_dx.split : p.to_dw.split) > 1) {
            // a share: 32 columns of 32 bits at a time
#pragma unroll 1
            for (int c = 0; c < 64 && n + c < p.K; c += 32) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(from + (uint32_t)c, r);
                tmem_wait_ld32(r);
                const uint8_t *buf = stage_words<per_warp, 32>(stage, piece, lane, r);
                if (lane == 0) {
                    tma_store_3d(dx ? &maps.part[0] : &maps.part[1], buf, n + c, (int)m_warp, u.part + (dx ? 0 : w * p.to_dw.split));
                    bulk_commit();
                }
            }
            return;
        }
        // 64 columns, a row of 128 bytes, by one TMA store
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t r[32], q[16];
            tmem_ld_32x32b_x32(from + (uint32_t)(c * 32), r);
            tmem_wait_ld32(r);
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
            words_of(v, p.dt, q);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4 *>(stage + lane * 128 + (((c * 4 + i) ^ (lane & 7)) << 4)) =
                    make_uint4(q[4 * i], q[4 * i + 1], q[4 * i + 2], q[4 * i + 3]);
        }
        if ((dx ? p.dx_rows : p.dw_rows[w]) && whole_words(p.K, n, 64)) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(dx ? &maps.dx : &maps.dw[w], stage, n, (int)m_warp);
                bulk_commit();
            }
        } else {
            __syncwarp();
            put_off_grid<32>(dx ? p.dx : p.dw[w], dx ? p.lddx : p.lddw[w], rows, p.K, stage, lane, m_warp, n);
        }
    }
};

// A warp adds 128 columns of a row's shares, which lie in L2, where the products left
// them; eight loads of a lane leave together, however few shares there are.
template <typename T>
__global__ void __launch_bounds__(256) back_join_kernel(const JoinArgs a)
{
    griddep_enter();
    const int lane = (int)threadIdx.x & 31;
    long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    int which = 0;
#pragma unroll
    for (int k = 0; k + 1 < kJoinMost; ++k) which += item >= a.items[k] ? 1 : 0;
    if (which >= a.count) return;
    const JoinResult &o = a.result[which];
    if (which > 0) item -= a.items[which - 1];
    const long long m = item / a.runs;
    const int k0 = (int)(item - m * a.runs) * 128;
    if (m >= o.rows) return;
    T *row = static_cast<T *>(o.out) + m * o.ld;
    const float *from = o.part + m * a.pitch + k0;
    const long long step = (long long)o.rows * a.pitch;
    if (o.vec) {
        // four columns a lane (the rows' last words have room)
        const int k = k0 + lane * 4;
        if (k >= a.cols) return;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < o.split; s += 8) {
            float4 w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = s + i < o.split ? *reinterpret_cast<const float4 *>(from + (s + i) * step + lane * 4)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) v.x += w[i].x, v.y += w[i].y, v.z += w[i].z, v.w += w[i].w;
        }
        alignas(8) const T t[4] = {T(v.x), T(v.y), T(v.z), T(v.w)};
        if (k + 4 <= a.cols) {
            *reinterpret_cast<uint2 *>(row + k) = *reinterpret_cast<const uint2 *>(t);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (k + i < a.cols) row[k + i] = t[i];
        }
        return;
    }
    // one of each 32 a lane
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < o.split; s += 8) {
        float w[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                w[i][j] = s + i < o.split && k0 + j * 32 + lane < a.cols ? from[(s + i) * step + j * 32 + lane] : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += w[i][j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (k0 + j * 32 + lane < a.cols) row[k0 + j * 32 + lane] = T(v[j]);
}

}  // namespace

cudaError_t launch_matmul_back(const BackArgs &a, const BackMaps &maps, int pairs, cudaStream_t stream)
{
    ProfScope prof("matmul_back", stream);
    return launch_pairs<BackJob>(a, maps, pairs, stream);
}

cudaError_t launch_back_join(JoinArgs &a, int dt, cudaStream_t stream)
{
    ProfScope prof("matmul_back_join", stream);
    a.runs = (a.cols + 127ll) / 128;
    long long end = 0;
    for (int k = 0; k < kJoinMost; ++k) a.items[k] = end += k < a.count ? a.result[k].rows * a.runs : 0;
    const long long blocks = (end + 7) / 8;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks);
    return dt == BIGEMM_F16 ? launch_pdl(back_join_kernel<__half>, grid, dim3(256), 0, stream, a)
                            : launch_pdl(back_join_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, a);
}

}  // namespace bigemm
