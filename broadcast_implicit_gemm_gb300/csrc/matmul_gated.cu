// matmul_gated.cu -- a gated layer's two products for many tokens, with the
// activation and the multiplication in the epilogue (matmul_gated.cuh).
//
// A pair's tile is 256 tokens by 128 channels of both products: the first CTA stages
// the gate's 128 rows of weights and the second one the up product's, so that the
// pair's MMA of 256 columns leaves g in columns 0 to 127 and u in 128 to 255 of each
// CTA's tokens, and a drain warp has both of its 32 channels at hand.  Nothing of the
// products goes to memory but what is asked for, and x is read for both at once.
#include "matmul_gated.cuh"

#include "matmul_pair.cuh"

namespace bigemm {

namespace {

struct GatedJob {
    // (five stages and twice the staging: 8192 x 4096 -> 16384 bf16 1102 us, 1084 so)
    static constexpr int stages = 6, per_warp = 2048;
    using Args = GatedArgs;
    using Maps = GatedMaps;
    struct Unit {
        Tile tile;
        int k0, k1;
    };

    static __device__ __forceinline__ bool unit(const Args &p, int turn, int pair, int pairs, Unit &u)
    {
        const int t = turn * pairs + pair;
        if (t >= p.m_tiles * p.n_tiles) return false;
        u.tile = tile_in(p.m_tiles, p.n_tiles, t);
        u.k0 = 0, u.k1 = p.k_blocks;
        return true;
    }

    static __device__ __forceinline__ void beside(const Args &, int, int, int) {}

    static __device__ __forceinline__ void load(const Maps &maps, const Args &, const Unit &u, int kb, int rank, uint8_t *sa,
                                                uint8_t *sb, uint32_t bar)
    {
        tma_load_2d_pair(sa, &maps.x, bar, kb * 64, u.tile.m * kManyTokens + rank * 128);
        tma_load_2d_pair(sb, &maps.w[rank], bar, kb * 64, u.tile.n * 128);
    }

    static __device__ __forceinline__ void mma(const Args &p, const Unit &, uint32_t d, uint32_t a, uint32_t b, uint32_t accum)
    {
        const uint32_t idesc = make_idesc(p.in_dt == BIGEMM_BF16 ? 1u : 0u, 0u, 0u, 256, 256);
        umma4_pair<2, 2>(d, operand_lo(a, false), operand_lo(b, false), desc_hi(1024u, 2u), idesc, accum);
    }

    // N sums of a lane's token from column col on, plus the bias of channels n on.
    template <int N>
    static __device__ __forceinline__ void sums(uint32_t tmem, const float *bias, bool vec, int n, long long cols, float (&v)[N])
    {
        uint32_t r[N];
        if constexpr (N == 32) {
            tmem_ld_32x32b_x32(tmem, r);
            tmem_wait_ld32(r);
        } else {
            tmem_ld_32x32b_x16(tmem, r);
            tmem_wait_ld16(r);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
        if (!bias) return;
        if (vec && n + N <= cols) {
            const float4 *b = reinterpret_cast<const float4 *>(bias + n);
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const float4 f = b[i];
                v[4 * i] += f.x, v[4 * i + 1] += f.y, v[4 * i + 2] += f.z, v[4 * i + 3] += f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (n + i < cols) v[i] += bias[n + i];
        }
    }

    static __device__ __forceinline__ void drain(const Maps &maps, const Args &p, const Unit &u, int rank, int q, int h,
                                                 uint32_t tmem, uint8_t *stage, int &piece, int lane)
    {
        const long long m_warp = (long long)u.tile.m * kManyTokens + rank * 128 + q * 32;
        const int n = u.tile.n * 128 + h * 32;
        if (n >= p.N) return;
        const uint32_t from[2] = {tmem + (uint32_t)(h * 32), tmem + (uint32_t)(128 + h * 32)};
        float v[32];
        if (p.gate) {
            sums<32>(from[0], p.bias, p.vec_bias, n, p.N, v);
            put16<per_warp>(&maps.kept[0], p.vec_gate, p.gate, p.ldgate, p.out_dt, p.M, p.N, stage, piece, lane, m_warp, n, v);
        }
        if (p.up) {
            sums<32>(from[1], p.bias_up, p.vec_bias_up, n, p.N, v);
            put16<per_warp>(&maps.kept[1], p.vec_up, p.up, p.ldup, p.out_dt, p.M, p.N, stage, piece, lane, m_warp, n, v);
        }
        // sixteen at a time: g and u together
#pragma unroll
        for (int c = 0; c < 32; c += 16) {
            float g[16], w[16];
            sums<16>(from[0] + (uint32_t)c, p.bias, p.vec_bias, n + c, p.N, g);
            sums<16>(from[1] + (uint32_t)c, p.bias_up, p.vec_bias_up, n + c, p.N, w);
            mm_act_all(p.act, g);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[c + i] = g[i] * w[i];
        }
        put16<per_warp>(&maps.out, p.vec_out, p.out, p.ldo, p.out_dt, p.M, p.N, stage, piece, lane, m_warp, n, v);
    }
};

}  // namespace

cudaError_t launch_gated_many(const GatedArgs &a, const GatedMaps &maps, int sms, cudaStream_t stream)
{
    ProfScope prof("matmul_gated", stream);
    const long long tiles = (long long)a.m_tiles * a.n_tiles;
    return launch_pairs<GatedJob>(a, maps, (int)(tiles < sms / 2 ? tiles : sms / 2), stream);
}

}  // namespace bigemm
