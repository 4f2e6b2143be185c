// matmul_many.cu -- the matrix product for many tokens: a pair of CTAs per tile
// of 256 tokens by BN output channels.
//
// Such a product is bound by the tensor cores.  The pair shares each MMA
// (M = 256: 128 tokens per CTA, half of the weights' rows in each), which halves
// what an SM's shared memory has to deliver for the weights: at 256 x 256 a CTA
// stages 32 KB per 64 elements of K (128 in 8 bits) for 4 MMAs of 128 cycles.
// Pairs are persistent; one warp loads, one issues MMAs, 8 or 16 drain: two
// or four per quarter of the tokens, a lane to a token.  Tiles
// are walked eight token tiles at a time across the channels, so that what runs
// at once shares its operands in L2.
//
// 16-bit operands: two accumulators fill tensor memory, and a tile's epilogue
// runs beside the next one's MMAs.  MX: the scales take columns too (12 per
// stage), so there is one accumulator; the drain warps take all of it to
// registers, hand it back, and go on from there.  For an MXFP8 output they add up
// pieces of 2048 elements there.
//
// FULL: a 32-bit output, sums of at most 512 or 2048 elements added up in registers
// (matmul_few.cu says why).
#include "matmul.cuh"

namespace bigemm {

namespace {

constexpr int kManyA = 128 * kRow;             // a CTA's tokens per stage

template <int BN, bool MX, bool FULL>
struct ManyCfg {
    static constexpr bool keep = MX || FULL;       // the tile's sums go to registers before the epilogue
    // A block is a warpgroup with the producer, the MMA warp and two idle ones, and the drain
    // warps' groups; the registers it launches with are dealt out anew between the two kinds.
    // Sixteen drain warps hide each other's latencies (8192 x 4096 x 512 bf16: 37 us with eight,
    // 32 with sixteen), but leave no room for a tile's sums.
    static constexpr int drain = keep ? 8 : 16, threads = 128 + 32 * drain;
    static constexpr int launch_regs = keep ? 168 : 96, lead_regs = keep ? 72 : 56, drain_regs = keep ? 216 : 104;
    static_assert(lead_regs + drain / 4 * drain_regs <= threads / 128 * launch_regs, "a larger sum would wait for ever");
    static constexpr int units = BN / 32 / (drain / 4);                       // of 32 channels, per drain warp
    static constexpr int b_bytes = BN / 2 * kRow;
    static constexpr int s_bytes = MX ? (1 + BN / 128) * kMxBlockBytes : 0;   // the CTA's tokens, all of BN
    static constexpr int stage = kManyA + b_bytes + s_bytes;
    static constexpr int per_warp = FULL ? 4096 : 2048;                       // output staging
    static constexpr int stages = BN == 128 ? 7 : FULL ? 5 : 6;
    static constexpr int accs = MX ? 1 : 2;
    static constexpr int smem = stages * stage + drain * per_warp + 256 + 1024;
    static_assert(smem <= 227 * 1024, "shared memory");
    static constexpr uint32_t cols = accs * BN + (MX ? stages * (4 + BN / 32) : 0) <= 256 ? 256 : 512;
    static_assert(accs * BN + (MX ? stages * (4 + BN / 32) : 0) <= 512, "tensor memory");
};

struct Tile {
    int m, n;
};

// Eight token tiles share a sweep over the channel tiles.
__device__ __forceinline__ Tile tile_of(const MatmulArgs &p, int t)
{
    constexpr int kGroup = 8;
    const int per = kGroup * p.n_tiles;
    const int g = t / per, r = t - g * per;
    const int rows = min(kGroup, p.m_tiles - g * kGroup);
    return {g * kGroup + r % rows, r / rows};
}

// A warp's 32 tokens by 32 channels of other come as they lie in memory, 4 (or,
// of 32 bits, 8) lanes to a token's 64 (128) bytes, and are turned round in
// shared memory: a lane that loads its own token's bytes makes each load touch
// 32 lines (8192 x 4096 x 64 bf16 with a gate: 63 us against 48).
struct Other32 {
    uint4 q[4];
};

// 16-bit ones are asked for before the sums are there.
__device__ __forceinline__ void other_ahead(const MatmulArgs &p, int lane, int m_warp, int n, Other32 &o)
{
    if (p.combine == BIGEMM_COMBINE_NONE || p.other_dt == BIGEMM_F32 || !p.by_rows || n + 32 > p.N) return;
    const int m = m_warp + (lane >> 2);
    const uint16_t *from = static_cast<const uint16_t *>(p.other) + (long long)m * p.ldother + n + (lane & 3) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (m + 8 * i < p.M) o.q[i] = *reinterpret_cast<const uint4 *>(from + 8 * i * p.ldother);
}

// A warp's part of a tile's other, a row per lane, to L2.
template <int UNITS>
__device__ __forceinline__ void other_to_l2(const MatmulArgs &p, Tile tile, int bn, int row, int h)
{
    const long long m = (long long)tile.m * kManyTokens + row;
    const int n = tile.n * bn + h * UNITS * 32;
    if (p.combine == BIGEMM_COMBINE_NONE || m >= p.M || n >= p.N) return;
    const int es = p.other_dt == BIGEMM_F32 ? 4 : 2, bytes = min(UNITS * 32, p.N - n) * es;
    const uint8_t *from = static_cast<const uint8_t *>(p.other) + (m * p.ldother + n) * es;
    for (int i = 0; i < bytes; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(from + i));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(from + bytes - 1));
}

// To the staging (free of the last output's reader after the wait), for
// epilogue32 to read a token per lane.
__device__ __forceinline__ void other_turn(const MatmulArgs &p, uint8_t *stage, int lane, const Other32 &o)
{
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = (lane >> 2) + 8 * i;
        *reinterpret_cast<uint4 *>(stage + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4)) = o.q[i];
    }
    __syncwarp();
}

// v * or + 32 values of other: 16-bit ones from the staging, 16 bytes at a time,
// swizzled by key; 32-bit ones as they are.
template <int DT, bool MUL>
__device__ __forceinline__ void combine_each(const void *row, int key, float (&v)[32])
{
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        float f[8];
        if (DT == BIGEMM_F32) mm_load8(row, c * 8, BIGEMM_F32, f);
        else mm_unpack8(reinterpret_cast<const uint4 *>(row)[c ^ key], DT, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c * 8 + j] = MUL ? v[c * 8 + j] * f[j] : v[c * 8 + j] + f[j];
    }
}

// 32 channels of one token from channel n on, all inside N: bias, act, combine.
__device__ __forceinline__ void epilogue32(const MatmulArgs &p, uint8_t *stage, int lane, long long m, int n,
                                           const Other32 &o, float (&v)[32])
{
    if (p.bias) {
        if (p.vec_bias) {
            const float4 *b = reinterpret_cast<const float4 *>(p.bias + n);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 f = b[i];
                v[4 * i] += f.x, v[4 * i + 1] += f.y, v[4 * i + 2] += f.z, v[4 * i + 3] += f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += p.bias[n + i];
        }
    }
    mm_act_all(p.act, v);
    if (p.combine == BIGEMM_COMBINE_NONE) return;
    const bool mul = p.combine == BIGEMM_COMBINE_MUL;
    if (p.other_dt == BIGEMM_F32) {
        if (m < p.M) {
            const float *from = static_cast<const float *>(p.other) + m * p.ldother + n;
            if (mul) combine_each<BIGEMM_F32, true>(from, 0, v);
            else combine_each<BIGEMM_F32, false>(from, 0, v);
        }
        return;
    }
    other_turn(p, stage, lane, o);
    // the type and the operation are chosen once for all 32
    const uint8_t *row = stage + lane * 64;
    const int key = (lane >> 1) & 3;
    if (p.other_dt == BIGEMM_F16) {
        if (mul) combine_each<BIGEMM_F16, true>(row, key, v);
        else combine_each<BIGEMM_F16, false>(row, key, v);
    } else {
        if (mul) combine_each<BIGEMM_BF16, true>(row, key, v);
        else combine_each<BIGEMM_BF16, false>(row, key, v);
    }
    __syncwarp();                    // every lane has its token before the output takes the staging
}

// 32 rows of WORDS 32-bit words, a lane's row in w, to global memory: through the
// staging (two buffers of it, where two fit) by TMA.
template <int PER_WARP, int WORDS>
__device__ __forceinline__ void put_words(const MatmulArgs &p, const CUtensorMap *map, uint8_t *stage, int &piece,
                                          int lane, int m_warp, int n, const uint32_t (&w)[WORDS])
{
    constexpr int bytes = WORDS * 128;
    constexpr bool two = 2 * bytes <= PER_WARP;
    uint8_t *buf = stage + (two ? (piece & 1) * bytes : 0);
    if (lane == 0) bulk_wait_read<two ? 1 : 0>();
    __syncwarp();
    // the swizzle of the output's map: rows of 128, 64 or 32 bytes
    const int key = WORDS == 32 ? lane & 7 : WORDS == 16 ? (lane >> 1) & 3 : (lane >> 2) & 1;
#pragma unroll
    for (int c = 0; c < WORDS / 4; ++c)
        *reinterpret_cast<uint4 *>(buf + lane * WORDS * 4 + ((c ^ key) << 4)) =
            make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0 && m_warp < p.M) {
        tma_store_2d(map, buf, n, m_warp);
        bulk_commit();
    }
    ++piece;
}

// A drain warp's output of 32 tokens by 32 channels, all inside N, a lane's
// token in v.  Returns the scale code of the lane's group for an e4m3 output.
template <int PER_WARP, bool MX, bool FULL>
__device__ __forceinline__ uint32_t put_rows(const MatmulArgs &p, const CUtensorMap *map, uint8_t *stage, int &piece,
                                             int lane, int m_warp, int n, float (&v)[32])
{
    if constexpr (FULL) {
        uint32_t w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i]);
        put_words<PER_WARP, 32>(p, map, stage, piece, lane, m_warp, n, w);
        return 0;
    }
    if (MX && p.out_dt == BIGEMM_MXF8) {
        uint32_t w[8];
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) top = mx_amax(top, v[i]);
        const uint32_t code = mx_scale_code(top);
        const float inv = mx_inv_scale(code);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = mx_pack4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
        put_words<PER_WARP, 8>(p, map, stage, piece, lane, m_warp, n, w);
        return code;
    }
    uint32_t w[16];
    if (p.out_dt == BIGEMM_F16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = mm_pack2(v[2 * i], v[2 * i + 1], BIGEMM_F16);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = mm_pack2(v[2 * i], v[2 * i + 1], BIGEMM_BF16);
    }
    put_words<PER_WARP, 16>(p, map, stage, piece, lane, m_warp, n, w);
    return 0;
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

template <typename T>
__device__ __forceinline__ void load_down(const uint8_t *at, long long ld, int rows, uint32_t (&v)[16])
{
#pragma unroll
    for (int r = 0; r < 16; ++r) {
        v[r] = r < rows ? *reinterpret_cast<const T *>(at) : 0;
        at += ld;
    }
}

// The same 32 by 32 sums where rows are off the 16-byte grid or the channels
// end inside: they are turned round in shared memory, 16 tokens at a time, so
// that a lane has one channel of each token and the warp's plain loads and
// stores cover a token's 32 channels at once.  All of the epilogue is here.
template <bool MX, bool FULL>
__device__ __forceinline__ uint32_t put_columns(const MatmulArgs &p, uint8_t *stage, int lane, int m_warp, int n,
                                                float (&v)[32])
{
    float *turn = reinterpret_cast<float *>(stage);
    const bool in = n + lane < p.N;
    const float bias = p.bias && in ? p.bias[n + lane] : 0.f;
    uint32_t code = 0;
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
        if (lane >> 4 == half) {
#pragma unroll
            for (int i = 0; i < 32; ++i) turn[(lane & 15) * 32 + (i ^ (lane & 15))] = v[i];
        }
        __syncwarp();
        const long long m0 = m_warp + half * 16;
        const int rows = in ? (int)min(16ll, p.M - m0) : 0;      // that this lane reads and writes
        uint32_t o[16];              // all loads leave before the first is used
        if (p.combine != BIGEMM_COMBINE_NONE) {
            const long long at = m0 * p.ldother + n + lane;
            if (p.other_dt == BIGEMM_F32)
                load_down<uint32_t>(static_cast<const uint8_t *>(p.other) + at * 4, p.ldother * 4, rows, o);
            else
                load_down<uint16_t>(static_cast<const uint8_t *>(p.other) + at * 2, p.ldother * 2, rows, o);
        }
        float y[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) y[r] = turn[r * 32 + (lane ^ r)] + bias;
        mm_act_all(p.act, y);
        if (p.combine != BIGEMM_COMBINE_NONE) {
#pragma unroll
            for (int r = 0; r < 16; ++r) y[r] = mm_combine(p.combine, y[r], mm_value(o[r], p.other_dt));
        }
        const long long at = m0 * p.ldo + n + lane;
        uint8_t *out = static_cast<uint8_t *>(p.out);
        if (MX && p.out_dt == BIGEMM_MXF8) {
            out += at;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const uint32_t top = __reduce_max_sync(0xffffffffu, in ? __float_as_uint(y[r]) & 0x7fffffffu : 0u);
                const uint32_t c = mx_scale_code(__uint_as_float(top));
                if (lane == half * 16 + r) code = c;
                if (r < rows) out[r * p.ldo] = (uint8_t)mx_pack4(y[r] * mx_inv_scale(c), 0.f, 0.f, 0.f);
            }
        } else if (FULL) {
            store_down<float>(out + at * 4, p.ldo * 4, rows, y);
        } else if (p.out_dt == BIGEMM_F16) {
            store_down<__half>(out + at * 2, p.ldo * 2, rows, y);
        } else {
            store_down<__nv_bfloat16>(out + at * 2, p.ldo * 2, rows, y);
        }
        __syncwarp();
    }
    return code;
}

template <int BN, bool MX, bool FULL>
__global__ void __launch_bounds__(ManyCfg<BN, MX, FULL>::threads, 1)
    matmul_many_kernel(const __grid_constant__ ManyMaps maps, const MatmulArgs p)
{
    using C = ManyCfg<BN, MX, FULL>;
    constexpr int S = C::stages, ACC = C::accs;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sa = smem, *sb = sa + S * kManyA, *out_stage = sb + S * C::b_bytes, *ss = out_stage + C::drain * C::per_warp;
    uint64_t *full = reinterpret_cast<uint64_t *>(ss + S * C::s_bytes);
    uint64_t *empty = full + S, *tfull = empty + S, *tempty = tfull + 2, *drain = tempty + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);
    const int tiles = p.m_tiles * p.n_tiles;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        // an accumulator comes back from both CTAs' drain warps
        for (int i = 0; i < 2; ++i) mbar_init(&tfull[i], 1), mbar_init(&tempty[i], 2 * C::drain);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.x);
        tma_prefetch_desc(&maps.w);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc_pair(tmem_holder, C::cols);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync_all();   // both CTAs' barriers initialised and tensor memory allocated
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    griddep_enter();

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::lead_regs));
        if (warp == 0) {
            // ------------------------------------------------------ producer
            if (lane == 0) {
                constexpr int per = MX ? kRow : kRow / 2;         // elements of K per stage
                const uint32_t full_even = mapa_shared(smem_u32(full), 0);
                int stage = 0;
                uint32_t phase = 0, last_parity[S];
                bool issued[S], ok = true;
                for (int i = 0; i < S; ++i) issued[i] = false, last_parity[i] = 0;
                for (int t = pair; ok && t < tiles; t += pairs) {
                    const Tile tile = tile_of(p, t);
                    const int m0 = tile.m * kManyTokens + rank * 128;
                    const int n0 = tile.n * BN + rank * (BN / 2);
                    for (int kb = 0; kb < p.k_blocks; ++kb) {
                        ok = mbar_wait(&empty[stage], phase ^ 1u, p.timeout_ns, abort_flag, p.err);
                        if (!ok) break;
                        if (leader) mbar_arrive_expect_tx(&full[stage], 2u * (uint32_t)C::stage);
                        issued[stage] = true, last_parity[stage] = phase;
                        const uint32_t bar = full_even + (uint32_t)stage * 8u;
                        tma_load_2d_pair(sa + stage * kManyA, &maps.x, bar, kb * per, m0);
                        tma_load_2d_pair(sb + stage * C::b_bytes, &maps.w, bar, kb * per, n0);
                        if (MX) {
                            uint8_t *s = ss + stage * C::s_bytes;
                            tma_load_3d_pair(s, &maps.xs, bar, 0, kb, m0 >> 7);
                            tma_load_3d_pair(s + kMxBlockBytes, &maps.ws, bar, 0, kb, (tile.n * BN) >> 7);
                        }
                        if (++stage == S) stage = 0, phase ^= 1u;
                    }
                }
                if (!ok) {
                    if (leader) {
                        int local_abort = 0;
                        for (int i = 0; i < S; ++i)
                            if (issued[i]) mbar_wait(&full[i], last_parity[i], p.timeout_ns, &local_abort, p.err);
                    } else {
                        // this CTA cannot wait on the even CTA's barriers: give its copies time to land
                        const uint64_t t0 = globaltimer_ns();
                        while (globaltimer_ns() - t0 < 20000ull) {
                        }
                    }
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------ MMA issuer
            if (leader && lane == 0) {
                const uint32_t idesc = MX ? make_idesc_mx(256, BN)
                                          : make_idesc(p.in_dt == BIGEMM_BF16 ? 1u : 0u, 0u, 0u, 256, BN);
                const uint32_t hi = desc_hi(1024u, 2u), s_hi = desc_hi(128u, 0u);
                int stage = 0, a = 0;
                uint32_t phase = 0, acc_phase = 0;
                bool ok = true, any = false;
                for (int t = pair; ok && t < tiles; t += pairs) {
                    for (int k0 = 0; ok && k0 < p.k_blocks; k0 += p.seg_blocks) {
                        ok = mbar_wait(&tempty[a], acc_phase ^ 1u, p.timeout_ns, abort_flag, p.err);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t d = tmem_base + (uint32_t)(a * BN);
                        const int k1 = min(p.k_blocks, k0 + p.seg_blocks);
                        for (int kb = k0; kb < k1; ++kb) {
                            ok = mbar_wait(&full[stage], phase, p.timeout_ns, abort_flag, p.err);
                            if (!ok) break;
                            tc_fence_after();
                            const uint32_t a_lo = desc_lo(smem_u32(sa + stage * kManyA), 16u);
                            const uint32_t b_lo = desc_lo(smem_u32(sb + stage * C::b_bytes), 16u);
                            if (MX) {
                                const uint32_t s_lo = desc_lo(smem_u32(ss + stage * C::s_bytes), 0u);
                                const uint32_t sf = tmem_base + (uint32_t)(ACC * BN + (4 + BN / 32) * stage);
    #pragma unroll
                                for (uint32_t i = 0; i < 1 + BN / 128; ++i)
                                    tmem_copy_scales_pair(sf + 4 * i, (uint64_t)s_hi << 32 | (s_lo + i * (kMxBlockBytes >> 4)));
    #pragma unroll
                                for (uint32_t k = 0; k < 4; ++k)
                                    umma_mx_pair(d, a_lo + 2 * k, hi, b_lo + 2 * k, hi, idesc | (k << 4) | (k << 29), sf,
                                                 sf + 4, (kb > k0 || k > 0) ? 1u : 0u);
                            } else {
                                umma4_kmajor_pair<false>(d, a_lo, hi, b_lo, hi, idesc, kb > k0 ? 1u : 0u);
                            }
                            any = true;
                            umma_commit_pair_mc(&empty[stage], (uint16_t)3u);
                            if (++stage == S) stage = 0, phase ^= 1u;
                        }
                        if (!ok) break;
                        umma_commit_pair_mc(&tfull[a], (uint16_t)3u);
                        if (++a == ACC) a = 0, acc_phase ^= 1u;
                    }
                }
                if (!ok && any) {
                    int local_abort = 0;
                    umma_commit_pair(drain);
                    mbar_wait(drain, 0, p.timeout_ns, &local_abort, p.err);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::drain_regs));
        // ------------------------------------------------------ drain and epilogue
        constexpr bool KEEP = C::keep;
        constexpr int UNITS = C::units;
        const int q = warp & 3, h = (warp - 4) >> 2;
        const uint32_t lane_base = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(h * UNITS * 32);
        const uint32_t tempty_even = mapa_shared(smem_u32(tempty), 0);
        uint8_t *stage = out_stage + (warp - 4) * C::per_warp;
        const int col_blocks = (int)((p.N + 127ll) / 128);
        int a = 0, piece = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        if (pair < tiles) other_to_l2<C::units>(p, tile_of(p, pair), BN, rank * 128 + q * 32 + lane, h);
        for (int t = pair; ok && t < tiles; t += pairs) {
            const Tile tile = tile_of(p, t);
            const int m_warp = tile.m * kManyTokens + rank * 128 + q * 32, n_warp = tile.n * BN + h * UNITS * 32;
            const long long m = m_warp + lane;
            // the next tile's part of other comes to L2 while this one is done
            if (t + pairs < tiles) other_to_l2<C::units>(p, tile_of(p, t + pairs), BN, rank * 128 + q * 32 + lane, h);
            Other32 ahead;
            other_ahead(p, lane, m_warp, n_warp, ahead);
            uint32_t codes = 0;
            float keep[KEEP ? UNITS : 1][32];
            for (int k0 = 0; k0 < p.k_blocks; k0 += p.seg_blocks) {
                ok = mbar_wait_warp(&tfull[a], acc_phase, p.timeout_ns, abort_flag, p.err);
                if (!ok) break;
                tc_fence_after();
                const uint32_t base = lane_base + (uint32_t)(a * BN);
                if (KEEP && !FULL && k0 == 0) {
                    uint32_t r[UNITS][32];
#pragma unroll
                    for (int u = 0; u < UNITS; ++u) tmem_ld_32x32b_x32(base + u * 32, r[u]);
#pragma unroll
                    for (int u = 0; u < UNITS; ++u) {
                        tmem_wait_ld32(r[u]);
#pragma unroll
                        for (int i = 0; i < 32; ++i) keep[KEEP ? u : 0][i] = __uint_as_float(r[u][i]);
                    }
                } else if constexpr (KEEP) {
#pragma unroll
                    for (int u = 0; u < UNITS; ++u) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(base + u * 32, r);
                        tmem_wait_ld32(r);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            keep[u][i] = k0 > 0 ? keep[u][i] + __uint_as_float(r[i]) : __uint_as_float(r[i]);
                    }
                } else {
#pragma unroll 1
                    for (int u = 0; u < UNITS; ++u) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(base + u * 32, r);
                        tmem_wait_ld32(r);
                        const int n = n_warp + u * 32;
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                        if (p.by_rows && n + 32 <= p.N) {
                            epilogue32(p, stage, lane, m, n, ahead, v);
                            put_rows<C::per_warp, MX, FULL>(p, &maps.out, stage, piece, lane, m_warp, n, v);
                            // (not before: the fence in there waits for loads in flight)
                            if (u + 1 < UNITS) other_ahead(p, lane, m_warp, n + 32, ahead);
                        } else if (n < p.N) {
                            put_columns<MX, FULL>(p, stage, lane, m_warp, n, v);
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(tempty_even + (uint32_t)a * 8u);
                if (++a == ACC) a = 0, acc_phase ^= 1u;
            }
            if constexpr (KEEP) {
                if (!ok) break;
#pragma unroll
                for (int u = 0; u < UNITS; ++u) {
                    const int n = n_warp + u * 32;
                    if (p.by_rows && n + 32 <= p.N) {
                        epilogue32(p, stage, lane, m, n, ahead, keep[u]);
                        codes |= put_rows<C::per_warp, MX, FULL>(p, &maps.out, stage, piece, lane, m_warp, n, keep[u]) << (8 * u);
                        if (u + 1 < UNITS) other_ahead(p, lane, m_warp, n + 32, ahead);
                    } else if (n < p.N) {
                        codes |= put_columns<MX, FULL>(p, stage, lane, m_warp, n, keep[u]) << (8 * u);
                    }
                }
                if (MX && p.out_dt == BIGEMM_MXF8 && m < p.M && (n_warp >> 7) < col_blocks) {
                    uint8_t *at = p.outs + mx_scale_offset(m, n_warp / kMxGroup, col_blocks);
                    if (UNITS == 4) *reinterpret_cast<uint32_t *>(at) = codes;
                    else *reinterpret_cast<uint16_t *>(at) = (uint16_t)codes;
                }
            }
        }
        // the staging is read before the block's shared memory goes
        if (lane == 0) bulk_wait<0>();
    }

    tc_fence_before();
    __syncwarp();
    cluster_sync_all();   // neither CTA leaves while its partner may still use its memory
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc_pair(tmem_base, C::cols);
    }
}

template <int BN, bool MX, bool FULL>
cudaError_t launch_one(const MatmulArgs &a, int grid, const ManyMaps &maps, cudaStream_t stream)
{
    auto kern = matmul_many_kernel<BN, MX, FULL>;
    constexpr int smem = ManyCfg<BN, MX, FULL>::smem;
    static unsigned long long attr_set = 0;   // bit per device: smem opt-in done
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !(attr_set >> dev & 1ull)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        // the split of registers counts on what the block is launched with
        cudaFuncAttributes fa;
        const cudaError_t f = cudaFuncGetAttributes(&fa, kern);
        if (f != cudaSuccess) return f;
        if (fa.numRegs != ManyCfg<BN, MX, FULL>::launch_regs) return cudaErrorInvalidConfiguration;
        if (dev < 64) attr_set |= 1ull << dev;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(ManyCfg<BN, MX, FULL>::threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, maps, a);
}

template <int BN>
cudaError_t launch_bn(const MatmulArgs &a, int grid, const ManyMaps &maps, cudaStream_t s)
{
    const bool full = a.out_dt == BIGEMM_F32;
    if (a.in_dt == BIGEMM_MXF8)
        return full ? launch_one<BN, true, true>(a, grid, maps, s) : launch_one<BN, true, false>(a, grid, maps, s);
    return full ? launch_one<BN, false, true>(a, grid, maps, s) : launch_one<BN, false, false>(a, grid, maps, s);
}

}  // namespace

cudaError_t launch_matmul_many(const MatmulArgs &a, int bn, int sms, const ManyMaps &maps, cudaStream_t stream)
{
    ProfScope prof("matmul_many", stream);
    const long long tiles = (long long)a.m_tiles * a.n_tiles;
    const int grid = 2 * (int)(tiles < sms / 2 ? tiles : sms / 2);
    return bn == 256 ? launch_bn<256>(a, grid, maps, stream) : launch_bn<128>(a, grid, maps, stream);
}

}  // namespace bigemm
