// matmul_few.cu -- the matrix product for few tokens: 128 output channels by
// BN tokens per CTA, the K axis shared by a cluster of CTAs.
//
// The weights are the 128-row operand of the MMA and the tokens its N side, so
// a handful of tokens wastes tensor work (which is free here) and no memory
// traffic.  Such a product is bound by the weights' bytes; one CTA per 128
// channels would leave most SMs without any, so `split` CTAs take a slice of K
// each, and as a cluster add up their fp32 partial sums through distributed
// shared memory: each rank sends every other one its sums of the tokens which
// that one finishes, and adds what it got in rank order, so that the result
// does not depend on timing, without a workspace and without a second launch.
// (Sent, not fetched: a fetch waits for each answer, and holds its owner in a
// second barrier: one token through 4096 x 4096 bf16 8.1 us against 7.8, 64 tokens
// 14.4 against 10.9.)
//
// MX: e4m3 operands; a stage's 128 bytes of a row are 128 elements, whose
// scales are one block of 512 bytes per operand.  They land beside the stage
// and go to tensor memory columns of that stage before its MMAs.
//
// FULL: K summed in pieces.  The tensor core cuts each addition into its fp32
// accumulator short, so the error of one long sum grows with K (measured
// 4.9e-6 relative at K = 4096, 1.9e-5 at 16384); sums of at most 512 elements
// (2048 in 8 bits) are added up in registers instead, two accumulators taking turns.
// So are a gated layer's past kLongestSum, whatever the number of tokens (64 x 65536 -> 1024
// bf16 60 us, 61 in one sum; 4096 x 65536 -> 1024 1351, 668 by pairs of CTAs in one).
//
// GATED: a gated layer's two products (matmul_gated.cuh).  The 128 rows are 64 of the
// gate's weights and the same 64 of the up product's, so that both sums of a channel
// and token meet in one CTA: nothing else changes before the epilogue.
#include "matmul.cuh"
#include "matmul_gated.cuh"

#include <type_traits>

namespace bigemm {

namespace {

constexpr int kFewThreads = 256;               // producer, MMA, two idle warps, four that drain
constexpr int kFewA = 128 * kRow;              // bytes of weights per stage

constexpr int kFewStages = 8;                  // at most
// A CTA asks for 110 KB, so that two share an SM and no third kernel that
// allocates tensor memory fits beside them (a cluster whose CTAs could wait for
// tensor memory held by another cluster's would not end), or, where the whole
// grid has an SM per CTA and tiles are large, for most of an SM.
constexpr int kFewShared = 110 * 1024;

template <int BN>
struct FewCfg {
    static constexpr int stage = kFewA + BN * kRow + 2 * kMxBlockBytes;
    static constexpr int half = BN == 128 ? 3 : BN == 64 ? 4 : BN == 32 ? 4 : 5;   // stages in half an SM
    static constexpr int whole = BN == 128 ? 6 : BN == 64 ? 8 : half;              // stages of a CTA alone
    // the ranks' shares of the tokens are whole groups; a rank's sums, of all ranks, are then of at
    // most BN tokens, and of a group more where three ranks share a tile.  Beside the stages for
    // small tiles, over them for large ones.
    static constexpr int group = BN / 8;
    static constexpr int sums = (BN + 2 * group) * 512;
    static constexpr bool beside = BN <= 32;
    static constexpr int bytes(int stages) { return stages * stage + (beside ? sums : 0) + 256 + 1024; }
    static constexpr int smem(int stages) { return bytes(stages) > kFewShared ? bytes(stages) : kFewShared; }
    static_assert(bytes(half) <= kFewShared && (beside || sums <= half * stage), "fits");
    static_assert(whole <= kFewStages && bytes(whole) <= 227 * 1024, "fits");
};

template <int BN, bool MX, bool FULL>
constexpr uint32_t few_cols()
{
    const int n = (FULL ? 2 : 1) * BN + (MX ? 8 * FewCfg<BN>::whole : 0);
    return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : 256;
}

template <bool GATED>
struct FewMaps {
    CUtensorMap w, x;
};
template <>
struct FewMaps<true> {
    CUtensorMap w, x, up;
};
template <bool GATED>
using FewArgs = std::conditional_t<GATED, GatedArgs, MatmulArgs>;

// act(g) u of 8 channels from n on of token m, g and u where they are kept; channels past N are not written.
__device__ __forceinline__ void gated_out8(const GatedArgs &p, int m, int n, float (&g)[8], const float (&u)[8])
{
    if (p.gate) mm_put8(p.gate, m * p.ldgate + n, p.out_dt, p.vec_gate, n, p.N, g);
    if (p.up) mm_put8(p.up, m * p.ldup + n, p.out_dt, p.vec_up, n, p.N, u);
    mm_act_all(p.act, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] *= u[j];
    mm_store8(p, m, n, g);
}

template <int BN, bool MX, bool FULL, bool GATED = false>
__global__ void __launch_bounds__(kFewThreads)
    matmul_few_kernel(const __grid_constant__ FewMaps<GATED> maps, const FewArgs<GATED> p)
{
    static_assert(!GATED || !MX, "16-bit operands and outputs");
    using C = FewCfg<BN>;
    constexpr int kChannels = GATED ? 64 : 128;      // of the output, per CTA
    constexpr int kPieces = kChannels / 8;           // of 8 channels, per token
    const int S = p.stages;
    constexpr int ACC = FULL ? 2 : 1;
    constexpr uint32_t kCols = few_cols<BN, MX, FULL>();
    static_assert(ACC * BN + (MX ? 8 * C::whole : 0) <= (int)kCols, "tensor memory");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sa = smem, *sb = smem + S * kFewA, *ss = sb + S * BN * kRow;   // weights, tokens, scales
    uint64_t *full = reinterpret_cast<uint64_t *>(ss + S * 2 * kMxBlockBytes);
    uint64_t *empty = full + S, *tfull = empty + S, *tempty = tfull + 2, *drain = tempty + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);
    // [split][tokens of a rank][128] sums
    float *part = reinterpret_cast<float *>(C::beside ? ss + S * 2 * kMxBlockBytes + 256 : smem);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = p.split;                       // CTAs of the cluster
    const int rank = split > 1 ? (int)cluster_ctarank() : 0;
    const int ct = (int)blockIdx.x / split, n0 = ct * kChannels;
    const int m0 = (int)blockIdx.y * BN;
    const int kb0 = (int)((long long)rank * p.k_blocks / split), kb1 = (int)((long long)(rank + 1) * p.k_blocks / split);

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&tfull[i], 1), mbar_init(&tempty[i], 4);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&maps.w);
        tma_prefetch_desc(&maps.x);
        if constexpr (GATED) tma_prefetch_desc(&maps.up);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(tmem_holder, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    if (C::beside && split > 1) cluster_arrive();   // this CTA runs: peers may write into its sums
    griddep_enter();

    bool good = true;
    float acc[FULL ? BN : 1];       // FULL, warps 4-7: the sums over finished segments
    if (FULL) {
#pragma unroll
        for (int i = 0; i < (FULL ? BN : 1); ++i) acc[i] = 0.f;
    }

    if (warp == 0) {
        // ------------------------------------------------------ producer
        if (lane == 0) {
            constexpr int per = MX ? kRow : kRow / 2;         // elements of K per stage
            int stage = 0;
            uint32_t phase = 0, last_parity[kFewStages];
            bool issued[kFewStages];
            for (int i = 0; i < kFewStages; ++i) issued[i] = false, last_parity[i] = 0;
            for (int kb = kb0; kb < kb1; ++kb) {
                good = mbar_wait(&empty[stage], phase ^ 1u, p.timeout_ns, abort_flag, p.err);
                if (!good) break;
                mbar_arrive_expect_tx(&full[stage], (uint32_t)(kFewA + BN * kRow + (MX ? 2 * kMxBlockBytes : 0)));
                issued[stage] = true, last_parity[stage] = phase;
                tma_load_2d(sa + stage * kFewA, &maps.w, &full[stage], kb * per, n0);
                if constexpr (GATED) tma_load_2d(sa + stage * kFewA + kFewA / 2, &maps.up, &full[stage], kb * per, n0);
                tma_load_2d(sb + stage * BN * kRow, &maps.x, &full[stage], kb * per, m0);
                if (MX) {
                    uint8_t *s = ss + stage * 2 * kMxBlockBytes;
                    bulk_load(s, p.ws + ((long long)(n0 >> 7) * p.k_blocks + kb) * kMxBlockBytes, kMxBlockBytes,
                              &full[stage]);
                    bulk_load(s + kMxBlockBytes, p.xs + ((long long)(m0 >> 7) * p.k_blocks + kb) * kMxBlockBytes,
                              kMxBlockBytes, &full[stage]);
                }
                if (++stage == S) stage = 0, phase ^= 1u;
            }
            if (!good) {
                int local_abort = 0;
                for (int i = 0; i < S; ++i)
                    if (issued[i]) mbar_wait(&full[i], last_parity[i], p.timeout_ns, &local_abort, p.err);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t idesc = MX ? make_idesc_mx(128, BN)
                                      : make_idesc(p.in_dt == BIGEMM_BF16 ? 1u : 0u, 0u, 0u, 128, BN);
            const uint32_t hi = desc_hi(1024u, 2u);
            // scales: rows of 16 bytes without a swizzle, 8-row groups 128 bytes apart
            const uint32_t s_hi = desc_hi(128u, 0u);
            // a 64-token tile's scales are the first or the second half of their block's columns
            const uint32_t sb_shift = (uint32_t)((m0 & 127) >> 5);
            int stage = 0, a = 0;
            uint32_t phase = 0, acc_phase = 0;
            bool ok = true, any = false;
            for (int k0 = kb0; ok && k0 < kb1; k0 += p.seg_blocks) {
                ok = mbar_wait(&tempty[a], acc_phase ^ 1u, p.timeout_ns, abort_flag, p.err);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(a * BN);
                const int k1 = min(kb1, k0 + p.seg_blocks);
                for (int kb = k0; kb < k1; ++kb) {
                    ok = mbar_wait(&full[stage], phase, p.timeout_ns, abort_flag, p.err);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t a_lo = desc_lo(smem_u32(sa + stage * kFewA), 16u);
                    const uint32_t b_lo = desc_lo(smem_u32(sb + stage * BN * kRow), 16u);
                    if (MX) {
                        const uint32_t s_lo = desc_lo(smem_u32(ss + stage * 2 * kMxBlockBytes), 0u);
                        const uint32_t sf = tmem_base + (uint32_t)(ACC * BN + 8 * stage);
                        tmem_copy_scales(sf, (uint64_t)s_hi << 32 | s_lo);
                        tmem_copy_scales(sf + 4, (uint64_t)s_hi << 32 | (s_lo + (kMxBlockBytes >> 4)));
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k)
                            umma_mx(d, a_lo + 2 * k, hi, b_lo + 2 * k, hi, idesc | (k << 4) | (k << 29), sf,
                                    sf + 4 + sb_shift, (kb > k0 || k > 0) ? 1u : 0u);
                    } else {
                        umma4_kmajor<false>(d, a_lo, hi, b_lo, hi, idesc, kb > k0 ? 1u : 0u);
                    }
                    any = true;
                    umma_commit(&empty[stage]);
                    if (++stage == S) stage = 0, phase ^= 1u;
                }
                if (!ok) break;
                umma_commit(&tfull[a]);
                if (++a == ACC) a = 0, acc_phase ^= 1u;
            }
            if (!ok && any) {
                int local_abort = 0;
                umma_commit(drain);
                mbar_wait(drain, 0, p.timeout_ns, &local_abort, p.err);
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------ other comes to L2 meanwhile
        if (p.combine != BIGEMM_COMBINE_NONE) {
            const int es = p.other_dt == BIGEMM_F32 ? 4 : 2, bytes = min(128, p.N - n0) * es;
            for (int t = lane; t < min(BN, p.M - m0); t += 32) {
                const uint8_t *from = static_cast<const uint8_t *>(p.other) + ((long long)(m0 + t) * p.ldother + n0) * es;
                for (int i = 0; i < bytes; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(from + i));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(from + bytes - 1));
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ------------------------------------------------------ drain: lane = channel, column = token
        const uint32_t lane_base = tmem_base + ((uint32_t)((warp & 3) * 32) << 16);
        int a = 0;
        uint32_t acc_phase = 0;
        for (int k0 = kb0; good && k0 < kb1; k0 += p.seg_blocks) {
            good = mbar_wait_warp(&tfull[a], acc_phase, p.timeout_ns, abort_flag, p.err);
            if (!good || !FULL) break;           // one segment: its sums stay in tensor memory for now
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < BN; c += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(lane_base + (uint32_t)(a * BN + c), r);
                tmem_wait_ld16(r);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[FULL ? c + i : 0] += __uint_as_float(r[i]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[a]);
            if (++a == ACC) a = 0, acc_phase ^= 1u;
        }
    }
    __syncwarp();

    // ---------------------------------------------------------- each token's sums to the rank that finishes it
    const int tokens = min(BN, p.M - m0);
    const int per_rank = ((tokens + split - 1) / split + C::group - 1) / C::group * C::group;
    const int t0 = rank * per_rank, mine = max(0, min(per_rank, tokens - t0));
    // a thread finishes 8 channels, always the same ones, of every 16th (GATED: 32nd) token of the rank's; its bias
    // and its first other are asked for now
    const int c = ((int)threadIdx.x & (kPieces - 1)) * 8;
    float bias[8], bias_up[GATED ? 8 : 1];
#pragma unroll
    for (int j = 0; j < 8; ++j) bias[j] = p.bias && n0 + c + j < p.N ? p.bias[n0 + c + j] : 0.f;
    if constexpr (GATED) {
#pragma unroll
        for (int j = 0; j < 8; ++j) bias_up[j] = p.bias_up && n0 + c + j < p.N ? p.bias_up[n0 + c + j] : 0.f;
    }
    Raw8 other;
    if (!GATED && (int)threadIdx.x < mine * kPieces) mm_other8(p, m0 + t0 + (int)threadIdx.x / kPieces, n0 + c, other);
    if (split > 1) {
        // the sums' memory is free: beside the stages since each peer began, over them since its
        // drain warps saw the last MMA done
        if (!C::beside) cluster_arrive();
        cluster_wait();
    }
    if (warp >= 4) {
        tc_fence_after();
        const uint32_t lane_base = tmem_base + ((uint32_t)((warp & 3) * 32) << 16);
        // slot of this rank in the owner's memory
        const uint32_t at = smem_u32(part + rank * per_rank * 128 + (warp & 3) * 32 + lane);
        uint32_t to = split > 1 ? mapa_shared(at, 0u) : at;
        int owner = 0, t = 0;
#pragma unroll
        for (int c = 0; c < BN; c += 16) {
            if (c >= tokens) break;
            uint32_t r[16];
            if (!FULL) {
                tmem_ld_32x32b_x16(lane_base + (uint32_t)c, r);
                tmem_wait_ld16(r);
            }
            // a group of tokens has one owner (what a last group holds past the tokens is zeros)
#pragma unroll
            for (int g = 0; g < 16; g += C::group) {
                const uint32_t slot = to + (uint32_t)t * 512u;
                if (c + g < tokens) {
#pragma unroll
                    for (int i = g; i < g + C::group; ++i) {
                        const float v = FULL ? acc[FULL ? c + i : 0] : __uint_as_float(r[i]);
                        if (split > 1) st_cluster_f32(slot + (uint32_t)(i - g) * 512u, v);
                        else st_shared_f32(slot + (uint32_t)(i - g) * 512u, v);
                    }
                }
                t += C::group;
                if (t == per_rank && split > 1) {
                    t = 0;
                    to = mapa_shared(at, (uint32_t)min(++owner, split - 1));
                }
            }
        }
        tc_fence_before();
    }
    __syncwarp();
    if (split > 1) {
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }

    // ---------------------------------------------------------- sum over the ranks and epilogue
    // pieces of 8 channels, 16 (8) to a token
    for (int i0 = 0; i0 < mine * kPieces; i0 += kFewThreads) {
        const int i = i0 + (int)threadIdx.x;
        const bool live = i < mine * kPieces;
        const int t = t0 + (live ? i / kPieces : 0);
        const Raw8 now = other;
        if (!GATED && i + kFewThreads < mine * kPieces) mm_other8(p, m0 + t0 + (i + kFewThreads) / kPieces, n0 + c, other);
        float v[8], up[GATED ? 8 : 1];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f, up[GATED ? j : 0] = 0.f;
        if (live) {
            const float4 *from = reinterpret_cast<const float4 *>(part + i / kPieces * 128 + c);
#pragma unroll 4
            for (int s = 0; s < split; ++s) {
                const float4 u0 = from[0], u1 = from[1];
                if constexpr (GATED) {
                    const float4 w0 = from[16], w1 = from[17];
                    up[0] += w0.x, up[1] += w0.y, up[2] += w0.z, up[3] += w0.w;
                    up[4] += w1.x, up[5] += w1.y, up[6] += w1.z, up[7] += w1.w;
                }
                from += per_rank * 32;
                v[0] += u0.x, v[1] += u0.y, v[2] += u0.z, v[3] += u0.w;
                v[4] += u1.x, v[5] += u1.y, v[6] += u1.z, v[7] += u1.w;
            }
            if constexpr (GATED) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += bias[j], up[j] += bias_up[j];
                gated_out8(p, m0 + t, n0 + c, v, up);
            } else {
                mm_epilogue8(p, n0 + c, bias, now, v);
            }
        }
        if (GATED) continue;
        if (p.out_dt == BIGEMM_MXF8) {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = mx_amax(m, v[j]);
            m = mx_amax(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = mx_amax(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t code = mx_scale_code(m);
            if (live) {
                if ((lane & 3) == 0)
                    p.outs[mx_scale_offset(m0 + t, (n0 + c) / kMxGroup, (int)((p.N + 127ll) / 128))] = (uint8_t)code;
                mm_store8_mx(p, m0 + t, n0 + c, v, mx_inv_scale(code));
            }
        } else if (live) {
            mm_store8(p, m0 + t, n0 + c, v);
        }
    }

    if (warp == 1) {
        tc_fence_after();
        __syncwarp();
        tmem_dealloc(tmem_base, kCols);
    }
}

template <int BN, bool MX, bool FULL, bool GATED = false>
cudaError_t launch_one(FewArgs<GATED> a, int split, bool alone, const FewMaps<GATED> &maps, cudaStream_t stream)
{
    a.stages = alone ? FewCfg<BN>::whole : FewCfg<BN>::half;
    auto kern = matmul_few_kernel<BN, MX, FULL, GATED>;
    constexpr int channels = GATED ? 64 : 128;
    static std::atomic<unsigned long long> attr_set{0};   // bit per device: smem opt-in done
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !(attr_set >> dev & 1ull)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   FewCfg<BN>::smem(FewCfg<BN>::whole));
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set |= 1ull << dev;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.N + channels - 1ll) / channels * split), (unsigned)((a.M + (long long)BN - 1) / BN));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = FewCfg<BN>::smem(a.stages);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, maps, a);
}

template <int BN>
cudaError_t launch_bn(const MatmulArgs &a, int split, bool alone, const FewMaps<false> &maps, cudaStream_t s)
{
    if (matmul_in_pieces(a)) {
        if constexpr (BN <= 64)
            return a.in_dt == BIGEMM_MXF8 ? launch_one<BN, true, true>(a, split, alone, maps, s)
                                          : launch_one<BN, false, true>(a, split, alone, maps, s);
        return cudaErrorInvalidValue;   // 128 running sums per thread would spill
    }
    return a.in_dt == BIGEMM_MXF8 ? launch_one<BN, true, false>(a, split, alone, maps, s)
                                  : launch_one<BN, false, false>(a, split, alone, maps, s);
}

}  // namespace

cudaError_t launch_matmul_few(const MatmulArgs &a, FewCut cut, const CUtensorMap &map_w,
                              const CUtensorMap &map_x, cudaStream_t stream)
{
    ProfScope prof("matmul_few", stream);
    // the scales of a 32-token tile inside a block of 128 would start at an odd column of tensor
    // memory, which the MMA does not take
    if (a.in_dt == BIGEMM_MXF8 && cut.bn < 64 && a.M > cut.bn) return cudaErrorInvalidValue;
    const FewMaps<false> maps = {map_w, map_x};
    switch (cut.bn) {
    case 16: return launch_bn<16>(a, cut.split, cut.alone, maps, stream);
    case 32: return launch_bn<32>(a, cut.split, cut.alone, maps, stream);
    case 64: return launch_bn<64>(a, cut.split, cut.alone, maps, stream);
    case 128: return launch_bn<128>(a, cut.split, cut.alone, maps, stream);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_gated_few(const GatedArgs &a, FewCut cut, const CUtensorMap &map_w, const CUtensorMap &map_up,
                             const CUtensorMap &map_x, cudaStream_t stream)
{
    ProfScope prof("matmul_gated_few", stream);
    const FewMaps<true> maps = {map_w, map_x, map_up};
    const bool pieces = a.seg_blocks < a.k_blocks;
    switch (cut.bn) {
    case 16:
        return pieces ? launch_one<16, false, true, true>(a, cut.split, cut.alone, maps, stream)
                      : launch_one<16, false, false, true>(a, cut.split, cut.alone, maps, stream);
    case 32:
        return pieces ? launch_one<32, false, true, true>(a, cut.split, cut.alone, maps, stream)
                      : launch_one<32, false, false, true>(a, cut.split, cut.alone, maps, stream);
    case 64:
        return pieces ? launch_one<64, false, true, true>(a, cut.split, cut.alone, maps, stream)
                      : launch_one<64, false, false, true>(a, cut.split, cut.alone, maps, stream);
    case 128: return pieces ? cudaErrorInvalidValue : launch_one<128, false, false, true>(a, cut.split, cut.alone, maps, stream);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace bigemm
