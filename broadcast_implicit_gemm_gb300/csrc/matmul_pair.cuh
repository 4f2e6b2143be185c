// matmul_pair.cuh -- the skeleton of the pair kernels of 16-bit operands whose tiles
// are not those of one plain product: the gated layer's two products
// (matmul_gated.cu) and the gradients (matmul_back.cu).  A Job says which units of
// work there are, and how each is loaded, multiplied and drained.
//
// As in matmul_many.cu: a pair of CTAs (cta_group::2) per 256 x 256 tile, each CTA
// with 128 of its rows and half of the other operand in 32 KB stages of 64 elements of
// the summed axis (5 or 6 of them), 4 MMAs of 128 cycles each; one warp loads, one issues,
// sixteen drain, and two accumulators fill tensor memory, so that a tile's epilogue
// runs beside the next one's MMAs.  One block per SM walks over its pair's units.
#pragma once
#include "matmul.cuh"
#include "matmul_drain.cuh"

namespace bigemm {

namespace {

// The registers that a block launches with are dealt out anew between the leading
// warpgroup (loads, MMAs) and the four that drain.
struct PairCfg {
    static constexpr int drain = 16, threads = 128 + 32 * drain;
    static constexpr int launch_regs = 96, lead_regs = 56, drain_regs = 104;
    static_assert(lead_regs + drain / 4 * drain_regs <= threads / 128 * launch_regs, "a larger sum would wait for ever");
    static constexpr int bn = 256;
    static constexpr int operand = 128 * kRow, box = 64 * kRow;      // bytes a CTA stages of each; of a TMA box
    static constexpr int smem(int stages, int per_warp) { return stages * 2 * operand + drain * per_warp + 256 + 1024; }
};

// The four MMAs of 64 elements of the summed axis for a CTA pair; an operand's start
// moves by STEP 16-byte units per MMA: 2 within K-major rows, 128 (16 rows) in
// MN-major ones.
template <int A_STEP, int B_STEP>
__device__ __forceinline__ void umma4_pair(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                           uint32_t accum_first)
{
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 ad, bd;\n\t.reg .b32 al, bl;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "setp.eq.b32 q, %5, %5;\n\t"
        "mov.b64 ad, {%1, %3};\n\tmov.b64 bd, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], ad, bd, %4, p;\n\t"
        "add.u32 al, %1, %6;\n\tadd.u32 bl, %2, %7;\n\t"
        "mov.b64 ad, {al, %3};\n\tmov.b64 bd, {bl, %3};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], ad, bd, %4, q;\n\t"
        "add.u32 al, al, %6;\n\tadd.u32 bl, bl, %7;\n\t"
        "mov.b64 ad, {al, %3};\n\tmov.b64 bd, {bl, %3};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], ad, bd, %4, q;\n\t"
        "add.u32 al, al, %6;\n\tadd.u32 bl, bl, %7;\n\t"
        "mov.b64 ad, {al, %3};\n\tmov.b64 bd, {bl, %3};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], ad, bd, %4, q;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accum_first), "n"(A_STEP), "n"(B_STEP)
        : "memory");
}

// Start of an operand in shared memory: rows of 128 bytes in the 128-byte swizzle,
// groups of 8 of them 1 KB apart.  MN-major: two boxes of 64 elements, 8 KB apart.
__device__ __forceinline__ uint32_t operand_lo(uint32_t addr, bool mn) { return desc_lo(addr, mn ? (uint32_t)PairCfg::box : 16u); }

// A lane's 32 sums as 16 words of 16-bit values.
__device__ __forceinline__ void words_of(const float (&v)[32], int dt, uint32_t (&w)[16])
{
    if (dt == BIGEMM_F16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = mm_pack2(v[2 * i], v[2 * i + 1], BIGEMM_F16);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = mm_pack2(v[2 * i], v[2 * i + 1], BIGEMM_BF16);
    }
}

// A warp's 32 rows of WORDS 32-bit words of 16-bit values, in its staging as stage_words
// leaves them, to a matrix of `rows` x `cols` whose rows are off the 16-byte grid, or end inside
// a 16-byte word: a lane
// a word of a row, which a row that starts on an odd element shifts by its neighbour's.
// (A lane a column of 16 rows: 16 x 5632 x 7449 gradients 84 us.)
template <int WORDS>
__device__ __forceinline__ void put_off_grid(void *out, long long ld, long long rows, long long cols, const uint8_t *buf,
                                             int lane, long long m_warp, int n)
{
    constexpr int PER = 32 / WORDS;              // rows at once
    const int l = lane % WORDS, sub = lane / WORDS;
    const long long c = n + 2 * l;
#pragma unroll 4
    for (int r0 = 0; r0 < 32; r0 += PER) {
        if (m_warp + r0 >= rows) break;
        const int r = r0 + sub, key = WORDS == 32 ? r & 7 : (r >> 1) & 3;
        const uint32_t w = *reinterpret_cast<const uint32_t *>(buf + r * WORDS * 4 + (((l >> 2) ^ key) << 4) + (l & 3) * 4);
        const uint32_t before = __shfl_up_sync(0xffffffffu, w, 1, WORDS);
        uint16_t *row = static_cast<uint16_t *>(out) + (m_warp + r) * ld, *at = row + c;
        if (m_warp + r >= rows) continue;
        if (reinterpret_cast<uintptr_t>(row) % 4 == 0) {     // (n is even)
            if (c + 1 < cols) *reinterpret_cast<uint32_t *>(at) = w;
            else if (c < cols) *at = (uint16_t)w;
        } else {
            if (l > 0 && c < cols) *reinterpret_cast<uint32_t *>(at - 1) = __funnelshift_r(before, w, 16);
            if (l > 0 && c == cols) at[-1] = (uint16_t)(before >> 16);
            if (l == 0 && c < cols) *at = (uint16_t)w;
            if (l == WORDS - 1 && c + 1 < cols) at[1] = (uint16_t)(w >> 16);
        }
    }
    __syncwarp();                                // before the staging is written again
}

// Whether TMA may store a box of `box` 16-bit columns from column n on of a matrix of `cols`.  It
// leaves alone rows past the matrix, but is not exact to the element at the end of a row (the
// element behind the last of 15, in rows of 16, became 0): a row has to end with a 16-byte word.
__device__ __forceinline__ bool whole_words(long long cols, int n, int box) { return cols % 8 == 0 || n + box <= cols; }

// A warp's 32 x 32 sums, a lane's row in v, to a 16-bit matrix, on the 16-byte grid
// (by_rows) by TMA.
template <int PER_WARP>
__device__ __forceinline__ void put16(const CUtensorMap *map, bool by_rows, void *out, long long ld, int dt, long long rows,
                                      long long cols, uint8_t *stage, int &piece, int lane, long long m_warp, int n,
                                      const float (&v)[32])
{
    uint32_t w[16];
    words_of(v, dt, w);
    const uint8_t *buf = stage_words<PER_WARP, 16>(stage, piece, lane, w);
    if (!by_rows || !whole_words(cols, n, 32)) {
        put_off_grid<16>(out, ld, rows, cols, buf, lane, m_warp, n);
    } else if (lane == 0 && m_warp < rows) {
        tma_store_2d(map, buf, n, (int)m_warp);
        bulk_commit();
    }
}

// Job:
//   stages of both operands, per_warp bytes of output staging
//   Args (with timeout_ns, err), Maps, Unit (with k0, k1: its blocks of the summed axis)
//   static bool unit(p, turn, pair, pairs, Unit &)   the pair's unit of this turn; false: none left
//   static void load(maps, p, u, kb, rank, sa, sb, bar)   this CTA's 2 x 16 KB of a block, counted on bar
//   static void mma(p, u, d, a, b, accum)   a block's MMAs from shared addresses a and b
//   static void beside(p, i, count, lane)   what one of the `count` warps does that are left over
//   static void drain(maps, p, u, rank, q, h, tmem, stage, piece, lane)   a warp's 32 rows (q of 4)
//       by 64 columns (h of 4) of this CTA's sums, at tensor-memory address tmem (of the quarter's lanes, column 0)
template <class Job>
__global__ void __launch_bounds__(PairCfg::threads, 1)
    matmul_pair_kernel(const __grid_constant__ typename Job::Maps maps, const typename Job::Args p)
{
    using C = PairCfg;
    constexpr int S = Job::stages, PER_WARP = Job::per_warp;
    static_assert(C::smem(S, PER_WARP) <= 227 * 1024, "shared memory");
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sa = smem, *sb = sa + S * C::operand, *out_stage = sb + S * C::operand;
    uint64_t *full = reinterpret_cast<uint64_t *>(out_stage + C::drain * PER_WARP);
    uint64_t *empty = full + S, *tfull = empty + S, *tempty = tfull + 2, *drain = tempty + 2;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        // an accumulator comes back from both CTAs' drain warps
        for (int i = 0; i < 2; ++i) mbar_init(&tfull[i], 1), mbar_init(&tempty[i], 2 * C::drain);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc_pair(tmem_holder, 512);
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
                const uint32_t full_even = mapa_shared(smem_u32(full), 0);
                int stage = 0;
                uint32_t phase = 0, last_parity[S];
                bool issued[S], ok = true;
                for (int i = 0; i < S; ++i) issued[i] = false, last_parity[i] = 0;
                typename Job::Unit u;
                for (int turn = 0; ok && Job::unit(p, turn, pair, pairs, u); ++turn) {
                    for (int kb = u.k0; kb < u.k1; ++kb) {
                        ok = mbar_wait(&empty[stage], phase ^ 1u, p.timeout_ns, abort_flag, p.err);
                        if (!ok) break;
                        if (leader) mbar_arrive_expect_tx(&full[stage], 4u * (uint32_t)C::operand);
                        issued[stage] = true, last_parity[stage] = phase;
                        Job::load(maps, p, u, kb, rank, sa + stage * C::operand, sb + stage * C::operand,
                                  full_even + (uint32_t)stage * 8u);
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
                int stage = 0, a = 0;
                uint32_t phase = 0, acc_phase = 0;
                bool ok = true, any = false;
                typename Job::Unit u;
                for (int turn = 0; ok && Job::unit(p, turn, pair, pairs, u); ++turn) {
                    ok = mbar_wait(&tempty[a], acc_phase ^ 1u, p.timeout_ns, abort_flag, p.err);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem_base + (uint32_t)(a * C::bn);
                    for (int kb = u.k0; kb < u.k1; ++kb) {
                        ok = mbar_wait(&full[stage], phase, p.timeout_ns, abort_flag, p.err);
                        if (!ok) break;
                        tc_fence_after();
                        Job::mma(p, u, d, smem_u32(sa + stage * C::operand), smem_u32(sb + stage * C::operand),
                                 kb > u.k0 ? 1u : 0u);
                        any = true;
                        umma_commit_pair_mc(&empty[stage], (uint16_t)3u);
                        if (++stage == S) stage = 0, phase ^= 1u;
                    }
                    if (!ok) break;
                    umma_commit_pair_mc(&tfull[a], (uint16_t)3u);
                    if (++a == 2) a = 0, acc_phase ^= 1u;
                }
                if (!ok && any) {
                    int local_abort = 0;
                    umma_commit_pair(drain);
                    mbar_wait(drain, 0, p.timeout_ns, &local_abort, p.err);
                }
            }
        } else {
            Job::beside(p, (int)blockIdx.x * 2 + warp - 2, 2 * (int)gridDim.x, lane);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::drain_regs));
        // ------------------------------------------------------ drain and epilogue
        const int q = warp & 3, h = (warp - 4) >> 2;
        const uint32_t lane_base = tmem_base + ((uint32_t)(q * 32) << 16);
        const uint32_t tempty_even = mapa_shared(smem_u32(tempty), 0);
        uint8_t *stage = out_stage + (warp - 4) * PER_WARP;
        int a = 0, piece = 0;
        uint32_t acc_phase = 0;
        typename Job::Unit u;
        for (int turn = 0; Job::unit(p, turn, pair, pairs, u); ++turn) {
            if (!mbar_wait_warp(&tfull[a], acc_phase, p.timeout_ns, abort_flag, p.err)) break;
            tc_fence_after();
            Job::drain(maps, p, u, rank, q, h, lane_base + (uint32_t)(a * C::bn), stage, piece, lane);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty_even + (uint32_t)a * 8u);
            if (++a == 2) a = 0, acc_phase ^= 1u;
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
        tmem_dealloc_pair(tmem_base, 512);
    }
}

template <class Job>
cudaError_t launch_pairs(const typename Job::Args &a, const typename Job::Maps &maps, int pairs, cudaStream_t stream)
{
    auto kern = matmul_pair_kernel<Job>;
    constexpr int smem = PairCfg::smem(Job::stages, Job::per_warp);
    static std::atomic<unsigned long long> attr_set{0};   // bit per device: smem opt-in done
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !(attr_set >> dev & 1ull)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        // the split of registers counts on what the block is launched with
        cudaFuncAttributes fa;
        const cudaError_t f = cudaFuncGetAttributes(&fa, kern);
        if (f != cudaSuccess) return f;
        if (fa.numRegs != PairCfg::launch_regs) return cudaErrorInvalidConfiguration;
        if (dev < 64) attr_set |= 1ull << dev;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2u * (unsigned)pairs);
    cfg.blockDim = dim3(PairCfg::threads);
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

}  // namespace

}  // namespace bigemm
