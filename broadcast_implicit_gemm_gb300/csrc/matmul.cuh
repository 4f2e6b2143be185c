// matmul.cuh -- pieces shared by the matrix-product kernels: the problem as a
// kernel sees it, the epilogue's arithmetic, and the tcgen05 wrappers that only
// these kernels use (block-scaled MMA, the copy of scales into tensor memory).
//
//   out[m,n] = combine(act(sum_k x[m,k] w[n,k] + bias[n]), other[m,n])
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "mx.cuh"
#include "ptx.cuh"

namespace bigemm {

struct MatmulArgs {
    int M, N, K;                     // tokens, output channels, the summed length
    int in_dt, out_dt, other_dt;     // bigemm_dtype
    int act, combine;
    const void *x, *w;               // [M,K], [N,K]; rows ldx and ldw elements apart
    long long ldx, ldw, ldo, ldother;
    const uint8_t *xs, *ws;          // MXFP8: blocked scales
    const float *bias;               // [N] or null
    const void *other;               // [M,N] or null
    void *out;
    uint8_t *outs;                   // MXFP8 output: blocked scales
    bool vec_out, vec_other;         // rows start on 16-byte boundaries (8 for e4m3 outputs)
    bool vec_bias;                   // bias starts on one
    int k_blocks;                    // 128-byte pieces of a row
    int seg_blocks;                  // of them, how many one tensor-memory accumulator sums
    int split;                       // few tokens: CTAs that share a tile's blocks, each at least one
    int stages;                      // few tokens: of shared memory
    int m_tiles, n_tiles;            // many tokens: tiles of the output, 256 tokens by BN channels
    bool by_rows;                    // many tokens: out and other have their rows on the 16-byte grid
    unsigned long long timeout_ns;
    int *err;
};

// Whether K is summed in pieces, added up in registers (matmul_few.cu says why):
// for 32-bit outputs, and for MXFP8 ones, where the error of one long sum shows as
// elements and scales rounded the other way (4096 x 8192 x 8192 with gelu, mean of 30
// inputs: 730 of 34 million elements and 0.7 of a million scales, in pieces 220 and
// 0.17; a plain fp32 product 1120 and 0.10).  What a 16-bit output's one rounding
// leaves is 25 times that error or more.
inline bool matmul_in_pieces(const MatmulArgs &a) { return a.out_dt == BIGEMM_F32 || a.out_dt == BIGEMM_MXF8; }

// Elements of a summed axis that one tensor-memory accumulator takes at most in a gated
// layer's products and in gradients.  It cuts each addition short, always towards zero: f16
// terms of one sign, 4096 x 4096 gradients, leave dw 2e-5 of the sum too small at 4096 tokens,
// 2e-4 at 32768 (as much as rounding dw once leaves in the 2-norm), 8e-4 at 131072, 3e-3 at
// 524288.
constexpr int kLongestSum = 32768;

namespace {

constexpr int kRow = 128;            // bytes of one row in a stage: a 128-byte swizzle row

// act(z) of one kind.  silu and the tanh form of gelu are both z / (1 + exp(-t)):
// with tanh(u) = 2 / (1 + exp(-2u)) - 1, gelu's 0.5 z (1 + tanh(u)) is
// z / (1 + exp(-2u)), u = sqrt(2/pi) (z + 0.044715 z^3).  The power of two and
// the reciprocal are the hardware's (2 and 1 ulp); an overflowing power gives 0.
__device__ __forceinline__ float mm_sigmoid2(float z, float t)   // z / (1 + 2^-t)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-t));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return z * r;
}

// z Phi(z).  For a = |z|, Phi(-a) = t P(t) exp(-a^2 / 2) with t = 1 / (1 + 0.305 a):
// P of degree 7, fitted by the Remez exchange to the least relative error of
// Phi(-a) exp(a^2 / 2) over 0 <= a <= 13.5 (9.4e-8), so that the small values of
// negative z are as exact as the others.  What is left there is the exponent's
// rounding, z^2 2^-24: 8e-7 at z = -3, 2e-6 at -6.  (0.5 z (1 + erf) takes erff, twice
// the instructions, and loses all digits towards z = -5.5.)
__device__ __forceinline__ float mm_normal_below(float z, float e)   // Phi(z), e = exp(-z^2 / 2)
{
    float t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(fabsf(z), 0.305f, 1.f)));
    float q = fmaf(t, 0.0366991852980769f, -0.15298828749580104f);    // Phi(-|z|)
    q = fmaf(t, q, 0.1857168536271935f);
    q = fmaf(t, q, -0.0379767771644137f);
    q = fmaf(t, q, 0.12102164846056378f);
    q = fmaf(t, q, 0.10342087620163884f);
    q = fmaf(t, q, 0.12246681530010683f);
    q = fmaf(t, q, 0.12163973276490539f);
    q *= t * e;
    return z < 0.f ? q : 1.f - q;
}

__device__ __forceinline__ float mm_gelu(float z)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * z * (-0.5f * 1.4426950408889634f)));
    return z * mm_normal_below(z, e);
}

template <int ACT>
__device__ __forceinline__ float mm_act(float z)
{
    constexpr float kLog2e = 1.4426950408889634f;
    if (ACT == BIGEMM_ACT_RELU) return z < 0.f ? 0.f : z;
    if (ACT == BIGEMM_ACT_GELU) return mm_gelu(z);
    if (ACT == BIGEMM_ACT_GELU_TANH) {
        constexpr float c = 2.f * 0.79788456080286536f * kLog2e;      // 2 sqrt(2/pi) log2(e)
        return mm_sigmoid2(z, z * (c + c * 0.044715f * (z * z)));
    }
    if (ACT == BIGEMM_ACT_SILU) return mm_sigmoid2(z, kLog2e * z);
    return z;
}

template <int ACT, int N>
__device__ __forceinline__ void mm_act_each(float (&v)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = mm_act<ACT>(v[i]);
}

// act of N values, chosen once for all of them.
template <int N>
__device__ __forceinline__ void mm_act_all(int act, float (&v)[N])
{
    switch (act) {
    case BIGEMM_ACT_RELU: mm_act_each<BIGEMM_ACT_RELU>(v); break;
    case BIGEMM_ACT_GELU: mm_act_each<BIGEMM_ACT_GELU>(v); break;
    case BIGEMM_ACT_GELU_TANH: mm_act_each<BIGEMM_ACT_GELU_TANH>(v); break;
    case BIGEMM_ACT_SILU: mm_act_each<BIGEMM_ACT_SILU>(v); break;
    default: break;
    }
}

__device__ __forceinline__ float mm_combine(int how, float z, float o)
{
    return how == BIGEMM_COMBINE_ADD ? z + o : how == BIGEMM_COMBINE_MUL ? z * o : z;
}

// The value of an element's bits.
__device__ __forceinline__ float mm_value(uint32_t bits, int dt)
{
    return dt == BIGEMM_F32   ? __uint_as_float(bits)
           : dt == BIGEMM_F16 ? __half2float(__ushort_as_half((unsigned short)bits))
                              : __uint_as_float(bits << 16);
}

// 8 16-bit values.
__device__ __forceinline__ void mm_unpack8(const uint4 &u, int dt, float (&v)[8])
{
    const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float2 f;
        if (dt == BIGEMM_F16)
            f = __half22float2(*reinterpret_cast<const __half2 *>(&q[j]));
        else
            f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&q[j]));
        v[2 * j] = f.x, v[2 * j + 1] = f.y;
    }
}

// 8 consecutive values from element i on, i * element size on a 16-byte boundary.
__device__ __forceinline__ void mm_load8(const void *p, long long i, int dt, float (&v)[8])
{
    if (dt == BIGEMM_F32) {
        const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 b = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i + 4);
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        return;
    }
    mm_unpack8(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i), dt, v);
}

__device__ __forceinline__ uint32_t mm_pack2(float a, float b, int dt)
{
    if (dt == BIGEMM_F16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 8 consecutive channels of other as they lie in memory: whole words where rows
// are on the 16-byte grid, else an element each.
struct Raw8 {
    uint32_t e[8];
};

__device__ __forceinline__ void mm_other8(const MatmulArgs &a, int m, int n, Raw8 &r)
{
    if (a.combine == BIGEMM_COMBINE_NONE) return;
    const long long at = (long long)m * a.ldother + n;
    const bool wide = a.other_dt == BIGEMM_F32;
    if (a.vec_other && n + 8 <= a.N) {
        const uint4 *from = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(a.other) + at * (wide ? 4 : 2));
        const uint4 u = from[0];
        r.e[0] = u.x, r.e[1] = u.y, r.e[2] = u.z, r.e[3] = u.w;
        if (wide) {
            const uint4 w = from[1];
            r.e[4] = w.x, r.e[5] = w.y, r.e[6] = w.z, r.e[7] = w.w;
        }
    } else if (wide) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.e[j] = n + j < a.N ? static_cast<const uint32_t *>(a.other)[at + j] : 0u;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r.e[j] = n + j < a.N ? static_cast<const uint16_t *>(a.other)[at + j] : 0u;
    }
}

// act(v + b), combined with other, in place; channels past N become 0.
__device__ __forceinline__ void mm_epilogue8(const MatmulArgs &a, int n, const float (&b)[8], const Raw8 &o, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += b[j];
    mm_act_all(a.act, v);
    if (a.combine != BIGEMM_COMBINE_NONE) {
        float f[8];
        if (a.other_dt != BIGEMM_F32 && a.vec_other && n + 8 <= a.N) {
            mm_unpack8(make_uint4(o.e[0], o.e[1], o.e[2], o.e[3]), a.other_dt, f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = mm_value(o.e[j], a.other_dt);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = mm_combine(a.combine, v[j], f[j]);
    }
    if (n + 8 > a.N) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = n + j < a.N ? v[j] : 0.f;
    }
}

// 8 channels from n on of a row of N, at element `at` of a 32- or 16-bit matrix; vec:
// its rows start on 16-byte boundaries.
template <typename T>
__device__ __forceinline__ void mm_store_each(void *out, long long at, int n, int N, const float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (n + j < N) static_cast<T *>(out)[at + j] = T(v[j]);
}

__device__ __forceinline__ void mm_put8(void *out, long long at, int dt, bool vec, int n, int N, const float (&v)[8])
{
    if (vec && n + 8 <= N) {
        if (dt == BIGEMM_F32) {
            float *p = static_cast<float *>(out) + at;
            *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at) =
                make_uint4(mm_pack2(v[0], v[1], dt), mm_pack2(v[2], v[3], dt), mm_pack2(v[4], v[5], dt),
                           mm_pack2(v[6], v[7], dt));
        }
    } else if (dt == BIGEMM_F32) {
        mm_store_each<float>(out, at, n, N, v);
    } else if (dt == BIGEMM_F16) {
        mm_store_each<__half>(out, at, n, N, v);
    } else {
        mm_store_each<__nv_bfloat16>(out, at, n, N, v);
    }
}

// 8 channels of a 32- or 16-bit output.
__device__ __forceinline__ void mm_store8(const MatmulArgs &a, int m, int n, const float (&v)[8])
{
    mm_put8(a.out, (long long)m * a.ldo + n, a.out_dt, a.vec_out, n, a.N, v);
}

// 8 channels of an e4m3 output, 1 / scale given.
__device__ __forceinline__ void mm_store8_mx(const MatmulArgs &a, int m, int n, const float (&v)[8], float inv)
{
    const uint32_t lo = mx_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    const uint32_t hi = mx_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    uint8_t *p = static_cast<uint8_t *>(a.out) + (long long)m * a.ldo + n;
    if (a.vec_out && n + 8 <= a.N) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (n + j < a.N) p[j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
    }
}

// ------------------------------------------------------------------ wrappers
// Untiled bulk copy into shared memory: both addresses on 16-byte boundaries,
// a multiple of 16 bytes.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// 512 bytes of scales (a block of 128 rows by 4 groups) from shared memory into
// four tensor-memory columns: 32 rows of 16 bytes, repeated for the four lane
// quadrants.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint64_t sdesc)
{
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

// D (+)= (A scaled) * (B scaled), e4m3 operands with an E8M0 scale per 32
// elements of K; the scales' byte within their tensor-memory column is in idesc.
__device__ __forceinline__ void umma_mx(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                        uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t accum)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
        "mov.b64 ad, {%1, %2};\n\t"
        "mov.b64 bd, {%3, %4};\n\t"
        "setp.ne.b32 p, %8, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], ad, bd, %5, [%6], [%7], p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(sa), "r"(sb), "r"(accum)
        : "memory");
}

// Instruction descriptor of the block-scaled MMA for K-major e4m3 operands and
// E8M0 scales: bit 23 the scales' type, N >> 3 at bit 17, M >> 7 at bit 27; the
// scales' byte goes to bits 4 (B) and 29 (A).
__host__ __device__ constexpr uint32_t make_idesc_mx(uint32_t M, uint32_t N)
{
    return (1u << 23) | ((N >> 3) << 17) | ((M >> 7) << 27);
}

// The same for a CTA pair: the copy goes from each CTA's shared memory into its
// own tensor memory, the MMA is the pair's.
__device__ __forceinline__ void tmem_copy_scales_pair(uint32_t taddr, uint64_t sdesc)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

__device__ __forceinline__ void umma_mx_pair(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                             uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t accum)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\t"
        "mov.b64 ad, {%1, %2};\n\t"
        "mov.b64 bd, {%3, %4};\n\t"
        "setp.ne.b32 p, %8, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], ad, bd, %5, [%6], [%7], p;\n\t}" ::"r"(d),
        "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(sa), "r"(sb), "r"(accum)
        : "memory");
}

// A 2-D box into this CTA's shared memory, counted on a barrier of either CTA
// of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, uint32_t cluster_bar, int c0, int c1)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(cluster_bar), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int c0, int c1)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                 "r"(smem_u32(src)), "r"(c0), "r"(c1)
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15])
                 :
                 : "memory");
}

// A store into shared memory of a CTA of the cluster (address from mapa_shared).
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ void st_shared_f32(uint32_t addr, float v)
{
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// The two halves of a barrier over all threads of the cluster.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

}  // namespace

// The kernel for few tokens (matmul_few.cu).  How a product is cut: tokens per
// tile (16, 32, 64 or 128), CTAs that share one tile's K, and whether each has
// an SM to itself.
struct FewCut {
    int bn, split;
    bool alone;
};
cudaError_t launch_matmul_few(const MatmulArgs &a, FewCut cut, const CUtensorMap &map_w, const CUtensorMap &map_x,
                              cudaStream_t stream);

// The kernel for many tokens (matmul_many.cu): tiles of 256 tokens by bn (128 or
// 256) channels.  maps: x, w, scales of x, scales of w, out.
constexpr int kManyTokens = 256;
struct ManyMaps {
    CUtensorMap x, w, xs, ws, out;
};
cudaError_t launch_matmul_many(const MatmulArgs &a, int bn, int sms, const ManyMaps &maps, cudaStream_t stream);

// Operands copied to rows on the 16-byte grid (matmul_pack.cu); rows = 0: none.
struct PackOperand {
    const uint8_t *src;
    uint8_t *dst;
    long long rows, src_pitch, dst_pitch, bytes, runs;     // bytes: of a row
};
constexpr int kPackMost = 3;
struct PackArgs {
    PackOperand op[kPackMost];
    long long items[kPackMost];      // up to the end of each
};
cudaError_t launch_matmul_pack(PackArgs &a, cudaStream_t stream);

}  // namespace bigemm
