// norm.cuh -- the kernels of norm.cu: the root-mean-square norm with the
// residual's addition, and pieces of it that the MXFP8 quantisation shares.
// A translation unit per input type instantiates the norm (norm_*.cu).
//
// A row stays in registers between its sum of squares and its outputs, so each
// byte moves once.  A thread holds pieces of 8 consecutive elements (16 bytes
// of a 16-bit type); the 32 elements of an MXFP8 scale are four neighbouring
// lanes.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "internal.h"
#include "mx.cuh"
#include "ptx.cuh"
#include "unaligned.cuh"

namespace bigemm {

struct NormArgs {
    int cols, col_blocks, pieces;     // pieces: of a row, padded to whole blocks of scales for MXFP8
    long long rows, ldx, ldr, ldh, ldo;
    const void *x, *residual;
    const float *weight;
    bool vec_weight;                  // there, on a 16-byte boundary
    float eps, inv_cols;              // 1 / cols
    void *h, *out;
    uint8_t *scale;
};

enum OutForm { OUT_SAME = 0, OUT_F32 = 1, OUT_MX = 2 };

namespace {

constexpr int kPiece = 8;            // elements per thread and step
constexpr int kMaxCols = 1 << 30;    // column indices are in 32 bits, byte offsets in 64

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <typename T>
struct alignas(16) Piece {
    T e[kPiece];
};

// Two products in one instruction.
__device__ __forceinline__ void mul2(float a0, float a1, float b0, float b1, float &c0, float &c1)
{
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 c, a, b;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "=f"(c0), "=f"(c1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

__device__ __forceinline__ void scale8(const float (&v)[kPiece], float by, float (&w)[kPiece])
{
#pragma unroll
    for (int i = 0; i < kPiece; i += 2) mul2(v[i], v[i + 1], by, by, w[i], w[i + 1]);
}

// 8 elements as they lie in memory.
template <typename T>
struct Raw {
    uint4 q[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ void unpack(const Raw<T> &p, float (&v)[kPiece])
{
    const T *e = reinterpret_cast<const T *>(&p);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) v[i] = to_f32<T>(e[i]);
}

// A piece on its way: 8 elements from column c on (up to 7 below 0 where pieces
// are shifted), zeros outside the row.  VEC: it starts on a 16-byte boundary;
// else a 16-bit piece is two aligned loads and a shift that waits until it is
// used, so that a thread's pieces are all in flight together.
template <typename T, bool VEC>
struct Held {
    static constexpr bool wide = !VEC && sizeof(T) == 2;
    std::conditional_t<wide, Wide, Raw<T>> d;
};

template <typename T>
__device__ __forceinline__ int first_byte(int c) { return c < 0 ? -c * (int)sizeof(T) : 0; }
template <typename T>
__device__ __forceinline__ int last_byte(int c, int cols)
{
    return c >= cols ? 0 : min(kPiece, cols - c) * (int)sizeof(T);
}

template <typename T, bool VEC>
__device__ __forceinline__ void hold(const T *row, int c, int cols, const Span &span, Held<T, VEC> &h)
{
    if constexpr (Held<T, VEC>::wide) {
        h.d = wide_load(reinterpret_cast<const uint8_t *>(row) + (long long)c * (int)sizeof(T), first_byte<T>(c),
                        last_byte<T>(c, cols), span);
    } else if (VEC && c + kPiece <= cols) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) h.d.q[i] = reinterpret_cast<const uint4 *>(row + c)[i];
    } else {
        T *e = reinterpret_cast<T *>(&h.d);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) e[i] = (VEC || c + i >= 0) && c + i < cols ? row[c + i] : from_f32<T>(0.f);
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void take(const Held<T, VEC> &h, int c, int cols, float (&v)[kPiece])
{
    if constexpr (Held<T, VEC>::wide) {
        Raw<T> r;
        r.q[0] = wide_take(h.d, first_byte<T>(c), last_byte<T>(c, cols));
        unpack<T>(r, v);
    } else {
        unpack<T>(h.d, v);
    }
}

__device__ __forceinline__ Span span_of(const void *p, long long rows, long long ld, int cols, size_t es)
{
    const uint8_t *b = static_cast<const uint8_t *>(p);
    return {b, b + ((rows - 1) * ld + cols) * (long long)es};
}

// 8 elements to column c on, those inside the row.  Off the 16-byte grid a
// piece that happens to start on it goes whole all the same.
template <typename T, bool VEC>
__device__ __forceinline__ void store_piece(T *row, int c, int cols, const float (&v)[kPiece])
{
    const bool inside = (VEC || c >= 0) && c + kPiece <= cols;
    if (inside && (VEC || reinterpret_cast<uintptr_t>(row + c) % 16 == 0)) {
        Piece<T> p;
#pragma unroll
        for (int i = 0; i < kPiece; ++i) p.e[i] = from_f32<T>(v[i]);
        *reinterpret_cast<Piece<T> *>(row + c) = p;
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if ((VEC || c + i >= 0) && c + i < cols) row[c + i] = from_f32<T>(v[i]);
    }
}

// One piece of an MXFP8 row: every lane of the warp takes part, `live` lanes
// hold a piece inside the row padded to whole blocks of scales.  scale: of the
// row.  VEC: the e4m3 piece starts on an 8-byte boundary.
template <bool VEC>
__device__ __forceinline__ void store_mx_piece(uint8_t *row, uint8_t *scale, int c, int cols, bool live,
                                               const float (&v)[kPiece])
{
    float top = mx_amax(mx_amax(mx_amax(v[0], v[1]), mx_amax(v[2], v[3])),
                        mx_amax(mx_amax(v[4], v[5]), mx_amax(v[6], v[7])));
    top = mx_amax(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = mx_amax(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const uint32_t code = mx_scale_code(top);
    if (!live) return;
    if ((threadIdx.x & 3) == 0) scale[mx_scale_group(c / kMxGroup)] = (uint8_t)code;
    const float inv = mx_inv_scale(code);
    float w[kPiece];
    scale8(v, inv, w);
    const uint32_t lo = mx_pack4(w[0], w[1], w[2], w[3]), hi = mx_pack4(w[4], w[5], w[6], w[7]);
    if (VEC && c + kPiece <= cols) {
        *reinterpret_cast<uint2 *>(row + c) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (c + i < cols) row[c + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
}


__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The outputs of one piece, from column c on.
template <int FORM, typename T, bool VEC>
__device__ __forceinline__ void norm_out(const NormArgs &a, long long r, int p, int c, float inv,
                                         const float (&h)[kPiece], const float (&g)[kPiece])
{
    if (a.h) store_piece<T, VEC>(static_cast<T *>(a.h) + r * a.ldh, c, a.cols, h);
    float y[kPiece];
    scale8(h, inv, y);
#pragma unroll
    for (int i = 0; i < kPiece; i += 2) mul2(y[i], y[i + 1], g[i], g[i + 1], y[i], y[i + 1]);
    if (FORM == OUT_MX && c + kPiece > a.cols) {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) y[i] = c + i < a.cols ? y[i] : 0.f;
    }
    if (FORM == OUT_MX)
        store_mx_piece<VEC>(static_cast<uint8_t *>(a.out) + r * a.ldo, a.scale + mx_scale_row(r, a.col_blocks), c, a.cols,
                            p < a.pieces, y);
    else if (FORM == OUT_F32)
        store_piece<float, VEC>(static_cast<float *>(a.out) + r * a.ldo, c, a.cols, y);
    else
        store_piece<T, VEC>(static_cast<T *>(a.out) + r * a.ldo, c, a.cols, y);
}

// How far a row's pieces are shifted to the left, so that they start on the
// output's 16-byte boundaries: not at all on the grid, and not for MXFP8, whose
// groups start at column 0.
template <int FORM, typename T, bool VEC>
__device__ __forceinline__ int row_shift(const NormArgs &a, long long r)
{
    if (VEC || FORM == OUT_MX) return 0;
    constexpr int es = FORM == OUT_F32 ? 4 : (int)sizeof(T);
    return (int)((reinterpret_cast<uintptr_t>(a.out) + (uintptr_t)(r * a.ldo) * es) % 16) / es;
}

__device__ __forceinline__ void load_weight(const NormArgs &a, int c, float (&g)[kPiece])
{
    if (a.vec_weight && c % 4 == 0 && c >= 0 && c + kPiece <= a.cols) {
        const float4 u = *reinterpret_cast<const float4 *>(a.weight + c);
        const float4 w = *reinterpret_cast<const float4 *>(a.weight + c + 4);
        g[0] = u.x, g[1] = u.y, g[2] = u.z, g[3] = u.w, g[4] = w.x, g[5] = w.y, g[6] = w.z, g[7] = w.w;
        return;
    }
#pragma unroll
    for (int i = 0; i < kPiece; ++i) g[i] = a.weight && c + i >= 0 && c + i < a.cols ? a.weight[c + i] : 1.f;
}

// Threads of a block with so many per row at most, and threads per SM that its
// registers leave room for: 1024 (64 registers), half as many for 32-bit rows
// and for rows off the 16-byte grid, which hold twice the bytes.
constexpr int norm_threads(int tpr) { return tpr < 128 ? 128 : tpr; }
constexpr int norm_room(size_t es, bool vec) { return es == 4 || !vec ? 512 : 1024; }
constexpr int norm_blocks(int tpr, size_t es, bool vec)
{
    return norm_room(es, vec) < norm_threads(tpr) ? 1 : norm_room(es, vec) / norm_threads(tpr);
}

// TPR threads per row at most (a warp, or the block), PPT pieces per thread in
// registers; a block walks over its rows and loads the next one before it
// sums the present one, so that memory works through the sums and the barrier.
// RES: there is a residual, and the weights come from L1 again for each row,
// because the rows in flight need the registers (16384 x 4096 f16: 6.2 TB/s).
// Without one they stay in registers: L1 delivered more of them than of rows
// (the same rows to MXFP8 took 54 us with them from L1, 37 us so).
// EXACT: the block has all of TPR (on the 16-byte grid, where reading the size of
// the block at run time costs: 8192 x 8192 f16 to MXFP8 38.8 us, 41.7 so).
// Otherwise it has the warps that the row needs (4096 x 2049 f16 with a residual:
// 36.6 us with TPR threads, 22.9 so).
template <typename T, int FORM, bool RES, int TPR, int PPT, bool VEC, bool EXACT>
__global__ void __launch_bounds__(norm_threads(TPR), norm_blocks(TPR, sizeof(T), VEC)) rmsnorm_kernel(const NormArgs a)
{
    griddep_enter();
    constexpr int THREADS = norm_threads(TPR), ROWS = THREADS / TPR;
    static_assert(TPR == 32 || ROWS == 1, "a row has a warp or the block");
    __shared__ float4 part[2][THREADS / 128];
    const int tpr = TPR == 32 || EXACT ? TPR : (int)blockDim.x, t = TPR == 32 ? (int)threadIdx.x & 31 : (int)threadIdx.x;
    if (TPR > 32 && !EXACT) {
        // a block may have fewer warps than the sums have places
        for (int i = threadIdx.x; i < 2 * THREADS / 32; i += blockDim.x) reinterpret_cast<float *>(part)[i] = 0.f;
        __syncthreads();
    }
    const long long step = (long long)gridDim.x * ROWS;
    long long r = (long long)blockIdx.x * ROWS + (TPR == 32 ? threadIdx.x / 32 : 0);
    Held<T, VEC> x[PPT], res[RES ? PPT : 1];
    const Span x_span = span_of(a.x, a.rows, a.ldx, a.cols, sizeof(T));
    const Span res_span = RES ? span_of(a.residual, a.rows, a.ldr, a.cols, sizeof(T)) : x_span;
    auto load = [&](long long row) {
        if (row >= a.rows) return;
        const int c0 = t * kPiece - row_shift<FORM, T, VEC>(a, row);
#pragma unroll
        for (int s = 0; s < PPT; ++s)
            hold<T, VEC>(static_cast<const T *>(a.x) + row * a.ldx, c0 + s * tpr * kPiece, a.cols, x_span, x[s]);
        if (RES) {
#pragma unroll
            for (int s = 0; s < PPT; ++s)
                hold<T, VEC>(static_cast<const T *>(a.residual) + row * a.ldr, c0 + s * tpr * kPiece, a.cols, res_span,
                             res[RES ? s : 0]);
        }
    };
    float kept[RES ? 1 : PPT][kPiece];
    constexpr bool SHIFTED = !VEC && FORM != OUT_MX;      // a row's pieces start where its output lies
    if (!RES && !SHIFTED) {
#pragma unroll
        for (int s = 0; s < PPT; ++s) load_weight(a, (s * tpr + t) * kPiece, kept[RES ? 0 : s]);
    }
    load(r);
    // the loop's condition is the block's first row, so that no warp leaves another at the barrier or in a shuffle
    for (int turn = 0; r - (ROWS > 1 ? threadIdx.x / 32 : 0) < a.rows; ++turn, r += step) {
        float h[PPT][kPiece];
        float sum = 0.f;
        const bool live = r < a.rows;
        const int c0 = t * kPiece - (live ? row_shift<FORM, T, VEC>(a, r) : 0);
#pragma unroll
        for (int s = 0; s < PPT; ++s) {
            take<T, VEC>(x[s], c0 + s * tpr * kPiece, a.cols, h[s]);
            if (RES) {
                float w[kPiece];
                take<T, VEC>(res[RES ? s : 0], c0 + s * tpr * kPiece, a.cols, w);
#pragma unroll
                for (int i = 0; i < kPiece; ++i) h[s][i] += w[i];
            }
        }
        load(r + step);
#pragma unroll
        for (int s = 0; s < PPT; ++s) {
#pragma unroll
            for (int i = 0; i < kPiece; ++i) sum += h[s][i] * h[s][i];
        }
        sum = warp_sum(sum);
        if (TPR > 32) {
            if ((threadIdx.x & 31) == 0) reinterpret_cast<float *>(part[turn & 1])[threadIdx.x >> 5] = sum;
            __syncthreads();
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < THREADS / 128; ++i) {
                const float4 f = part[turn & 1][i];
                sum += (f.x + f.y) + (f.z + f.w);
            }
        }
        const float inv = rsqrtf(sum * a.inv_cols + a.eps);
        if (!live) continue;
#pragma unroll
        for (int s = 0; s < PPT; ++s) {
            const int c = c0 + s * tpr * kPiece;
            if constexpr (RES || SHIFTED) {
                float g[kPiece];
                load_weight(a, c, g);
                norm_out<FORM, T, VEC>(a, r, s * tpr + t, c, inv, h[s], g);
            } else {
                norm_out<FORM, T, VEC>(a, r, s * tpr + t, c, inv, h[s], kept[s]);
            }
        }
    }
}

// Rows too long for registers: one block per row, read a second time for the
// outputs.
template <typename T, int FORM, bool VEC>
__global__ void __launch_bounds__(512) rmsnorm_long_kernel(const NormArgs a)
{
    griddep_enter();
    __shared__ float part[16];
    const long long r = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + r * a.ldx;
    const T *res = a.residual ? static_cast<const T *>(a.residual) + r * a.ldr : nullptr;
    const int steps = (a.pieces + 511) / 512, shift = row_shift<FORM, T, VEC>(a, r);
    const Span x_span = span_of(a.x, a.rows, a.ldx, a.cols, sizeof(T));
    const Span res_span = res ? span_of(a.residual, a.rows, a.ldr, a.cols, sizeof(T)) : x_span;
    auto sum_at = [&](int c, float (&h)[kPiece]) {
        Held<T, VEC> p, q;
        hold<T, VEC>(x, c, a.cols, x_span, p);
        if (res) hold<T, VEC>(res, c, a.cols, res_span, q);
        take<T, VEC>(p, c, a.cols, h);
        if (res) {
            float w[kPiece];
            take<T, VEC>(q, c, a.cols, w);
#pragma unroll
            for (int i = 0; i < kPiece; ++i) h[i] += w[i];
        }
    };
    float sum = 0.f;
    for (int s = 0; s < steps; ++s) {
        float h[kPiece];
        sum_at((s * 512 + (int)threadIdx.x) * kPiece - shift, h);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) sum += h[i] * h[i];
    }
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += part[i];
    const float inv = rsqrtf(sum * a.inv_cols + a.eps);
    for (int s = 0; s < steps; ++s) {
        const int p = s * 512 + (int)threadIdx.x, c = p * kPiece - shift;
        float h[kPiece], g[kPiece];
        sum_at(c, h);
        load_weight(a, c, g);
        norm_out<FORM, T, VEC>(a, r, p, c, inv, h, g);
    }
}

template <typename T, int FORM, bool RES, int TPR, int PPT, bool VEC>
cudaError_t launch_norm_rows(const NormArgs &a, int sms, cudaStream_t s)
{
    // as many warps as hold the row's pieces, and one wave of such blocks
    const int threads = TPR == 32 ? norm_threads(TPR) : ((a.pieces + PPT - 1) / PPT + 31) / 32 * 32;
    const int rows = TPR == 32 ? threads / 32 : 1, beside = norm_room(sizeof(T), VEC) / threads;
    const long long most = (long long)sms * (beside < 1 ? 1 : beside), need = (a.rows + rows - 1) / rows;
    const dim3 grid((unsigned)(need < most ? need : most));
    if constexpr (VEC && TPR > 32) {
        if (threads == TPR)
            return launch_pdl(rmsnorm_kernel<T, FORM, RES, TPR, PPT, VEC, true>, grid, dim3(threads), 0, s, a);
    }
    return launch_pdl(rmsnorm_kernel<T, FORM, RES, TPR, PPT, VEC, false>, grid, dim3(threads), 0, s, a);
}

// The fewest threads whose pieces hold a row.
template <typename T, int FORM, bool RES, bool VEC>
cudaError_t launch_norm_res(const NormArgs &a, int sms, cudaStream_t s)
{
    if (a.pieces <= 32) return launch_norm_rows<T, FORM, RES, 32, 1, VEC>(a, sms, s);
    if (a.pieces <= 64) return launch_norm_rows<T, FORM, RES, 32, 2, VEC>(a, sms, s);
    if (a.pieces <= 128) return launch_norm_rows<T, FORM, RES, 128, 1, VEC>(a, sms, s);
    if (a.pieces <= 256) return launch_norm_rows<T, FORM, RES, 128, 2, VEC>(a, sms, s);
    if (a.pieces <= 512) return launch_norm_rows<T, FORM, RES, 256, 2, VEC>(a, sms, s);
    if (a.pieces <= 1024) return launch_norm_rows<T, FORM, RES, 512, 2, VEC>(a, sms, s);
    if (a.pieces <= 2048) return launch_norm_rows<T, FORM, RES, 1024, 2, VEC>(a, sms, s);
    return launch_pdl(rmsnorm_long_kernel<T, FORM, VEC>, dim3((unsigned)a.rows), dim3(512), 0, s, a);
}

template <typename T, int FORM, bool VEC>
cudaError_t launch_norm_form(const NormArgs &a, int sms, cudaStream_t s)
{
    ProfScope prof("rmsnorm", s);
    return a.residual ? launch_norm_res<T, FORM, true, VEC>(a, sms, s) : launch_norm_res<T, FORM, false, VEC>(a, sms, s);
}

}  // namespace

// The norm of one input type (norm_f32.cu, norm_f16.cu, norm_bf16.cu).
cudaError_t launch_norm_f32(const NormArgs &a, int form, bool vec, int sms, cudaStream_t s);
cudaError_t launch_norm_f16(const NormArgs &a, int form, bool vec, int sms, cudaStream_t s);
cudaError_t launch_norm_bf16(const NormArgs &a, int form, bool vec, int sms, cudaStream_t s);

namespace {

template <typename T>
cudaError_t launch_norm_type(const NormArgs &a, int form, bool vec, int sms, cudaStream_t s)
{
    if constexpr (sizeof(T) == 2) {   // a 32-bit type's own output is OUT_SAME
        if (form == OUT_F32) return vec ? launch_norm_form<T, OUT_F32, true>(a, sms, s) : launch_norm_form<T, OUT_F32, false>(a, sms, s);
    }
    if (form == OUT_MX) return vec ? launch_norm_form<T, OUT_MX, true>(a, sms, s) : launch_norm_form<T, OUT_MX, false>(a, sms, s);
    return vec ? launch_norm_form<T, OUT_SAME, true>(a, sms, s) : launch_norm_form<T, OUT_SAME, false>(a, sms, s);
}

}  // namespace

}  // namespace bigemm
