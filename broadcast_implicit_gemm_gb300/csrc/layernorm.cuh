// layernorm.cuh -- the layer norm with the residual's addition, and its entry's
// arguments.  A translation unit per input type instantiates it (layernorm_*.cu).
//
//   h = x (+ residual);  m = mean_k h;  v = mean_k (h - m)^2
//   y = (h - m) rsqrt(v + eps) (* weight) (+ bias)
//
// in fp32 from the inputs to the one rounding of each output.  Bound by memory: a
// row stays in registers, so each byte moves once, and a block loads its next row
// before it sums the present one (norm.cuh, whose pieces and loads these are).
// 8192 x 8192 f16 with residual 85 us (6.3 TB/s), f32 177 (6.1), bf16 to f32 108 (6.2).
// Not bound by it:
//   to MXFP8 (16384 x 4096 bf16 75 us, 2.7 TB/s): issue slots 69 %, and the weights and
//     biases, 8 bytes for each element's 3, take 64 % of L1's cycles;
//   f32 without a residual (8192 x 8192 114 us, 4.7 TB/s): a block of 16 warps an SM;
//   rows off the 16-byte grid (2000 x 7001 bf16 with residual 45 us, on it 24): 112
//     registers a thread for two words per piece, one block an SM, a row in flight.
// Spilled, to L1: at 64 registers up to 132 bytes a thread of rows of 257 to 512 columns;
// off the grid and of 32 bits up to 372 from 8193 columns on (2000 x 12001 106 us).
//
// The variance is that of differences from the mean, not of a difference of sums,
// which would lose the digits that a row far from zero has in common.  One barrier
// per row all the same: each warp finds the mean of its own part and the squares
// around it, and the parts join by
//   sum (h - m)^2 = sum_w [ sum (h - m_w)^2 + n_w (m_w - m)^2 ].
#pragma once
#include "norm.cuh"

namespace bigemm {

struct LayerNormArgs : NormArgs {
    const float *bias;
    bool vec_bias;                    // there, on a 16-byte boundary
    float *mean, *rstd;               // [rows] or null
};

namespace {

// A piece of a vector (vec: on a 16-byte boundary), `other` outside it or without one.
// Pieces of rows off the grid start anywhere in a word: three words and a choice that the
// row's lanes share (eight single loads: 2000 x 7001 bf16 with residual 55 us, 45 so).
template <bool VEC>
__device__ __forceinline__ void load_vector(const float *v, bool vec, int c, int cols, float other, float (&g)[kPiece])
{
    if (VEC && vec && c + kPiece <= cols) {
        const float4 u = *reinterpret_cast<const float4 *>(v + c);
        const float4 w = *reinterpret_cast<const float4 *>(v + c + 4);
        g[0] = u.x, g[1] = u.y, g[2] = u.z, g[3] = u.w, g[4] = w.x, g[5] = w.y, g[6] = w.z, g[7] = w.w;
        return;
    }
    const int first = c & ~3;
    if (!VEC && vec && c >= 0 && first + 12 <= cols) {
        float f[12];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            if (i == 2 && c == first) break;
            const float4 u = *reinterpret_cast<const float4 *>(v + first + 4 * i);
            f[4 * i] = u.x, f[4 * i + 1] = u.y, f[4 * i + 2] = u.z, f[4 * i + 3] = u.w;
        }
        switch (c - first) {
        case 0:
#pragma unroll
            for (int i = 0; i < kPiece; ++i) g[i] = f[i];
            break;
        case 1:
#pragma unroll
            for (int i = 0; i < kPiece; ++i) g[i] = f[i + 1];
            break;
        case 2:
#pragma unroll
            for (int i = 0; i < kPiece; ++i) g[i] = f[i + 2];
            break;
        default:
#pragma unroll
            for (int i = 0; i < kPiece; ++i) g[i] = f[i + 3];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kPiece; ++i) g[i] = v && c + i >= 0 && c + i < cols ? v[c + i] : other;
}

// The outputs of one piece, from column c on.
template <int FORM, typename T, bool VEC>
__device__ __forceinline__ void layernorm_out(const LayerNormArgs &a, long long r, int p, int c, float mean, float inv,
                                              const float (&h)[kPiece])
{
    if (a.h) store_piece<T, VEC>(static_cast<T *>(a.h) + r * a.ldh, c, a.cols, h);
    float y[kPiece], g[kPiece], b[kPiece];
    load_vector<VEC>(a.weight, a.vec_weight, c, a.cols, 1.f, g);
    load_vector<VEC>(a.bias, a.vec_bias, c, a.cols, 0.f, b);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) y[i] = fmaf((h[i] - mean) * inv, g[i], b[i]);
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

// Sum over a piece's elements inside the row of (h - m)^2.
__device__ __forceinline__ float piece_squares(const float (&h)[kPiece], float m, int c, int cols)
{
    float q = 0.f;
    if (c >= 0 && c + kPiece <= cols) {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) q = fmaf(h[i] - m, h[i] - m, q);
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (c + i >= 0 && c + i < cols) q = fmaf(h[i] - m, h[i] - m, q);
    }
    return q;
}

// How many of the n columns from c on are inside the row.
__device__ __forceinline__ int inside(int c, int n, int cols) { return max(0, min(c + n, cols) - max(c, 0)); }

// A warp's part of a row: its sum, its squares around its own mean, its length.
struct Moments {
    float sum, squares, n;
};

// The same of several parts, one per lane (n = 0: none).
__device__ __forceinline__ void join(const Moments &w, float inv_cols, float &mean, float &squares)
{
    mean = warp_sum(w.sum) * inv_cols;
    const float d = w.n > 0.f ? w.sum / w.n - mean : 0.f;
    squares = warp_sum(w.squares + w.n * d * d);
}

// TPR threads per row at most (a warp, or the block, which has the warps that the
// row needs), PPT pieces per thread.
template <typename T, int FORM, bool RES, int TPR, int PPT, bool VEC>
__global__ void __launch_bounds__(norm_threads(TPR), norm_blocks(TPR, sizeof(T), VEC)) layernorm_kernel(const LayerNormArgs a)
{
    griddep_enter();
    constexpr int THREADS = norm_threads(TPR), ROWS = THREADS / TPR;
    static_assert(TPR == 32 || ROWS == 1, "a row has a warp or the block");
    __shared__ Moments part[2][THREADS / 32];
    const int tpr = TPR == 32 ? TPR : (int)blockDim.x, t = TPR == 32 ? (int)threadIdx.x & 31 : (int)threadIdx.x;
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
    const long long step = (long long)gridDim.x * ROWS;
    long long r = (long long)blockIdx.x * ROWS + (TPR == 32 ? warp : 0);
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
    load(r);
    // the loop's condition is the block's first row, so that no warp leaves another at the barrier or in a shuffle
    for (int turn = 0; r - (ROWS > 1 ? warp : 0) < a.rows; ++turn, r += step) {
        float h[PPT][kPiece];
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
        Moments mine = {0.f, 0.f, 0.f};
        int n = 0;
#pragma unroll
        for (int s = 0; s < PPT; ++s) {
#pragma unroll
            for (int i = 0; i < kPiece; ++i) mine.sum += h[s][i];           // zeros outside the row
            n += inside(c0 - lane * kPiece + s * tpr * kPiece, 32 * kPiece, a.cols);
        }
        mine.sum = warp_sum(mine.sum);
        mine.n = (float)n;
        const float m = n > 0 ? mine.sum / mine.n : 0.f;
#pragma unroll
        for (int s = 0; s < PPT; ++s) mine.squares += piece_squares(h[s], m, c0 + s * tpr * kPiece, a.cols);
        mine.squares = warp_sum(mine.squares);
        float mean = m, squares = mine.squares;
        if (TPR > 32) {
            if (lane == 0) part[turn & 1][warp] = mine;
            __syncthreads();
            Moments w = {0.f, 0.f, 0.f};
            if (lane < tpr >> 5) w = part[turn & 1][lane];
            join(w, a.inv_cols, mean, squares);
        }
        const float inv = rsqrtf(squares * a.inv_cols + a.eps);
        if (!live) continue;
        if (t == 0) {
            if (a.mean) a.mean[r] = mean;
            if (a.rstd) a.rstd[r] = inv;
        }
#pragma unroll
        for (int s = 0; s < PPT; ++s)
            layernorm_out<FORM, T, VEC>(a, r, s * tpr + t, c0 + s * tpr * kPiece, mean, inv, h[s]);
    }
}

// Rows too long for registers: one block per row, read again for the squares and
// for the outputs.
template <typename T, int FORM, bool VEC>
__global__ void __launch_bounds__(512) layernorm_long_kernel(const LayerNormArgs a)
{
    griddep_enter();
    __shared__ float part[2][16];
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
    auto block_sum = [&](int which, float v) {
        v = warp_sum(v);
        if ((threadIdx.x & 31) == 0) part[which][threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) v += part[which][i];
        return v;
    };
    float sum = 0.f, squares = 0.f;
    for (int s = 0; s < steps; ++s) {
        float h[kPiece];
        sum_at((s * 512 + (int)threadIdx.x) * kPiece - shift, h);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) sum += h[i];
    }
    const float mean = block_sum(0, sum) * a.inv_cols;
    for (int s = 0; s < steps; ++s) {
        const int c = (s * 512 + (int)threadIdx.x) * kPiece - shift;
        float h[kPiece];
        sum_at(c, h);
        squares += piece_squares(h, mean, c, a.cols);
    }
    const float inv = rsqrtf(block_sum(1, squares) * a.inv_cols + a.eps);
    if (threadIdx.x == 0) {
        if (a.mean) a.mean[r] = mean;
        if (a.rstd) a.rstd[r] = inv;
    }
    for (int s = 0; s < steps; ++s) {
        const int p = s * 512 + (int)threadIdx.x, c = p * kPiece - shift;
        float h[kPiece];
        sum_at(c, h);
        layernorm_out<FORM, T, VEC>(a, r, p, c, mean, inv, h);
    }
}

template <typename T, int FORM, bool RES, int TPR, int PPT, bool VEC>
cudaError_t launch_layernorm_rows(const LayerNormArgs &a, int sms, cudaStream_t s)
{
    // as many warps as hold the row's pieces, and one wave of such blocks
    const int threads = TPR == 32 ? norm_threads(TPR) : ((a.pieces + PPT - 1) / PPT + 31) / 32 * 32;
    const int rows = TPR == 32 ? threads / 32 : 1, beside = norm_room(sizeof(T), VEC) / threads;
    const long long most = (long long)sms * (beside < 1 ? 1 : beside), need = (a.rows + rows - 1) / rows;
    const dim3 grid((unsigned)(need < most ? need : most));
    return launch_pdl(layernorm_kernel<T, FORM, RES, TPR, PPT, VEC>, grid, dim3(threads), 0, s, a);
}

// The fewest threads whose pieces hold a row.
template <typename T, int FORM, bool RES, bool VEC>
cudaError_t launch_layernorm_res(const LayerNormArgs &a, int sms, cudaStream_t s)
{
    if (a.pieces <= 32) return launch_layernorm_rows<T, FORM, RES, 32, 1, VEC>(a, sms, s);
    if (a.pieces <= 64) return launch_layernorm_rows<T, FORM, RES, 32, 2, VEC>(a, sms, s);
    if (a.pieces <= 512) return launch_layernorm_rows<T, FORM, RES, 256, 2, VEC>(a, sms, s);
    if (a.pieces <= 1024) return launch_layernorm_rows<T, FORM, RES, 512, 2, VEC>(a, sms, s);
    if (a.pieces <= 2048) return launch_layernorm_rows<T, FORM, RES, 1024, 2, VEC>(a, sms, s);
    return launch_pdl(layernorm_long_kernel<T, FORM, VEC>, dim3((unsigned)a.rows), dim3(512), 0, s, a);
}

template <typename T, int FORM, bool VEC>
cudaError_t launch_layernorm_form(const LayerNormArgs &a, int sms, cudaStream_t s)
{
    ProfScope prof("layernorm", s);
    return a.residual ? launch_layernorm_res<T, FORM, true, VEC>(a, sms, s)
                      : launch_layernorm_res<T, FORM, false, VEC>(a, sms, s);
}

}  // namespace

// The norm of one input type (layernorm_f32.cu, layernorm_f16.cu, layernorm_bf16.cu).
cudaError_t launch_layernorm_f32(const LayerNormArgs &a, int form, bool vec, int sms, cudaStream_t s);
cudaError_t launch_layernorm_f16(const LayerNormArgs &a, int form, bool vec, int sms, cudaStream_t s);
cudaError_t launch_layernorm_bf16(const LayerNormArgs &a, int form, bool vec, int sms, cudaStream_t s);

namespace {

template <typename T>
cudaError_t launch_layernorm_type(const LayerNormArgs &a, int form, bool vec, int sms, cudaStream_t s)
{
    if constexpr (sizeof(T) == 2) {   // a 32-bit type's own output is OUT_SAME
        if (form == OUT_F32)
            return vec ? launch_layernorm_form<T, OUT_F32, true>(a, sms, s) : launch_layernorm_form<T, OUT_F32, false>(a, sms, s);
    }
    if (form == OUT_MX)
        return vec ? launch_layernorm_form<T, OUT_MX, true>(a, sms, s) : launch_layernorm_form<T, OUT_MX, false>(a, sms, s);
    return vec ? launch_layernorm_form<T, OUT_SAME, true>(a, sms, s) : launch_layernorm_form<T, OUT_SAME, false>(a, sms, s);
}

}  // namespace

}  // namespace bigemm
