// norm_back.cuh -- gradients of the layer norm and of the root-mean-square norm,
// and the sums over all rows that make their weights' gradients.  A translation
// unit per type instantiates the row kernels (norm_back_*.cu).
//
// Layer norm, of xh = (x - m) rstd and g = dout * weight:
//   dx = rstd (g - mean_k g - xh mean_k (g xh)) (+ dsum)
//   dweight = sum_rows dout xh,   dbias = sum_rows dout
// RMS norm, of rstd = rsqrt(mean_k x^2 + eps), found again from the row, and xh = x rstd:
//   dx = rstd (g - xh mean_k (g xh)) (+ dsum),   dweight = sum_rows dout xh
//
// All in fp32, each output rounded once.  Bound by memory: one pass reads dout, x and
// dsum and writes dx.  A block walks over its rows with the next one's loads in
// flight; a thread keeps the same columns all the way, so it adds up its part of the
// weights' gradients in registers.  Each block leaves one row of partial sums (a
// block of the machine's one wave: 152 rows of 8192 columns against 8192 rows), which
// a second launch adds in their order: the result does not depend on timing.
#pragma once
#include "norm.cuh"

namespace bigemm {

struct NormBackArgs {
    int cols;
    long long rows, ldd, ldx, lds, ldo;
    const void *dout, *x, *dsum;      // dsum: or null
    const float *weight, *mean, *rstd;
    bool vec_weight;                  // there, on a 16-byte boundary
    float eps, inv_cols;
    void *dx;
    float *dweight, *dbias;           // a row of `parts` per block, `cols` apart
};

constexpr int kBackSms = 152;         // of the machine: one wave of blocks
constexpr int kBackMaxCols = 8192;    // of the one-pass kernels

// Blocks of the one-pass kernel for these rows and how many threads they have;
// at most 1024 threads per SM.
struct BackGrid {
    int threads, rows;                // rows: that a block takes at once
    int blocks;
};

inline BackGrid back_grid(long long rows, int cols, size_t es, bool vec)
{
    const int pieces = (cols + kPiece - 1) / kPiece;
    BackGrid g;
    g.threads = pieces <= 32 ? 128 : (pieces + 31) / 32 * 32;
    g.rows = pieces <= 32 ? 4 : 1;
    const int room = es == 4 || !vec ? 512 : 1024, beside = room / g.threads < 1 ? 1 : room / g.threads;
    const long long need = (rows + g.rows - 1) / g.rows, most = (long long)kBackSms * beside;
    g.blocks = (int)(need < most ? need : most);
    return g;
}

namespace {

// Where a thread's 8 elements of a row lie: consecutive ones on the 16-byte grid;
// off it, one of each eighth of the block's columns, so that a warp's plain loads and
// stores cover consecutive elements and a thread's columns are the same in every row.
template <bool VEC>
struct Columns {
    int c0, by;
    __device__ __forceinline__ Columns(int t, int tpr) : c0(VEC ? t * kPiece : t), by(VEC ? 1 : tpr) {}
    __device__ __forceinline__ int at(int i) const { return c0 + i * by; }
};

// Elements as loaded.
template <typename T, bool VEC>
struct Kept {
    std::conditional_t<VEC, Raw<T>, T[kPiece]> d;
};

template <typename T, bool VEC>
__device__ __forceinline__ void keep(const T *row, const Columns<VEC> &c, int cols, Kept<T, VEC> &k)
{
    if constexpr (VEC) {
        if (c.c0 + kPiece <= cols) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) k.d.q[i] = reinterpret_cast<const uint4 *>(row + c.c0)[i];
            return;
        }
        T *e = reinterpret_cast<T *>(&k.d);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) e[i] = c.c0 + i < cols ? row[c.c0 + i] : from_f32<T>(0.f);
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) k.d[i] = c.at(i) < cols ? row[c.at(i)] : from_f32<T>(0.f);
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void values(const Kept<T, VEC> &k, float (&v)[kPiece])
{
    if constexpr (VEC) {
        unpack<T>(k.d, v);
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) v[i] = to_f32<T>(k.d[i]);
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void put(T *row, const Columns<VEC> &c, int cols, const float (&v)[kPiece])
{
    if constexpr (VEC) {
        store_piece<T, true>(row, c.c0, cols, v);
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (c.at(i) < cols) row[c.at(i)] = from_f32<T>(v[i]);
    }
}

template <bool VEC>
__device__ __forceinline__ void weights(const NormBackArgs &a, const Columns<VEC> &c, float (&g)[kPiece])
{
    if (VEC && a.vec_weight && c.c0 + kPiece <= a.cols) {
        const float4 u = *reinterpret_cast<const float4 *>(a.weight + c.c0);
        const float4 w = *reinterpret_cast<const float4 *>(a.weight + c.c0 + 4);
        g[0] = u.x, g[1] = u.y, g[2] = u.z, g[3] = u.w, g[4] = w.x, g[5] = w.y, g[6] = w.z, g[7] = w.w;
        return;
    }
#pragma unroll
    for (int i = 0; i < kPiece; ++i) g[i] = a.weight && c.at(i) < a.cols ? a.weight[c.at(i)] : 1.f;
}

// TPR: most threads of a row (a warp of four, or the block).
template <typename T, bool LAYER, bool SUM, int TPR, bool VEC>
__global__ void __launch_bounds__(norm_threads(TPR), norm_blocks(TPR, sizeof(T), VEC)) norm_back_kernel(const NormBackArgs a)
{
    griddep_enter();
    constexpr int THREADS = norm_threads(TPR), ROWS = THREADS / TPR;
    __shared__ float2 part[2][THREADS / 32];
    __shared__ float total[ROWS > 1 ? 2 * ROWS * TPR * kPiece : 1];
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31;
    const int tpr = TPR == 32 ? 32 : (int)blockDim.x, t = TPR == 32 ? lane : (int)threadIdx.x;
    const Columns<VEC> c(t, tpr);
    const long long step = (long long)gridDim.x * ROWS;
    long long r = (long long)blockIdx.x * ROWS + (TPR == 32 ? warp : 0);
    Kept<T, VEC> dk, xk, sk;
    auto load = [&](long long row) {
        if (row >= a.rows) return;
        keep<T, VEC>(static_cast<const T *>(a.dout) + row * a.ldd, c, a.cols, dk);
        keep<T, VEC>(static_cast<const T *>(a.x) + row * a.ldx, c, a.cols, xk);
        if (SUM) keep<T, VEC>(static_cast<const T *>(a.dsum) + row * a.lds, c, a.cols, sk);
    };
    float dw[kPiece], db[LAYER ? kPiece : 1];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) dw[i] = 0.f, db[LAYER ? i : 0] = 0.f;
    load(r);
    // the loop's condition is the block's first row, so that no warp leaves another at the barrier or in a shuffle
    for (int turn = 0; r - (ROWS > 1 ? warp : 0) < a.rows; ++turn, r += step) {
        const bool live = r < a.rows;
        float d[kPiece], x[kPiece], s[kPiece];
        values<T, VEC>(dk, d);
        values<T, VEC>(xk, x);
        if (SUM) values<T, VEC>(sk, s);
        load(r + step);
        float rstd = 0.f;
        if (LAYER) {
            const float m = live ? a.mean[r] : 0.f;
            rstd = live ? a.rstd[r] : 0.f;
#pragma unroll
            for (int i = 0; i < kPiece; ++i) x[i] = (x[i] - m) * rstd;      // (outside the row d is 0)
        }
        float g[kPiece];
        weights<VEC>(a, c, g);
        // sums over the row: of g xh and g; of g x and x x
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
            g[i] *= d[i];
            sum.x = fmaf(g[i], x[i], sum.x);
            sum.y = LAYER ? sum.y + g[i] : fmaf(x[i], x[i], sum.y);
        }
        sum.x = warp_sum(sum.x), sum.y = warp_sum(sum.y);
        if (TPR > 32) {
            if (lane == 0) part[turn & 1][warp] = sum;
            __syncthreads();
            const float2 p = lane < tpr >> 5 ? part[turn & 1][lane] : make_float2(0.f, 0.f);
            sum.x = warp_sum(p.x), sum.y = warp_sum(p.y);
        }
        if (!live) continue;
        float o[kPiece];
        if (LAYER) {
            const float by = sum.x * a.inv_cols, level = sum.y * a.inv_cols;
#pragma unroll
            for (int i = 0; i < kPiece; ++i) {
                o[i] = rstd * (g[i] - level - x[i] * by);
                dw[i] = fmaf(d[i], x[i], dw[i]);
                db[LAYER ? i : 0] += d[i];
            }
        } else {
            rstd = rsqrtf(sum.y * a.inv_cols + a.eps);
            const float by = rstd * rstd * (sum.x * a.inv_cols);
#pragma unroll
            for (int i = 0; i < kPiece; ++i) {
                o[i] = rstd * (g[i] - x[i] * by);
                dw[i] = fmaf(d[i] * rstd, x[i], dw[i]);
            }
        }
        if (SUM) {
#pragma unroll
            for (int i = 0; i < kPiece; ++i) o[i] += s[i];
        }
        put<T, VEC>(static_cast<T *>(a.dx) + r * a.ldo, c, a.cols, o);
    }
    float *to_w = a.dweight + (long long)blockIdx.x * a.cols, *to_b = LAYER ? a.dbias + (long long)blockIdx.x * a.cols : nullptr;
    if (ROWS > 1) {
        // four warps, the same columns
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
            total[(warp * 2) * 32 * kPiece + i * 32 + lane] = dw[i];
            total[(warp * 2 + 1) * 32 * kPiece + i * 32 + lane] = db[LAYER ? i : 0];
        }
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
#pragma unroll
            for (int w = 1; w < ROWS; ++w) {
                dw[i] += total[(w * 2) * 32 * kPiece + i * 32 + lane];
                if (LAYER) db[LAYER ? i : 0] += total[(w * 2 + 1) * 32 * kPiece + i * 32 + lane];
            }
    }
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
        if (c.at(i) < a.cols) {
            to_w[c.at(i)] = dw[i];
            if (LAYER) to_b[c.at(i)] = db[LAYER ? i : 0];
        }
}

// Rows of more than 8192 columns take two kernels.  The first adds up the weights'
// gradients (before the second may write dx over dout): 256 threads, a column each, a
// run of rows per block.
template <typename T, bool LAYER>
__global__ void __launch_bounds__(256) norm_back_columns_kernel(const NormBackArgs a, const float *rstds, int parts)
{
    griddep_enter();
    const long long c = (long long)blockIdx.x * 256 + threadIdx.x;
    if (c >= a.cols) return;
    const long long r0 = a.rows * blockIdx.y / parts, r1 = a.rows * (blockIdx.y + 1) / parts;
    const T *d = static_cast<const T *>(a.dout) + c, *x = static_cast<const T *>(a.x) + c;
    float dw = 0.f, db = 0.f;
#pragma unroll 4
    for (long long r = r0; r < r1; ++r) {
        const float dv = to_f32<T>(d[r * a.ldd]), xv = to_f32<T>(x[r * a.ldx]);
        dw = fmaf(dv, LAYER ? (xv - a.mean[r]) * rstds[r] : xv * rstds[r], dw);
        if (LAYER) db += dv;
    }
    a.dweight[blockIdx.y * (long long)a.cols + c] = dw;
    if (LAYER) a.dbias[blockIdx.y * (long long)a.cols + c] = db;
}

// Two sums over the block's threads; every thread gets them.
__device__ __forceinline__ float2 block_sum2(float2 v, float2 *part)
{
    v.x = warp_sum(v.x), v.y = warp_sum(v.y);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 16; ++i) v.x += part[i].x, v.y += part[i].y;
    return v;
}

// The roots of the RMS norm's rows, for the kernel above.
template <typename T, bool VEC>
__global__ void __launch_bounds__(512) norm_back_root_kernel(const NormBackArgs a, float *rstds)
{
    griddep_enter();
    __shared__ float2 part[16];
    const T *x = static_cast<const T *>(a.x) + (long long)blockIdx.x * a.ldx;
    float2 sum = make_float2(0.f, 0.f);
    for (long long c = (long long)threadIdx.x * (VEC ? kPiece : 1); c < a.cols; c += 512 * (VEC ? kPiece : 1)) {
        if (VEC && c + kPiece <= a.cols) {
            float v[kPiece];
            unpack<T>(*reinterpret_cast<const Raw<T> *>(x + c), v);
#pragma unroll
            for (int i = 0; i < kPiece; ++i) sum.x = fmaf(v[i], v[i], sum.x);
        } else {
            for (int i = 0; i < (VEC ? kPiece : 1) && c + i < a.cols; ++i) {
                const float v = to_f32<T>(x[c + i]);
                sum.x = fmaf(v, v, sum.x);
            }
        }
    }
    sum = block_sum2(sum, part);
    if (threadIdx.x == 0) rstds[blockIdx.x] = rsqrtf(sum.x * a.inv_cols + a.eps);
}

// A block per row: its sums, then dx, the row read again.
template <typename T, bool LAYER, bool VEC>
__global__ void __launch_bounds__(512) norm_back_long_kernel(const NormBackArgs a, const float *rstds)
{
    griddep_enter();
    __shared__ float2 part[16];
    const long long r = blockIdx.x;
    const T *dr = static_cast<const T *>(a.dout) + r * a.ldd, *xr = static_cast<const T *>(a.x) + r * a.ldx;
    const T *sr = a.dsum ? static_cast<const T *>(a.dsum) + r * a.lds : nullptr;
    T *to = static_cast<T *>(a.dx) + r * a.ldo;
    const float m = LAYER ? a.mean[r] : 0.f, rstd = rstds[r];
    const int steps = (a.cols + 512 * kPiece - 1) / (512 * kPiece);
    auto row_at = [&](int s, Columns<VEC> &c, float (&g)[kPiece], float (&xh)[kPiece]) {
        c.c0 = s * 512 * kPiece + (VEC ? (int)threadIdx.x * kPiece : (int)threadIdx.x);
        Kept<T, VEC> k, q;
        keep<T, VEC>(dr, c, a.cols, k);
        keep<T, VEC>(xr, c, a.cols, q);
        float d[kPiece], x[kPiece];
        values<T, VEC>(k, d);
        values<T, VEC>(q, x);
        weights<VEC>(a, c, g);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) g[i] *= d[i], xh[i] = (x[i] - m) * rstd;
    };
    Columns<VEC> c(0, 512);
    float g[kPiece], xh[kPiece];
    float2 sum = make_float2(0.f, 0.f);
    for (int s = 0; s < steps; ++s) {
        row_at(s, c, g, xh);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) sum.x = fmaf(g[i], xh[i], sum.x), sum.y += g[i];
    }
    sum = block_sum2(sum, part);
    const float by = sum.x * a.inv_cols, level = LAYER ? sum.y * a.inv_cols : 0.f;
    for (int s = 0; s < steps; ++s) {
        row_at(s, c, g, xh);
        float o[kPiece];
#pragma unroll
        for (int i = 0; i < kPiece; ++i) o[i] = rstd * (g[i] - level - xh[i] * by);
        if (sr) {
            Kept<T, VEC> k;
            float v[kPiece];
            keep<T, VEC>(sr, c, a.cols, k);
            values<T, VEC>(k, v);
#pragma unroll
            for (int i = 0; i < kPiece; ++i) o[i] += v[i];
        }
        put<T, VEC>(to, c, a.cols, o);
    }
}

template <typename T, bool LAYER, bool SUM, bool VEC>
cudaError_t launch_back_rows(const NormBackArgs &a, cudaStream_t s)
{
    const BackGrid g = back_grid(a.rows, a.cols, sizeof(T), VEC);
    const dim3 grid((unsigned)g.blocks), block((unsigned)g.threads);
    if (g.rows > 1) return launch_pdl(norm_back_kernel<T, LAYER, SUM, 32, VEC>, grid, block, 0, s, a);
    if (g.threads <= 256) return launch_pdl(norm_back_kernel<T, LAYER, SUM, 256, VEC>, grid, block, 0, s, a);
    if (g.threads <= 512) return launch_pdl(norm_back_kernel<T, LAYER, SUM, 512, VEC>, grid, block, 0, s, a);
    return launch_pdl(norm_back_kernel<T, LAYER, SUM, 1024, VEC>, grid, block, 0, s, a);
}

template <typename T, bool LAYER, bool VEC>
cudaError_t launch_back_vec(const NormBackArgs &a, float *rstds, int parts, cudaStream_t s)
{
    ProfScope prof(LAYER ? "layernorm_backward" : "rmsnorm_backward", s);
    if (a.cols <= kBackMaxCols)
        return a.dsum ? launch_back_rows<T, LAYER, true, VEC>(a, s) : launch_back_rows<T, LAYER, false, VEC>(a, s);
    const dim3 rows((unsigned)a.rows);
    const float *roots = LAYER ? a.rstd : rstds;
    if (!LAYER) {
        const cudaError_t e = launch_pdl(norm_back_root_kernel<T, VEC>, rows, dim3(512), 0, s, a, rstds);
        if (e != cudaSuccess) return e;
    }
    const dim3 cols((unsigned)((a.cols + 255ll) / 256), (unsigned)parts);
    const cudaError_t e = launch_pdl(norm_back_columns_kernel<T, LAYER>, cols, dim3(256), 0, s, a, roots, parts);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_back_long_kernel<T, LAYER, VEC>, rows, dim3(512), 0, s, a, roots);
}

}  // namespace

// The gradients of one type (norm_back_*.cu): dx, and partial sums in a.dweight and
// a.dbias; rstds: [rows] for the roots of long RMS rows; parts: of long rows.
cudaError_t launch_norm_back_f32(const NormBackArgs &a, bool layer, bool vec, float *rstds, int parts, cudaStream_t s);
cudaError_t launch_norm_back_f16(const NormBackArgs &a, bool layer, bool vec, float *rstds, int parts, cudaStream_t s);
cudaError_t launch_norm_back_bf16(const NormBackArgs &a, bool layer, bool vec, float *rstds, int parts, cudaStream_t s);

namespace {

template <typename T>
cudaError_t launch_norm_back_type(const NormBackArgs &a, bool layer, bool vec, float *rstds, int parts, cudaStream_t s)
{
    if (layer)
        return vec ? launch_back_vec<T, true, true>(a, rstds, parts, s) : launch_back_vec<T, true, false>(a, rstds, parts, s);
    return vec ? launch_back_vec<T, false, true>(a, rstds, parts, s) : launch_back_vec<T, false, false>(a, rstds, parts, s);
}

}  // namespace

}  // namespace bigemm
