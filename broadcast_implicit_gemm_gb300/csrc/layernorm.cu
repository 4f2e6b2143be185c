// layernorm.cu -- entry points of the layer norm and of the norms' gradients:
// checks of arguments, and the partial sums' place in the workspace.
#include "column_sums.cuh"
#include "layernorm.cuh"
#include "norm_back.cuh"

using namespace bigemm;

namespace {

bool aligned(const void *p, long long ld, size_t size, size_t to)
{
    return !p || (reinterpret_cast<uintptr_t>(p) % to == 0 && (ld * (long long)size) % (long long)to == 0);
}

// Rows of partial sums that the gradients of these rows leave at most: one per block of the
// one-pass kernels (or cluster), or of the runs of long rows, eight blocks of 256 columns per SM.
int back_parts(long long rows, int cols)
{
    if (cols <= kBackMaxCols) return back_grid(rows, cols).parts;
    const long long wide = (cols + 255ll) / 256, want = (8ll * kBackSms + wide - 1) / wide;
    return (int)(rows < want ? rows : want);
}

// Of those, what the device runs at once: a cluster's walk over its rows is as long as any, so
// that one that begins late ends as late.
int resident_parts(long long rows, int cols)
{
    const int most = back_parts(rows, cols), cluster = cols <= kBackMaxCols ? back_grid(rows, cols).cluster : 1;
    const int fit = cluster > 1 ? back_clusters(cluster) : 0;
    return fit > 0 && fit < most ? fit : most;
}

uint64_t back_workspace(long long rows, int cols)
{
    const uint64_t parts = (uint64_t)back_parts(rows, cols);
    return (parts * 2 * (uint64_t)sum_pitch(cols) + (cols > kBackMaxCols ? (uint64_t)rows : 0)) * 4;
}

bigemm_status norm_backward(NormBackArgs &a, bool layer, int dtype, void *workspace, uint64_t bytes, void *stream)
{
    if (a.rows < 0 || a.cols < 1 || dtype < BIGEMM_F32 || dtype > BIGEMM_BF16) return BIGEMM_ERR_INVALID_ARG;
    if (a.cols > kMaxCols) return BIGEMM_ERR_UNSUPPORTED;
    if (!a.dweight || (layer && !a.dbias) || !aligned(a.dweight, 0, 1, 4) || !aligned(a.dbias, 0, 1, 4))
        return BIGEMM_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    ColumnSums sums = {};
    sums.count = layer ? 2 : 1, sums.cols = a.cols;
    sums.out[0] = a.dweight, sums.out[1] = a.dbias;
    if (a.rows == 0) {
        if (!device_state()) return BIGEMM_ERR_CUDA;
        return launch_column_sums(sums, s) == cudaSuccess ? BIGEMM_OK : BIGEMM_ERR_CUDA;
    }
    const size_t es = dtype_size(dtype);
    if (!a.dout || !a.x || !a.dx || (layer && (!a.mean || !a.rstd))) return BIGEMM_ERR_INVALID_ARG;
    if (a.ldd < a.cols || a.ldx < a.cols || a.ldo < a.cols || (a.dsum && a.lds < a.cols)) return BIGEMM_ERR_INVALID_ARG;
    if (!aligned(a.dout, 0, 1, es) || !aligned(a.x, 0, 1, es) || !aligned(a.dx, 0, 1, es) || !aligned(a.dsum, 0, 1, es) ||
        !aligned(a.weight, 0, 1, 4) || !aligned(a.mean, 0, 1, 4) || !aligned(a.rstd, 0, 1, 4))
        return BIGEMM_ERR_INVALID_ARG;
    // dx takes the place of what a thread has read; the sums are written while other rows are still read
    if (!distinct({a.dout, a.x, a.dsum, a.weight, a.mean, a.rstd, a.dx, a.dweight, a.dbias}, 7) ||
        !distinct({a.weight, a.mean, a.rstd, a.dx}, 3) || !apart_or_in_place(a.dx, a.ldo, a.dout, a.ldd, a.rows) ||
        !apart_or_in_place(a.dx, a.ldo, a.x, a.ldx, a.rows) || !apart_or_in_place(a.dx, a.ldo, a.dsum, a.lds, a.rows))
        return BIGEMM_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 0, 1, 16) || bytes < back_workspace(a.rows, a.cols)) return BIGEMM_ERR_INVALID_ARG;
    DeviceState *ds = device_state();
    if (!ds) return BIGEMM_ERR_CUDA;
    a.timeout_ns = wait_timeout_ns();
    a.err = ds->err;
    const bool vec = aligned(a.dout, a.ldd, es, 16) && aligned(a.x, a.ldx, es, 16) && aligned(a.dx, a.ldo, es, 16) &&
                     aligned(a.dsum, a.lds, es, 16);
    a.inv_cols = 1.0f / (float)a.cols;
    const int parts = resident_parts(a.rows, a.cols);
    float *space = static_cast<float *>(workspace);
    if (parts > 1) {             // (one row of sums is the result)
        a.dweight = space, a.dbias = space + parts * sum_pitch(a.cols);
        sums.from[0] = a.dweight, sums.from[1] = a.dbias, sums.parts = parts;
    }
    float *rstds = space + 2 * parts * sum_pitch(a.cols);
    const cudaError_t e = dtype == BIGEMM_F32   ? launch_norm_back_f32(a, layer, vec, rstds, parts, s)
                          : dtype == BIGEMM_F16 ? launch_norm_back_f16(a, layer, vec, rstds, parts, s)
                                                : launch_norm_back_bf16(a, layer, vec, rstds, parts, s);
    if (e != cudaSuccess) return BIGEMM_ERR_CUDA;
    return parts == 1 || launch_column_sums(sums, s) == cudaSuccess ? BIGEMM_OK : BIGEMM_ERR_CUDA;
}

}  // namespace

extern "C" {

bigemm_status layernorm_run(int rows, int cols, bigemm_dtype in_dtype, const void *x, int64_t ldx, const void *residual,
                            int64_t ldr, const float *weight, const float *bias, float eps, void *sum_out, int64_t lds,
                            bigemm_dtype out_dtype, void *out, int64_t ldo, void *out_scale, float *mean, float *rstd,
                            void *stream)
{
    if (rows < 0 || cols < 1) return BIGEMM_ERR_INVALID_ARG;
    if (in_dtype < BIGEMM_F32 || in_dtype > BIGEMM_BF16) return BIGEMM_ERR_INVALID_ARG;
    if (out_dtype < BIGEMM_F32 || out_dtype > BIGEMM_MXF8) return BIGEMM_ERR_INVALID_ARG;
    if (out_dtype != in_dtype && out_dtype != BIGEMM_F32 && out_dtype != BIGEMM_MXF8) return BIGEMM_ERR_UNSUPPORTED;
    if (rows == 0) return BIGEMM_OK;
    if (cols > kMaxCols) return BIGEMM_ERR_UNSUPPORTED;
    if (!x || !out || (out_dtype == BIGEMM_MXF8) != (out_scale != nullptr)) return BIGEMM_ERR_INVALID_ARG;
    if (ldx < cols || ldo < cols || (residual && ldr < cols) || (sum_out && lds < cols)) return BIGEMM_ERR_INVALID_ARG;
    const size_t es = dtype_size(in_dtype), os = out_dtype == BIGEMM_MXF8 ? 1 : dtype_size(out_dtype);
    if (!aligned(x, 0, 1, es) || !aligned(residual, 0, 1, es) || !aligned(sum_out, 0, 1, es) || !aligned(out, 0, 1, os) ||
        !aligned(weight, 0, 1, 4) || !aligned(bias, 0, 1, 4) || !aligned(out_scale, 0, 1, 16) || !aligned(mean, 0, 1, 4) ||
        !aligned(rstd, 0, 1, 4))
        return BIGEMM_ERR_INVALID_ARG;
    // out (of x's type) and sum_out may take the place of what a thread has read, row by row
    if (!distinct({weight, bias, out, sum_out, out_scale, mean, rstd}, 2) || !distinct({x, residual, out_scale, mean, rstd}, 2) ||
        !apart_or_in_place(sum_out, lds, x, ldx, rows) || !apart_or_in_place(sum_out, lds, residual, ldr, rows) ||
        !apart_or_in_place(out, ldo, x, ldx, rows) || !apart_or_in_place(out, ldo, residual, ldr, rows) ||
        (out_dtype != in_dtype && (out == x || out == residual)))
        return BIGEMM_ERR_INVALID_ARG;
    DeviceState *ds = device_state();
    if (!ds) return BIGEMM_ERR_CUDA;
    const bool vec = aligned(x, ldx, es, 16) && aligned(residual, ldr, es, 16) && aligned(sum_out, lds, es, 16) &&
                     aligned(out, ldo, os, out_dtype == BIGEMM_MXF8 ? 8 : 16);
    LayerNormArgs a = {};
    a.rows = rows, a.cols = cols;
    a.col_blocks = (int)(((long long)cols + kMxBlock - 1) / kMxBlock);
    a.pieces = out_dtype == BIGEMM_MXF8 ? a.col_blocks * (kMxBlock / kPiece)
                                        : (int)(((long long)cols + (vec ? 0 : kPiece - 1) + kPiece - 1) / kPiece);
    a.ldx = ldx, a.ldr = ldr, a.ldh = lds, a.ldo = ldo;
    a.x = x, a.residual = residual, a.weight = weight, a.bias = bias, a.eps = eps, a.inv_cols = 1.0f / (float)cols;
    a.vec_weight = weight && aligned(weight, 0, 1, 16), a.vec_bias = bias && aligned(bias, 0, 1, 16);
    a.h = sum_out, a.out = out, a.scale = static_cast<uint8_t *>(out_scale), a.mean = mean, a.rstd = rstd;
    const int form = out_dtype == BIGEMM_MXF8 ? OUT_MX : out_dtype == in_dtype ? OUT_SAME : OUT_F32;
    const cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = in_dtype == BIGEMM_F32   ? launch_layernorm_f32(a, form, vec, ds->sm_count, s)
                          : in_dtype == BIGEMM_F16 ? launch_layernorm_f16(a, form, vec, ds->sm_count, s)
                                                   : launch_layernorm_bf16(a, form, vec, ds->sm_count, s);
    return e == cudaSuccess ? BIGEMM_OK : BIGEMM_ERR_CUDA;
}

uint64_t norm_backward_workspace_bytes(int rows, int cols)
{
    return rows < 1 || cols < 1 || cols > kMaxCols ? 0 : back_workspace(rows, cols);
}

bigemm_status layernorm_backward_run(int rows, int cols, bigemm_dtype dtype, const void *dout, int64_t lddout, const void *x,
                                     int64_t ldx, const float *mean, const float *rstd, const float *weight,
                                     const void *dsum, int64_t lddsum, void *dx, int64_t lddx, float *dweight, float *dbias,
                                     void *workspace, uint64_t workspace_bytes, void *stream)
{
    NormBackArgs a = {};
    a.rows = rows, a.cols = cols, a.ldd = lddout, a.ldx = ldx, a.lds = lddsum, a.ldo = lddx;
    a.dout = dout, a.x = x, a.dsum = dsum, a.weight = weight, a.mean = mean, a.rstd = rstd;
    a.dx = dx, a.dweight = dweight, a.dbias = dbias;
    return norm_backward(a, true, dtype, workspace, workspace_bytes, stream);
}

bigemm_status rmsnorm_backward_run(int rows, int cols, bigemm_dtype dtype, const void *dout, int64_t lddout, const void *x,
                                   int64_t ldx, const float *weight, float eps, const void *dsum, int64_t lddsum, void *dx,
                                   int64_t lddx, float *dweight, void *workspace, uint64_t workspace_bytes, void *stream)
{
    NormBackArgs a = {};
    a.rows = rows, a.cols = cols, a.ldd = lddout, a.ldx = ldx, a.lds = lddsum, a.ldo = lddx;
    a.dout = dout, a.x = x, a.dsum = dsum, a.weight = weight, a.eps = eps, a.dx = dx, a.dweight = dweight;
    return norm_backward(a, false, dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
