// norm.cu -- the root-mean-square norm with the residual's addition, and the
// quantisation of a matrix to MXFP8.
//
//   h[r,k] = x[r,k] (+ residual[r,k])
//   y[r,k] = h[r,k] * rsqrt(mean_k h[r,k]^2 + eps) (* weight[k])
//
// in fp32 from the inputs to the one rounding of each output.  Both operators
// move each byte once and are bound by memory: a row stays in registers between
// its sum of squares and its outputs.  A thread holds pieces of 8 consecutive
// elements (16 bytes of a 16-bit type), so the 32 elements of an MXFP8 scale
// are four neighbouring lanes.
#include "norm.cuh"

namespace bigemm {

namespace {

// A warp takes a run of 1024 columns of a row: four pieces per lane, all loaded
// before the first is written.  The runs of all rows are numbered one after the
// other, eight to a block.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const NormArgs a, int runs, FastDiv by_runs)
{
    griddep_enter();
    constexpr int U = 4;
    const int lane = threadIdx.x & 31;
    // work items are (row, run); the block's first row in 64 bits, the rest from there
    const long long first = (long long)blockIdx.x * 8, r0 = first / runs;
    uint32_t run;
    const long long r = r0 + fd_divmod((uint32_t)(first - r0 * runs) + (threadIdx.x >> 5), by_runs, &run);
    if (r >= a.rows) return;
    const T *row = static_cast<const T *>(a.x) + r * a.ldx;
    const int p0 = (int)run * 32 * U + lane;
    const Span span = span_of(a.x, a.rows, a.ldx, a.cols, sizeof(T));
    Held<T, VEC> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (p0 + u * 32 < a.pieces) hold<T, VEC>(row, (p0 + u * 32) * kPiece, a.cols, span, x[u]);
    uint8_t *out = static_cast<uint8_t *>(a.out) + r * a.ldo, *scale = a.scale + mx_scale_row(r, a.col_blocks);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int p = p0 + u * 32;
        if (p - lane >= a.pieces) return;     // the whole warp is past the row
        float v[kPiece];
        if (p < a.pieces) {
            take<T, VEC>(x[u], p * kPiece, a.cols, v);
        } else {
#pragma unroll
            for (int i = 0; i < kPiece; ++i) v[i] = 0.f;
        }
        store_mx_piece<VEC>(out, scale, p * kPiece, a.cols, p < a.pieces, v);
    }
}

template <typename T>
cudaError_t launch_quantize_type(const NormArgs &a, bool vec, cudaStream_t s)
{
    const int runs = (a.pieces + 127) / 128;
    const long long blocks = (a.rows * runs + 7) / 8;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const FastDiv by = make_fastdiv((uint32_t)runs);
    const dim3 grid((unsigned)blocks);
    ProfScope prof("mx_quantize", s);
    return vec ? launch_pdl(mx_quantize_kernel<T, true>, grid, dim3(256), 0, s, a, runs, by)
               : launch_pdl(mx_quantize_kernel<T, false>, grid, dim3(256), 0, s, a, runs, by);
}

// Whether rows of `ld` elements of `size` bytes start on `to`-byte boundaries.
bool aligned(const void *p, long long ld, size_t size, size_t to)
{
    return !p || (reinterpret_cast<uintptr_t>(p) % to == 0 && (ld * (long long)size) % (long long)to == 0);
}

}  // namespace

}  // namespace bigemm

using namespace bigemm;

extern "C" {

bigemm_status rmsnorm_run(int rows, int cols, bigemm_dtype in_dtype, const void *x, int64_t ldx,
                          const void *residual, int64_t ldr, const float *weight, float eps,
                          void *sum_out, int64_t lds, bigemm_dtype out_dtype, void *out, int64_t ldo,
                          void *out_scale, void *stream)
{
    if (rows < 0 || cols < 1) return BIGEMM_ERR_INVALID_ARG;
    if (in_dtype < BIGEMM_F32 || in_dtype > BIGEMM_BF16) return BIGEMM_ERR_INVALID_ARG;
    if (out_dtype < BIGEMM_F32 || out_dtype > BIGEMM_MXF8) return BIGEMM_ERR_INVALID_ARG;
    if (out_dtype != in_dtype && out_dtype != BIGEMM_F32 && out_dtype != BIGEMM_MXF8)
        return BIGEMM_ERR_UNSUPPORTED;
    if (rows == 0) return BIGEMM_OK;
    if (cols > kMaxCols) return BIGEMM_ERR_UNSUPPORTED;
    if (!x || !out || (out_dtype == BIGEMM_MXF8) != (out_scale != nullptr)) return BIGEMM_ERR_INVALID_ARG;
    if (ldx < cols || ldo < cols || (residual && ldr < cols) || (sum_out && lds < cols))
        return BIGEMM_ERR_INVALID_ARG;
    const size_t es = dtype_size(in_dtype), os = out_dtype == BIGEMM_MXF8 ? 1 : dtype_size(out_dtype);
    if (!aligned(x, 0, 1, es) || !aligned(residual, 0, 1, es) || !aligned(sum_out, 0, 1, es) ||
        !aligned(out, 0, 1, os) || !aligned(weight, 0, 1, 4) || !aligned(out_scale, 0, 1, 16))
        return BIGEMM_ERR_INVALID_ARG;
    DeviceState *ds = device_state();
    if (!ds) return BIGEMM_ERR_CUDA;
    const bool vec = aligned(x, ldx, es, 16) && aligned(residual, ldr, es, 16) &&
                     aligned(sum_out, lds, es, 16) && aligned(out, ldo, os, out_dtype == BIGEMM_MXF8 ? 8 : 16);
    NormArgs a = {};
    a.rows = rows;
    a.cols = cols;
    a.col_blocks = (int)(((long long)cols + kMxBlock - 1) / kMxBlock);
    a.pieces = out_dtype == BIGEMM_MXF8 ? a.col_blocks * (kMxBlock / kPiece)
                                        : (int)(((long long)cols + (vec ? 0 : kPiece - 1) + kPiece - 1) / kPiece);
    a.ldx = ldx, a.ldr = ldr, a.ldh = lds, a.ldo = ldo;
    a.x = x, a.residual = residual, a.weight = weight, a.eps = eps, a.inv_cols = 1.0f / (float)cols;
    a.vec_weight = weight && aligned(weight, 0, 1, 16);
    a.h = sum_out, a.out = out, a.scale = static_cast<uint8_t *>(out_scale);
    const int form = out_dtype == BIGEMM_MXF8 ? OUT_MX : out_dtype == in_dtype ? OUT_SAME : OUT_F32;
    const cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = in_dtype == BIGEMM_F32   ? launch_norm_f32(a, form, vec, ds->sm_count, s)
                          : in_dtype == BIGEMM_F16 ? launch_norm_f16(a, form, vec, ds->sm_count, s)
                                                   : launch_norm_bf16(a, form, vec, ds->sm_count, s);
    return e == cudaSuccess ? BIGEMM_OK : BIGEMM_ERR_CUDA;
}

bigemm_status mx_quantize_run(int rows, int cols, bigemm_dtype in_dtype, const void *x, int64_t ldx,
                              void *out, int64_t ldo, void *scale, void *stream)
{
    if (rows < 0 || cols < 1) return BIGEMM_ERR_INVALID_ARG;
    if (in_dtype < BIGEMM_F32 || in_dtype > BIGEMM_BF16) return BIGEMM_ERR_INVALID_ARG;
    if (rows == 0) return BIGEMM_OK;
    if (cols > kMaxCols) return BIGEMM_ERR_UNSUPPORTED;
    if (!x || !out || !scale || ldx < cols || ldo < cols) return BIGEMM_ERR_INVALID_ARG;
    const size_t es = dtype_size(in_dtype);
    if (!aligned(x, 0, 1, es) || !aligned(scale, 0, 1, 16)) return BIGEMM_ERR_INVALID_ARG;
    if (!device_state()) return BIGEMM_ERR_CUDA;
    NormArgs a = {};
    a.rows = rows;
    a.cols = cols;
    a.col_blocks = (int)(((long long)cols + kMxBlock - 1) / kMxBlock);
    a.pieces = a.col_blocks * (kMxBlock / kPiece);
    a.ldx = ldx, a.ldo = ldo, a.x = x, a.out = out, a.scale = static_cast<uint8_t *>(scale);
    const bool vec = aligned(x, ldx, es, 16) && aligned(out, ldo, 1, 8);
    const cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = in_dtype == BIGEMM_F32   ? launch_quantize_type<float>(a, vec, s)
                          : in_dtype == BIGEMM_F16 ? launch_quantize_type<__half>(a, vec, s)
                                                   : launch_quantize_type<__nv_bfloat16>(a, vec, s);
    return e == cudaSuccess ? BIGEMM_OK : BIGEMM_ERR_CUDA;
}

uint64_t bigemm_mx_scale_bytes(int rows, int cols)
{
    if (rows < 1 || cols < 1) return 0;
    return (uint64_t)(((long long)rows + kMxBlock - 1) / kMxBlock) * (uint64_t)(((long long)cols + kMxBlock - 1) / kMxBlock) *
           kMxBlockBytes;
}

}  // extern "C"
