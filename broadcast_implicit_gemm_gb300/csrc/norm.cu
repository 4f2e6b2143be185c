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
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "mx.cuh"
#include "ptx.cuh"

namespace bigemm {

namespace {

constexpr int kPiece = 8;            // elements per thread and step
constexpr int kMaxCols = 1 << 30;    // index arithmetic within a row is in 32 bits

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

// 8 elements from column c on; zeros past the row's end.  VEC: the piece starts
// on a 16-byte boundary.
template <typename T, bool VEC>
__device__ __forceinline__ void load_piece(const T *row, int c, int cols, float (&v)[kPiece])
{
    if (VEC && c + kPiece <= cols) {
        const Piece<T> p = *reinterpret_cast<const Piece<T> *>(row + c);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) v[i] = to_f32<T>(p.e[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) v[i] = c + i < cols ? to_f32<T>(row[c + i]) : 0.f;
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_piece(T *row, int c, int cols, const float (&v)[kPiece])
{
    if (VEC && c + kPiece <= cols) {
        Piece<T> p;
#pragma unroll
        for (int i = 0; i < kPiece; ++i) p.e[i] = from_f32<T>(v[i]);
        *reinterpret_cast<Piece<T> *>(row + c) = p;
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (c + i < cols) row[c + i] = from_f32<T>(v[i]);
    }
}

// One piece of an MXFP8 row: every lane of the warp takes part, `live` lanes
// hold a piece inside the row padded to whole blocks of scales.  VEC: the e4m3
// piece starts on an 8-byte boundary.
template <bool VEC>
__device__ __forceinline__ void store_mx_piece(uint8_t *row, uint8_t *scale, long long r, int c,
                                               int cols, int col_blocks, bool live,
                                               const float (&v)[kPiece])
{
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) a = mx_amax(a, v[i]);
    a = mx_amax(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = mx_amax(a, __shfl_xor_sync(0xffffffffu, a, 2));
    const uint32_t code = mx_scale_code(a);
    // the four codes of a block of scales leave as one word
    uint32_t word = code << (8 * ((threadIdx.x >> 2) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if (!live) return;
    if ((threadIdx.x & 15) == 0)
        *reinterpret_cast<uint32_t *>(scale + mx_scale_offset(r, c / kMxGroup, col_blocks)) = word;
    const float inv = mx_inv_scale(code);
    const uint32_t lo = mx_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    const uint32_t hi = mx_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    if (VEC && c + kPiece <= cols) {
        *reinterpret_cast<uint2 *>(row + c) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (c + i < cols) row[c + i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
}

struct NormArgs {
    int cols, col_blocks, pieces;     // pieces: of a row, padded to whole blocks of scales for MXFP8
    long long rows, ldx, ldr, ldh, ldo;
    const void *x, *residual;
    const float *weight;
    float eps;
    void *h, *out;
    uint8_t *scale;
};

enum OutForm { OUT_SAME = 0, OUT_F32 = 1, OUT_MX = 2 };

// One block per row, PPT pieces per thread kept in registers; a row longer than
// that is read again for its outputs (PPT = 0).
template <typename T, int FORM, int THREADS, int PPT, bool VEC>
__global__ void __launch_bounds__(THREADS) rmsnorm_kernel(const NormArgs a)
{
    griddep_enter();
    constexpr int KEEP = PPT > 0 ? PPT : 1;
    __shared__ float part[THREADS / 32];
    const long long r = blockIdx.x;
    const T *x = static_cast<const T *>(a.x) + r * a.ldx;
    const T *res = a.residual ? static_cast<const T *>(a.residual) + r * a.ldr : nullptr;
    T *h = a.h ? static_cast<T *>(a.h) + r * a.ldh : nullptr;
    const int steps = PPT > 0 ? PPT : (a.pieces + THREADS - 1) / THREADS;
    float v[KEEP][kPiece];
    float sum = 0.f;
    auto take = [&](int s, float (&w)[kPiece]) {
        const int c = (s * THREADS + (int)threadIdx.x) * kPiece;
        load_piece<T, VEC>(x, c, a.cols, w);
        if (res) {
            float t[kPiece];
            load_piece<T, VEC>(res, c, a.cols, t);
#pragma unroll
            for (int i = 0; i < kPiece; ++i) w[i] += t[i];
        }
    };
#pragma unroll
    for (int s = 0; s < KEEP; ++s) {
        if (PPT > 0) take(s, v[s]);
    }
    if (PPT > 0) {
#pragma unroll
        for (int s = 0; s < KEEP; ++s) {
#pragma unroll
            for (int i = 0; i < kPiece; ++i) sum += v[s][i] * v[s][i];
        }
    } else {
        for (int s = 0; s < steps; ++s) {
            take(s, v[0]);
#pragma unroll
            for (int i = 0; i < kPiece; ++i) sum += v[0][i] * v[0][i];
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i) total += part[i];
    const float inv = 1.0f / sqrtf(total / (float)a.cols + a.eps);
    auto put = [&](int s, float (&w)[kPiece]) {
        const int p = s * THREADS + (int)threadIdx.x, c = p * kPiece;
        if (h) store_piece<T, VEC>(h, c, a.cols, w);
        float g[kPiece];
        if (a.weight) {
            load_piece<float, false>(a.weight, c, a.cols, g);
        } else {
#pragma unroll
            for (int i = 0; i < kPiece; ++i) g[i] = 1.f;
        }
        float y[kPiece];
#pragma unroll
        for (int i = 0; i < kPiece; ++i) y[i] = c + i < a.cols ? w[i] * inv * g[i] : 0.f;
        if (FORM == OUT_MX)
            store_mx_piece<VEC>(static_cast<uint8_t *>(a.out) + r * a.ldo, a.scale, r, c, a.cols,
                                a.col_blocks, p < a.pieces, y);
        else if (FORM == OUT_F32)
            store_piece<float, VEC>(static_cast<float *>(a.out) + r * a.ldo, c, a.cols, y);
        else
            store_piece<T, VEC>(static_cast<T *>(a.out) + r * a.ldo, c, a.cols, y);
    };
    if (PPT > 0) {
#pragma unroll
        for (int s = 0; s < KEEP; ++s) put(s, v[s]);
    } else {
        for (int s = 0; s < steps; ++s) {
            take(s, v[0]);
            put(s, v[0]);
        }
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) mx_quantize_kernel(const NormArgs a)
{
    griddep_enter();
    const long long total = a.rows * a.pieces;
    const long long step = (long long)gridDim.x * 256;
    // pieces of a row are a multiple of 16, so a group's lanes stay together
    for (long long i0 = (long long)blockIdx.x * 256; i0 < total; i0 += step) {
        const long long i = i0 + threadIdx.x;
        const bool live = i < total;
        const long long r = live ? i / a.pieces : 0;
        const int c = live ? (int)(i - r * a.pieces) * kPiece : 0;
        float v[kPiece];
        if (live) {
            load_piece<T, VEC>(static_cast<const T *>(a.x) + r * a.ldx, c, a.cols, v);
        } else {
#pragma unroll
            for (int j = 0; j < kPiece; ++j) v[j] = 0.f;
        }
        store_mx_piece<VEC>(static_cast<uint8_t *>(a.out) + r * a.ldo, a.scale, r, c, a.cols,
                            a.col_blocks, live, v);
    }
}

template <typename T, int FORM, bool VEC>
cudaError_t launch_norm_form(const NormArgs &a, cudaStream_t s)
{
    const dim3 grid((unsigned)a.rows);
    ProfScope prof("rmsnorm", s);
    if (a.pieces <= 128) return launch_pdl(rmsnorm_kernel<T, FORM, 128, 1, VEC>, grid, dim3(128), 0, s, a);
    if (a.pieces <= 256) return launch_pdl(rmsnorm_kernel<T, FORM, 256, 1, VEC>, grid, dim3(256), 0, s, a);
    if (a.pieces <= 512) return launch_pdl(rmsnorm_kernel<T, FORM, 256, 2, VEC>, grid, dim3(256), 0, s, a);
    if (a.pieces <= 1024) return launch_pdl(rmsnorm_kernel<T, FORM, 512, 2, VEC>, grid, dim3(512), 0, s, a);
    if (a.pieces <= 2048) return launch_pdl(rmsnorm_kernel<T, FORM, 512, 4, VEC>, grid, dim3(512), 0, s, a);
    return launch_pdl(rmsnorm_kernel<T, FORM, 512, 0, VEC>, grid, dim3(512), 0, s, a);
}

template <typename T>
cudaError_t launch_norm_type(const NormArgs &a, int form, bool vec, cudaStream_t s)
{
    switch (form) {
    case OUT_SAME: return vec ? launch_norm_form<T, OUT_SAME, true>(a, s) : launch_norm_form<T, OUT_SAME, false>(a, s);
    case OUT_F32: return vec ? launch_norm_form<T, OUT_F32, true>(a, s) : launch_norm_form<T, OUT_F32, false>(a, s);
    default: return vec ? launch_norm_form<T, OUT_MX, true>(a, s) : launch_norm_form<T, OUT_MX, false>(a, s);
    }
}

template <typename T>
cudaError_t launch_quantize_type(const NormArgs &a, bool vec, cudaStream_t s)
{
    const long long blocks = (a.rows * a.pieces + 255) / 256;
    const dim3 grid((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20)));
    ProfScope prof("mx_quantize", s);
    return vec ? launch_pdl(mx_quantize_kernel<T, true>, grid, dim3(256), 0, s, a)
               : launch_pdl(mx_quantize_kernel<T, false>, grid, dim3(256), 0, s, a);
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
    if (!device_state()) return BIGEMM_ERR_CUDA;
    NormArgs a = {};
    a.rows = rows;
    a.cols = cols;
    a.col_blocks = (int)(((long long)cols + kMxBlock - 1) / kMxBlock);
    a.pieces = out_dtype == BIGEMM_MXF8 ? a.col_blocks * (kMxBlock / kPiece)
                                        : (int)(((long long)cols + kPiece - 1) / kPiece);
    a.ldx = ldx, a.ldr = ldr, a.ldh = lds, a.ldo = ldo;
    a.x = x, a.residual = residual, a.weight = weight, a.eps = eps;
    a.h = sum_out, a.out = out, a.scale = static_cast<uint8_t *>(out_scale);
    const bool vec = aligned(x, ldx, es, 16) && aligned(residual, ldr, es, 16) &&
                     aligned(sum_out, lds, es, 16) && aligned(out, ldo, os, 16);
    const int form = out_dtype == BIGEMM_MXF8 ? OUT_MX : out_dtype == in_dtype ? OUT_SAME : OUT_F32;
    const cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = in_dtype == BIGEMM_F32   ? launch_norm_type<float>(a, form, vec, s)
                          : in_dtype == BIGEMM_F16 ? launch_norm_type<__half>(a, form, vec, s)
                                                   : launch_norm_type<__nv_bfloat16>(a, form, vec, s);
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
