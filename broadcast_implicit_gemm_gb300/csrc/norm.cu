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

// 8 elements from column c on; zeros past the row's end.  VEC: the piece starts
// on a 16-byte boundary.  Otherwise a 16-bit piece is cut out of the two
// aligned 16-byte words around it where both lie inside the row, which takes 2
// loads for 8; pieces at the row's ends go element by element.
template <typename T, bool VEC>
__device__ __forceinline__ Raw<T> load_raw(const T *row, int c, int cols)
{
    Raw<T> p;
    if (VEC && c + kPiece <= cols) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) p.q[i] = reinterpret_cast<const uint4 *>(row + c)[i];
        return p;
    }
    if (!VEC && sizeof(T) == 2 && c < cols) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + c), lo = at & ~(uintptr_t)15;
        if (lo >= reinterpret_cast<uintptr_t>(row) && lo + 32 <= reinterpret_cast<uintptr_t>(row + cols)) {
            const uint4 a = reinterpret_cast<const uint4 *>(lo)[0], b = reinterpret_cast<const uint4 *>(lo)[1];
            uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            const uint32_t by = (uint32_t)(at - lo);
            if (by & 8) {
#pragma unroll
                for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
            }
            if (by & 4) {
#pragma unroll
                for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
            }
            const uint32_t sh = (by & 2) * 8;
            p.q[0] = make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh),
                                __funnelshift_r(w[2], w[3], sh), __funnelshift_r(w[3], w[4], sh));
            return p;
        }
    }
    T *e = reinterpret_cast<T *>(&p);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) e[i] = c + i < cols ? row[c + i] : from_f32<T>(0.f);
    return p;
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
    // the four codes of a block of scales leave as one word
    uint32_t word = code << (8 * ((threadIdx.x >> 2) & 3));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if (!live) return;
    if ((threadIdx.x & 15) == 0)
        *reinterpret_cast<uint32_t *>(scale + (long long)(c / kMxBlock) * kMxBlockBytes) = word;
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
    bool vec_weight;                  // there, on a 16-byte boundary
    float eps;
    void *h, *out;
    uint8_t *scale;
};

enum OutForm { OUT_SAME = 0, OUT_F32 = 1, OUT_MX = 2 };

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int FORM, typename T, bool VEC>
__device__ __forceinline__ void norm_out(const NormArgs &a, long long r, int p, float inv, const float (&h)[kPiece],
                                         const float (&g)[kPiece])
{
    const int c = p * kPiece;
    float y[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) y[i] = c + i < a.cols ? h[i] * inv * g[i] : 0.f;
    if (FORM == OUT_MX)
        store_mx_piece<VEC>(static_cast<uint8_t *>(a.out) + r * a.ldo, a.scale + mx_scale_row(r, a.col_blocks), c, a.cols,
                            p < a.pieces, y);
    else if (FORM == OUT_F32)
        store_piece<float, VEC>(static_cast<float *>(a.out) + r * a.ldo, c, a.cols, y);
    else
        store_piece<T, VEC>(static_cast<T *>(a.out) + r * a.ldo, c, a.cols, y);
}

__device__ __forceinline__ void load_weight(const NormArgs &a, int c, float (&g)[kPiece])
{
    if (a.vec_weight && c + kPiece <= a.cols) {
        const float4 u = __ldg(reinterpret_cast<const float4 *>(a.weight + c));
        const float4 w = __ldg(reinterpret_cast<const float4 *>(a.weight + c + 4));
        g[0] = u.x, g[1] = u.y, g[2] = u.z, g[3] = u.w, g[4] = w.x, g[5] = w.y, g[6] = w.z, g[7] = w.w;
        return;
    }
#pragma unroll
    for (int i = 0; i < kPiece; ++i) g[i] = a.weight && c + i < a.cols ? __ldg(a.weight + c + i) : 1.f;
}

// TPR threads per row, PPT pieces per thread in registers; a block of
// max(TPR, 128) threads walks over its rows and loads the next one before it
// sums the present one, so that memory works through the sums and the barrier.
// (The weights come from L1 again for each row: as registers they cost a third
// of the rows in flight.)
template <typename T, int FORM, int TPR, int PPT, bool VEC>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, TPR < 128 ? 8 : 1024 / TPR) rmsnorm_kernel(const NormArgs a)
{
    griddep_enter();
    constexpr int THREADS = TPR < 128 ? 128 : TPR, ROWS = THREADS / TPR;
    static_assert(TPR == 32 || ROWS == 1, "a row has a warp or the block");
    __shared__ float part[2][THREADS / 32];
    const int t = (int)threadIdx.x % TPR;
    const long long step = (long long)gridDim.x * ROWS;
    long long r = (long long)blockIdx.x * ROWS + threadIdx.x / TPR;
    Raw<T> x[PPT], res[PPT];
    auto load = [&](long long row) {
        if (row >= a.rows) return;
#pragma unroll
        for (int s = 0; s < PPT; ++s)
            x[s] = load_raw<T, VEC>(static_cast<const T *>(a.x) + row * a.ldx, (s * TPR + t) * kPiece, a.cols);
        if (a.residual) {
#pragma unroll
            for (int s = 0; s < PPT; ++s)
                res[s] = load_raw<T, VEC>(static_cast<const T *>(a.residual) + row * a.ldr, (s * TPR + t) * kPiece,
                                          a.cols);
        }
    };
    load(r);
    // a warp without a row stays for the shuffles; a block's last turn is all of its warps'
    for (int turn = 0; r - (ROWS > 1 ? threadIdx.x / TPR : 0) < a.rows; ++turn, r += step) {
        float h[PPT][kPiece];
        float sum = 0.f;
        const bool live = r < a.rows;
#pragma unroll
        for (int s = 0; s < PPT; ++s) {
            unpack<T>(x[s], h[s]);
            if (a.residual) {
                float w[kPiece];
                unpack<T>(res[s], w);
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
            if ((threadIdx.x & 31) == 0) part[turn & 1][threadIdx.x >> 5] = sum;
            __syncthreads();
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < THREADS / 32; ++i) sum += part[turn & 1][i];
        }
        const float inv = 1.0f / sqrtf(sum / (float)a.cols + a.eps);
        if (!live) continue;
#pragma unroll
        for (int s = 0; s < PPT; ++s) {
            const int p = s * TPR + t;
            if (a.h) store_piece<T, VEC>(static_cast<T *>(a.h) + r * a.ldh, p * kPiece, a.cols, h[s]);
            float g[kPiece];
            load_weight(a, p * kPiece, g);
            norm_out<FORM, T, VEC>(a, r, p, inv, h[s], g);
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
    const int steps = (a.pieces + 511) / 512;
    auto take = [&](int p, float (&h)[kPiece]) {
        unpack<T>(load_raw<T, VEC>(x, p * kPiece, a.cols), h);
        if (res) {
            float w[kPiece];
            unpack<T>(load_raw<T, VEC>(res, p * kPiece, a.cols), w);
#pragma unroll
            for (int i = 0; i < kPiece; ++i) h[i] += w[i];
        }
    };
    float sum = 0.f;
    for (int s = 0; s < steps; ++s) {
        float h[kPiece];
        take(s * 512 + (int)threadIdx.x, h);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) sum += h[i] * h[i];
    }
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += part[i];
    const float inv = 1.0f / sqrtf(sum / (float)a.cols + a.eps);
    for (int s = 0; s < steps; ++s) {
        const int p = s * 512 + (int)threadIdx.x;
        float h[kPiece], g[kPiece];
        take(p, h);
        if (a.h) store_piece<T, VEC>(static_cast<T *>(a.h) + r * a.ldh, p * kPiece, a.cols, h);
        load_weight(a, p * kPiece, g);
        norm_out<FORM, T, VEC>(a, r, p, inv, h, g);
    }
}

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
    Raw<T> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (p0 + u * 32 < a.pieces) x[u] = load_raw<T, VEC>(row, (p0 + u * 32) * kPiece, a.cols);
    uint8_t *out = static_cast<uint8_t *>(a.out) + r * a.ldo, *scale = a.scale + mx_scale_row(r, a.col_blocks);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int p = p0 + u * 32;
        if (p - lane >= a.pieces) return;     // the whole warp is past the row
        float v[kPiece];
        if (p >= a.pieces) x[u] = Raw<T>{};
        unpack<T>(x[u], v);
        store_mx_piece<VEC>(out, scale, p * kPiece, a.cols, p < a.pieces, v);
    }
}

template <typename T, int FORM, int TPR, int PPT, bool VEC>
cudaError_t launch_norm_rows(const NormArgs &a, int sms, cudaStream_t s)
{
    constexpr int THREADS = TPR < 128 ? 128 : TPR, ROWS = THREADS / TPR;
    // one wave: 1024 threads per SM fit, whatever the registers
    const long long most = (long long)sms * (1024 / THREADS), need = (a.rows + ROWS - 1) / ROWS;
    return launch_pdl(rmsnorm_kernel<T, FORM, TPR, PPT, VEC>, dim3((unsigned)(need < most ? need : most)),
                      dim3(THREADS), 0, s, a);
}

// The fewest threads whose two pieces each hold a row, one piece for the
// shortest rows: 32 up to 512 columns, 1024 up to 16384.
template <typename T, int FORM, bool VEC>
cudaError_t launch_norm_form(const NormArgs &a, int sms, cudaStream_t s)
{
    ProfScope prof("rmsnorm", s);
    if (a.pieces <= 32) return launch_norm_rows<T, FORM, 32, 1, VEC>(a, sms, s);
    if (a.pieces <= 64) return launch_norm_rows<T, FORM, 32, 2, VEC>(a, sms, s);
    if (a.pieces <= 128) return launch_norm_rows<T, FORM, 128, 1, VEC>(a, sms, s);
    if (a.pieces <= 256) return launch_norm_rows<T, FORM, 128, 2, VEC>(a, sms, s);
    if (a.pieces <= 512) return launch_norm_rows<T, FORM, 256, 2, VEC>(a, sms, s);
    if (a.pieces <= 1024) return launch_norm_rows<T, FORM, 512, 2, VEC>(a, sms, s);
    if (a.pieces <= 2048) return launch_norm_rows<T, FORM, 1024, 2, VEC>(a, sms, s);
    return launch_pdl(rmsnorm_long_kernel<T, FORM, VEC>, dim3((unsigned)a.rows), dim3(512), 0, s, a);
}

template <typename T>
cudaError_t launch_norm_type(const NormArgs &a, int form, bool vec, int sms, cudaStream_t s)
{
    switch (form) {
    case OUT_SAME: return vec ? launch_norm_form<T, OUT_SAME, true>(a, sms, s) : launch_norm_form<T, OUT_SAME, false>(a, sms, s);
    case OUT_F32: return vec ? launch_norm_form<T, OUT_F32, true>(a, sms, s) : launch_norm_form<T, OUT_F32, false>(a, sms, s);
    default: return vec ? launch_norm_form<T, OUT_MX, true>(a, sms, s) : launch_norm_form<T, OUT_MX, false>(a, sms, s);
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
    NormArgs a = {};
    a.rows = rows;
    a.cols = cols;
    a.col_blocks = (int)(((long long)cols + kMxBlock - 1) / kMxBlock);
    a.pieces = out_dtype == BIGEMM_MXF8 ? a.col_blocks * (kMxBlock / kPiece)
                                        : (int)(((long long)cols + kPiece - 1) / kPiece);
    a.ldx = ldx, a.ldr = ldr, a.ldh = lds, a.ldo = ldo;
    a.x = x, a.residual = residual, a.weight = weight, a.eps = eps;
    a.vec_weight = weight && aligned(weight, 0, 1, 16);
    a.h = sum_out, a.out = out, a.scale = static_cast<uint8_t *>(out_scale);
    const bool vec = aligned(x, ldx, es, 16) && aligned(residual, ldr, es, 16) &&
                     aligned(sum_out, lds, es, 16) && aligned(out, ldo, os, 16);
    const int form = out_dtype == BIGEMM_MXF8 ? OUT_MX : out_dtype == in_dtype ? OUT_SAME : OUT_F32;
    const cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = in_dtype == BIGEMM_F32   ? launch_norm_type<float>(a, form, vec, ds->sm_count, s)
                          : in_dtype == BIGEMM_F16 ? launch_norm_type<__half>(a, form, vec, ds->sm_count, s)
                                                   : launch_norm_type<__nv_bfloat16>(a, form, vec, ds->sm_count, s);
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
