// matmul.cu -- entry points of the matrix products (16-bit and MXFP8 operands):
// argument checks, tensor maps, and the choice of kernel.
#include <algorithm>

#include "matmul.cuh"

using namespace bigemm;

namespace {

bool on_grid(const void *p, long long ld, long long size, long long to)
{
    return reinterpret_cast<uintptr_t>(p) % (uintptr_t)to == 0 && (ld * size) % to == 0;
}

// The scales of a rows x cols MXFP8 matrix as boxes of `blocks` blocks, one below the other.
bool scale_map(CUtensorMap *map, const void *p, long long rows, long long cols, int blocks)
{
    const uint64_t cb = (uint64_t)((cols + kMxBlock - 1) / kMxBlock);
    const uint64_t dims[3] = {kMxBlockBytes / 4, cb, (uint64_t)((rows + kMxBlock - 1) / kMxBlock)};
    const uint64_t strides[2] = {kMxBlockBytes, cb * kMxBlockBytes};
    const uint32_t box[3] = {kMxBlockBytes / 4, 1, (uint32_t)blocks};
    const uint32_t ones[3] = {1, 1, 1};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_INT32, 3, p, dims, strides, box, ones, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// The output as boxes of 32 tokens by 32 channels, swizzled over the box's rows.
bool out_map(CUtensorMap *map, const MatmulArgs &a)
{
    const uint64_t es = a.out_dt == BIGEMM_MXF8 ? 1 : dtype_size(a.out_dt);
    const uint64_t dims[2] = {(uint64_t)a.N, (uint64_t)a.M};
    const uint64_t strides[1] = {(uint64_t)a.ldo * es};
    const uint32_t box[2] = {32, 32};
    const uint32_t ones[2] = {1, 1};
    const CUtensorMapDataType t = a.out_dt == BIGEMM_MXF8  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                  : a.out_dt == BIGEMM_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                  : a.out_dt == BIGEMM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                           : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encode_tiled(map, t, 2, a.out, dims, strides, box, ones,
                        es == 4   ? CU_TENSOR_MAP_SWIZZLE_128B
                        : es == 2 ? CU_TENSOR_MAP_SWIZZLE_64B
                                  : CU_TENSOR_MAP_SWIZZLE_32B);
}

// A row-major operand as boxes of box_rows rows by 128 bytes, 128-byte swizzle.
bool operand_map(CUtensorMap *map, const void *p, int dt, long long rows, long long cols, long long ld, int box_rows)
{
    const size_t es = dt == BIGEMM_MXF8 ? 1 : 2;
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows};
    const uint64_t strides[1] = {(uint64_t)ld * es};
    const uint32_t box[2] = {(uint32_t)(kRow / es), (uint32_t)box_rows};
    const uint32_t ones[2] = {1, 1};
    const CUtensorMapDataType t = dt == BIGEMM_MXF8  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                  : dt == BIGEMM_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    return encode_tiled(map, t, 2, p, dims, strides, box, ones, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Which kernel, and how it is cut.  The estimates are in hundredths of a
// microsecond, from sizes measured with 16-bit operands; a block (128 bytes) of
// K takes 1.3 to 1.4 times as long with MXFP8 ones, in every form alike.
struct Choice {
    bool many;
    int bn;          // many tokens: channels per tile
    FewCut few;
};

long long up(long long a, long long b) { return (a + b - 1) / b; }

// Few tokens: tiles of the fewest tokens that hold them all (each tile reads the
// weights again), K shared by as many CTAs as fit beside each other, two per SM
// for small tiles, one for large ones, up to the cluster's eight, as long as
// each keeps four blocks.
//   64 x 4096 x 4096: 23.3 us with K whole, 15.2 in 2, 11.5 in 4 (128 CTAs), 14.5 in 8
//   1 x 4096 x 4096: 19.2, 12.1, 8.5 and 8.1 us
FewCut cut_few(const MatmulArgs &a, int sms, int bn, bool alone)
{
    const long long tiles = up(a.N, 128) * up(a.M, bn), room = (alone ? 1 : 2) * (long long)sms;
    const long long most = std::min<long long>(a.k_blocks / 4, room / tiles);
    FewCut c;
    c.bn = bn;
    // clusters of 5 to 7 leave SMs of their processor cluster idle (300 x 1000 x 2048: 13.6 us in 7, 8.9 in 4)
    c.split = most >= 8 ? 8 : most >= 4 ? 4 : most >= 1 ? (int)most : 1;
    c.alone = alone && tiles * c.split <= sms;
    return c;
}

// A wave of it: a start and an end of 5.7 us, and per block of K 0.33 us for a
// CTA alone on its SM with 128 tokens, 0.37 for two with 64 each, 0.52 for two
// with 128.
long long few_cost(const MatmulArgs &a, int sms, const FewCut &c)
{
    const long long grid = up(a.N, 128) * up(a.M, c.bn) * c.split, per = up(a.k_blocks, c.split);
    // rows off the 16-byte grid leave element by element: 0.15 us a token (777 x 5001 x 1000: 34 us against 22 in pairs)
    const int ragged = a.vec_out && (a.combine == BIGEMM_COMBINE_NONE || a.vec_other) ? 0 : 15 * c.bn;
    return ragged + (c.alone ? 600 + 33 * per : up(grid, 2ll * sms) * (570 + (c.bn == 128 ? 52 : 37) * per));
}

// The pair kernel: 3.5 us, and per wave of tiles over the SM pairs and block of
// K 0.33 us at 256 channels, 0.26 at 128 (where shared memory, not the tensor
// core, sets the pace).
long long many_cost(const MatmulArgs &a, int sms, int bn)
{
    const long long waves = up(up(a.M, kManyTokens) * up(a.N, bn), sms / 2);
    return 350 + waves * a.k_blocks * (bn == 256 ? 33 : 26);
}

// Up to 128 tokens one tile of tokens is enough, and the few-token kernel has
// no rival: 128 x 4096 x 4096 13 us against 20.  Above, the least estimate:
// 256 x 4096 x 4096 17.7 us (64 tokens, K in 2) against 20.4 and 24.4 in pairs,
// 512 x 4096 x 4096 25 against 20.9 and 24.7, 1024 x 1024 x 8192 25.5 against
// 34.5 and 40.9.
Choice choose(const MatmulArgs &a, int sms)
{
    const bool full = a.out_dt == BIGEMM_F32;      // its running sums are in registers: at most 64 tokens
    Choice c = {};
    if (a.M <= 128) {
        c.few = cut_few(a, sms, a.M <= 16 ? 16 : a.M <= 32 ? 32 : a.M <= 64 || full ? 64 : 128, a.M > 32);
        return c;
    }
    c.few = cut_few(a, sms, 64, false);
    long long least = few_cost(a, sms, c.few);
    if (!full) {
        const FewCut large = cut_few(a, sms, 128, true);
        if (few_cost(a, sms, large) < least) c.few = large, least = few_cost(a, sms, large);
    }
    for (int bn = 128; bn <= 256; bn += 128) {
        const long long cost = many_cost(a, sms, bn);
        if (cost < least) c.many = true, c.bn = bn, least = cost;
    }
    return c;
}

constexpr int kMaxSize = 1 << 30;   // index arithmetic within a row is in 32 bits

// 128-byte pieces of a row that one tensor-memory accumulator sums for a 32-bit
// output: 512 products of 16-bit operands (32 additions), 2048 of MXFP8 ones
// (64; they have one accumulator, and each hand-over costs 1 us).
int full_segment(bool mx) { return mx ? 16 : 8; }

constexpr long long kFar = 1ll << 40;           // TMA: strides below 2^40 bytes

// Whether TMA can address an operand's rows.
bool addressable(const void *p, long long ld, long long es) { return on_grid(p, ld, es, 16) && ld * es < kFar; }

long long packed_bytes(long long rows, long long cols, long long es) { return up(rows * up(cols * es, 16) * 16, 256) * 256; }

uint64_t workspace_for(long long M, long long N, long long K, long long es, const void *x, long long ldx, const void *w,
                       long long ldw)
{
    return (uint64_t)((addressable(w, ldw, es) ? 0 : packed_bytes(N, K, es)) +
                      (addressable(x, ldx, es) ? 0 : packed_bytes(M, K, es)));
}

// Copies what TMA cannot address to `workspace` and makes it the operand; w
// first.  (Warps that brought such rows into the product's stages themselves, by
// aligned loads and shifts, took 26.5 us for 1 x 4097 x 4097 bf16 against 20.7,
// 6.5 for 8 x 64 x 65 against 5.0, 360 for 1000 x 4096 x 4097 against 45.)
cudaError_t pack(MatmulArgs &a, long long es, uint8_t *workspace, cudaStream_t stream)
{
    PackArgs k = {};
    if (!addressable(a.w, a.ldw, es)) {
        const long long pitch = up(a.K * es, 16) * 16;
        k.op[0] = {static_cast<const uint8_t *>(a.w), workspace, a.N, a.ldw * es, pitch, a.K * es, 0};
        a.w = workspace, a.ldw = pitch / es;
        workspace += packed_bytes(a.N, a.K, es);
    }
    if (!addressable(a.x, a.ldx, es)) {
        const long long pitch = up(a.K * es, 16) * 16;
        k.op[1] = {static_cast<const uint8_t *>(a.x), workspace, a.M, a.ldx * es, pitch, a.K * es, 0};
        a.x = workspace, a.ldx = pitch / es;
    }
    return launch_matmul_pack(k, stream);
}

bigemm_status product(MatmulArgs &a, void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (a.M < 0 || a.N < 1 || a.K < 1) return BIGEMM_ERR_INVALID_ARG;
    const bool mx = a.in_dt == BIGEMM_MXF8;
    if (a.act < BIGEMM_ACT_NONE || a.act > BIGEMM_ACT_SILU) return BIGEMM_ERR_INVALID_ARG;
    if (a.combine < BIGEMM_COMBINE_NONE || a.combine > BIGEMM_COMBINE_MUL) return BIGEMM_ERR_INVALID_ARG;
    if (a.M == 0) return BIGEMM_OK;
    if (a.M > kMaxSize || a.N > kMaxSize || a.K > kMaxSize) return BIGEMM_ERR_UNSUPPORTED;
    if (!a.x || !a.w || !a.out || (mx && (!a.xs || !a.ws))) return BIGEMM_ERR_INVALID_ARG;
    if ((a.out_dt == BIGEMM_MXF8) != (a.outs != nullptr)) return BIGEMM_ERR_INVALID_ARG;
    if (a.ldx < a.K || a.ldw < a.K || a.ldo < a.N) return BIGEMM_ERR_INVALID_ARG;
    const long long es = mx ? 1 : 2, os = a.out_dt == BIGEMM_MXF8 ? 1 : (long long)dtype_size(a.out_dt);
    if (!on_grid(a.x, 0, 1, es) || !on_grid(a.w, 0, 1, es) || !on_grid(a.out, 0, 1, os)) return BIGEMM_ERR_INVALID_ARG;
    if (!on_grid(a.xs, 0, 1, 16) || !on_grid(a.ws, 0, 1, 16) || !on_grid(a.outs, 0, 1, 16) ||
        !on_grid(a.bias, 0, 1, 4))
        return BIGEMM_ERR_INVALID_ARG;
    if (a.combine != BIGEMM_COMBINE_NONE) {
        if (a.other_dt < BIGEMM_F32 || a.other_dt > BIGEMM_BF16) return BIGEMM_ERR_INVALID_ARG;
        const long long ts = (long long)dtype_size(a.other_dt);
        if (!a.other || a.ldother < a.N || !on_grid(a.other, 0, 1, ts)) return BIGEMM_ERR_INVALID_ARG;
        a.vec_other = on_grid(a.other, a.ldother, ts, 16);
    }
    const uint64_t space = workspace_for(a.M, a.N, a.K, es, a.x, a.ldx, a.w, a.ldw);
    if (!on_grid(workspace, 0, 1, 16) || (space > 0 && (!workspace || workspace_bytes < space)))
        return BIGEMM_ERR_INVALID_ARG;
    DeviceState *ds = device_state();
    if (!ds) return BIGEMM_ERR_CUDA;
    a.vec_out = on_grid(a.out, a.ldo, os, a.out_dt == BIGEMM_MXF8 ? 8 : 16);
    a.vec_bias = on_grid(a.bias, 0, 1, 16);
    a.k_blocks = (int)((a.K * es + kRow - 1) / kRow);
    a.timeout_ns = wait_timeout_ns();
    a.err = ds->err;
    if (space > 0 && pack(a, es, static_cast<uint8_t *>(workspace), (cudaStream_t)stream) != cudaSuccess)
        return BIGEMM_ERR_CUDA;
    a.seg_blocks = a.out_dt == BIGEMM_F32 ? full_segment(mx) : a.k_blocks;
    const Choice pick = choose(a, ds->sm_count);
    if (pick.many) {
        const int bn = pick.bn;
        const long long mt = (a.M + kManyTokens - 1ll) / kManyTokens, nt = (a.N + bn - 1ll) / bn;
        if (mt * nt > 0x7fffffff) return BIGEMM_ERR_UNSUPPORTED;
        a.m_tiles = (int)mt, a.n_tiles = (int)nt;
        a.by_rows = on_grid(a.out, a.ldo, os, 16) && a.ldo * os < kFar && (a.combine == BIGEMM_COMBINE_NONE || a.vec_other);
        ManyMaps maps = {};
        if (!operand_map(&maps.x, a.x, a.in_dt, a.M, a.K, a.ldx, 128) ||
            !operand_map(&maps.w, a.w, a.in_dt, a.N, a.K, a.ldw, bn / 2) ||
            (mx && (!scale_map(&maps.xs, a.xs, a.M, a.K, 1) || !scale_map(&maps.ws, a.ws, a.N, a.K, bn / 128))) ||
            (a.by_rows && !out_map(&maps.out, a)))
            return BIGEMM_ERR_CUDA;
        const cudaError_t e = launch_matmul_many(a, bn, ds->sm_count, maps, (cudaStream_t)stream);
        return e == cudaSuccess ? BIGEMM_OK : BIGEMM_ERR_CUDA;
    }
    const FewCut cut = pick.few;
    if ((a.M + (long long)cut.bn - 1) / cut.bn > 65535) return BIGEMM_ERR_UNSUPPORTED;
    a.split = cut.split;
    CUtensorMap mw = {}, mxm = {};
    if ((!operand_map(&mw, a.w, a.in_dt, a.N, a.K, a.ldw, 128) ||
                    !operand_map(&mxm, a.x, a.in_dt, a.M, a.K, a.ldx, cut.bn)))
        return BIGEMM_ERR_CUDA;
    const cudaError_t e = launch_matmul_few(a, cut, mw, mxm, (cudaStream_t)stream);
    return e == cudaSuccess ? BIGEMM_OK : BIGEMM_ERR_CUDA;
}

}  // namespace

extern "C" {

uint64_t matmul_workspace_bytes(int M, int N, int K, bigemm_dtype in_dtype, const void *x, int64_t ldx, const void *w,
                                int64_t ldw)
{
    if (M < 1 || N < 1 || K < 1 || in_dtype < BIGEMM_F16 || in_dtype > BIGEMM_MXF8) return 0;
    return workspace_for(M, N, K, in_dtype == BIGEMM_MXF8 ? 1 : 2, x, ldx, w, ldw);
}

bigemm_status matmul_run(int M, int N, int K, bigemm_dtype in_dtype, const void *x, int64_t ldx, const void *w,
                         int64_t ldw, const float *bias, int act, int combine, bigemm_dtype other_dtype,
                         const void *other, int64_t ldother, bigemm_dtype out_dtype, void *out, int64_t ldo,
                         void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (in_dtype < BIGEMM_F32 || in_dtype > BIGEMM_BF16) return BIGEMM_ERR_INVALID_ARG;
    if (out_dtype < BIGEMM_F32 || out_dtype > BIGEMM_BF16) return BIGEMM_ERR_INVALID_ARG;
    if (in_dtype == BIGEMM_F32) return BIGEMM_ERR_UNSUPPORTED;
    MatmulArgs a = {};
    a.M = M, a.N = N, a.K = K, a.in_dt = in_dtype, a.out_dt = out_dtype, a.other_dt = other_dtype;
    a.act = act, a.combine = combine, a.x = x, a.w = w, a.ldx = ldx, a.ldw = ldw, a.ldo = ldo, a.ldother = ldother;
    a.bias = bias, a.other = other, a.out = out;
    return product(a, workspace, workspace_bytes, stream);
}

bigemm_status matmul_mx_run(int M, int N, int K, const void *x, int64_t ldx, const void *x_scale, const void *w,
                            int64_t ldw, const void *w_scale, const float *bias, int act, int combine,
                            bigemm_dtype other_dtype, const void *other, int64_t ldother, bigemm_dtype out_dtype,
                            void *out, int64_t ldo, void *out_scale, void *workspace, uint64_t workspace_bytes,
                            void *stream)
{
    if (out_dtype < BIGEMM_F32 || out_dtype > BIGEMM_MXF8) return BIGEMM_ERR_INVALID_ARG;
    MatmulArgs a = {};
    a.M = M, a.N = N, a.K = K, a.in_dt = BIGEMM_MXF8, a.out_dt = out_dtype, a.other_dt = other_dtype;
    a.act = act, a.combine = combine, a.x = x, a.w = w, a.ldx = ldx, a.ldw = ldw, a.ldo = ldo, a.ldother = ldother;
    a.xs = static_cast<const uint8_t *>(x_scale), a.ws = static_cast<const uint8_t *>(w_scale);
    a.bias = bias, a.other = other, a.out = out, a.outs = static_cast<uint8_t *>(out_scale);
    return product(a, workspace, workspace_bytes, stream);
}

}  // extern "C"
