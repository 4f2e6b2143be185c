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

// Which kernel, and how it is cut: the least of estimates in nanoseconds whose
// terms were fitted to measurements (each term says to which).
struct Choice {
    bool many;
    int bn;          // many tokens: channels per tile
    FewCut few;
};

long long up(long long a, long long b) { return (a + b - 1) / b; }

// Few tokens: bn tokens per tile, `split` CTAs on a tile's K.  A start and an end
// of 3.6 us; a block of K (128 bytes of each row) in 0.165 us, or as long as it
// takes to reach an SM that `beside` CTAs share, (128 + bn) rows at 1 ns each;
// 23 ns per token that a CTA finishes and 22 per token of the tile.  N = K = 1024
// bf16: 12.0, 9.4 and 7.8 us for 128 tokens in one tile with K whole, in 2 and
// in 4; 9.1, 7.2 and 6.1 in tiles of 64; 7.0 and 5.5 in tiles of 16 with K whole
// and in 2; 100 x 300 x 304: 13.0 us with 128-token tiles, 5.2 with 16.  2 ns per
// token and further rank for the sums that cross between SMs (100 x 4096 x 4096:
// 12.9 us for 128-token tiles in 4, 16.5 in 8).
// Weights that fill the machine come at 6.8 TB/s: 1 x 4096 x 4096 in 8: 8.1 us.
// Rows of the output or of other off the 16-byte grid go element by element, 60
// ns a token (777 x 5001 x 1000: 34 us, 128 tokens to a tile).
long long few_cost(const MatmulArgs &a, int sms, const FewCut &c)
{
    const long long grid = up(a.N, 128) * up(a.M, c.bn) * c.split;
    const long long beside = c.alone ? 1 : std::min<long long>(2, up(grid, sms)), waves = up(grid, beside * sms);
    const long long mine = up(std::min(a.M, c.bn), c.split);
    const bool ragged = !a.vec_out || (a.combine != BIGEMM_COMBINE_NONE && !a.vec_other);
    const long long one = up(a.k_blocks, c.split) * std::max<long long>(165, beside * (128 + c.bn)) + 23 * mine + 22 * c.bn +
                          2 * (c.split - 1) * beside * c.bn + (ragged ? 60 * mine * beside : 0);
    const long long memory = (long long)a.k_blocks * kRow * a.N / 6800;
    return 3600 + std::max(memory, waves * one);
}

// Many tokens, in pairs of CTAs: 3.5 us, and per wave of tiles over the pairs
// and block of K 0.33 us at 256 channels and 0.26 at 128 (where shared memory,
// not the tensor core, sets the pace), with MXFP8 operands 0.44 and 0.36.
// 4096 x 4096 x 4096 bf16: 79.6 us in 4 waves of 256, 110 in 7 of 128; 512 x 4096
// x 4096 24.7 in one wave of 256, 20.9 in one of 128.
long long many_cost(const MatmulArgs &a, int sms, int bn)
{
    const long long waves = up(up(a.M, kManyTokens) * up(a.N, bn), sms / 2);
    const bool mx = a.in_dt == BIGEMM_MXF8;
    return 3500 + waves * a.k_blocks * (bn == 256 ? (mx ? 440 : 330) : (mx ? 360 : 260));
}

// 256 x 4096 x 4096 bf16: 17.9 us for few (64 tokens, K in 2) against 20.4 and
// 24.4 in pairs; 512 x 4096 x 4096: 25 against 20.9 and 24.7; 1024 x 1024 x 8192:
// 25.5 against 34.5 and 40.9.
Choice choose(const MatmulArgs &a, int sms)
{
    const bool mx = a.in_dt == BIGEMM_MXF8;
    Choice c = {};
    long long least = -1;
    for (int bn = 16; bn <= 128; bn *= 2) {
        // running sums over pieces are in registers, of at most 64 tokens; smaller MXFP8 tiles
        // would start inside a block of scales
        if ((bn == 128 && matmul_in_pieces(a)) || (mx && bn < 64 && a.M > bn)) continue;
        if (up(a.M, bn) > 65535) continue;     // the grid's second axis
        const long long tiles = up(a.N, 128) * up(a.M, bn);
        // clusters of 5 to 7 CTAs leave SMs of their neighbourhood idle (300 x 1000 x 2048: 13.6 us in
        // 7, 8.9 in 4)
        for (int split : {1, 2, 3, 4, 8}) {
            if (split > 1 && (split * 4 > a.k_blocks || tiles * split > 2ll * sms)) break;
            for (int alone = 0; alone <= (bn >= 64 && tiles * split <= sms ? 1 : 0); ++alone) {
                const FewCut cut = {bn, split, alone != 0};
                const long long cost = few_cost(a, sms, cut);
                if (least < 0 || cost <= least) c.few = cut, least = cost;
            }
        }
        if (bn >= a.M) break;                  // larger tiles hold no more
    }
    if (a.M > 128)
        for (int bn = 128; bn <= 256; bn += 128) {
            const long long cost = many_cost(a, sms, bn);
            if (least < 0 || cost < least) c.many = true, c.bn = bn, least = cost;
        }
    return c;
}

constexpr int kMaxSize = 1 << 30;   // indices within a row are in 32 bits, byte offsets in 64

// 128-byte pieces of a row that one tensor-memory accumulator sums where K is
// summed in pieces: 512 products of 16-bit operands (32 additions), 2048 of MXFP8 ones
// (64; their sums lose less per addition, and with one accumulator each hand-over
// costs 1 us per wave of tiles).  4096 x 8192 x 8192 MXFP8, error of the sums against
// 64 bits in the 2-norm and time to MXFP8 (graph replay): one sum 7.0e-7 and 182 us,
// pieces of 4096 3.3e-7 and 191, of 2048 1.5e-7 and 216, of 1024 1.0e-7 and 265; a
// plain fp32 product 1.5e-7.
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
    a.seg_blocks = matmul_in_pieces(a) ? full_segment(mx) : a.k_blocks;
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
    a.split = cut.split;
    CUtensorMap mw = {}, mxm = {};
    if (!operand_map(&mw, a.w, a.in_dt, a.N, a.K, a.ldw, 128) ||
        !operand_map(&mxm, a.x, a.in_dt, a.M, a.K, a.ldx, cut.bn))
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
