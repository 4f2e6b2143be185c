// matmul.cu -- entry points of the matrix products (16-bit and MXFP8 operands):
// argument checks, tensor maps, and the choice of kernel.
#include <algorithm>

#include "matmul.cuh"
#include "matmul_gated.cuh"
#include "matmul_host.cuh"

using namespace bigemm;

namespace {

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

// Which kernel, and how it is cut: the least of estimates in nanoseconds whose
// terms were fitted to measurements (each term says to which).
struct Choice {
    bool many;
    int bn;          // many tokens: channels per tile
    FewCut few;
};

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
// GATED: tiles of 64 channels, and twice the weights.  Its terms were fitted to every cut of
// 99 gated layers (1 to 1024 tokens, 256 to 14336 channels): a block in 0.2 us, rows at 1.3 ns,
// 7, 15 and 4 ns for the others.  What is chosen takes 1.3 % more than the least of them in
// the mean (5.2 with the terms above: 16 x 2048 -> 2048 6.2 us with K in 8, 5.1 in 4;
// 256 x 1000 -> 1000 8.2 in tiles of 32, 6.8 of 64).
template <bool GATED>
long long few_cost(const MatmulArgs &a, int sms, const FewCut &c)
{
    const long long grid = up(a.N, GATED ? 64 : 128) * up(a.M, c.bn) * c.split;
    const long long beside = c.alone ? 1 : std::min<long long>(2, up(grid, sms)), waves = up(grid, beside * sms);
    const long long mine = up(std::min(a.M, c.bn), c.split);
    const bool ragged = !a.vec_out || (a.combine != BIGEMM_COMBINE_NONE && !a.vec_other);
    const long long block = GATED ? std::max<long long>(200, beside * (128 + c.bn) * 13 / 10)
                                  : std::max<long long>(165, beside * (128 + c.bn));
    const long long one = up(a.k_blocks, c.split) * block + (GATED ? 7 : 23) * mine + (GATED ? 15 : 22) * c.bn +
                          (GATED ? 4 : 2) * (c.split - 1) * beside * c.bn + (ragged ? 60 * mine * beside : 0);
    const long long memory = (long long)a.k_blocks * kRow * a.N * (GATED ? 2 : 1) / 6800;
    return 3600 + std::max(memory, waves * one);
}

// Many tokens, in pairs of CTAs: 3.5 us, and per wave of tiles over the pairs
// and block of K 0.33 us at 256 channels and 0.26 at 128 (where shared memory,
// not the tensor core, sets the pace), with MXFP8 operands 0.44 and 0.36.
// 4096 x 4096 x 4096 bf16: 79.6 us in 4 waves of 256, 110 in 7 of 128; 512 x 4096
// x 4096 24.7 in one wave of 256, 20.9 in one of 128.  A gated tile's end takes 3.1 us
// longer (256 x 256 -> 704 6.5 us, 4.2 for few tokens; 400 x 1000 -> 1000 11.5 and 8.5).
long long many_cost(const MatmulArgs &a, int sms, int bn, int channels, bool gated)
{
    const long long waves = up(up(a.M, kManyTokens) * up(a.N, channels), sms / 2);
    const bool mx = a.in_dt == BIGEMM_MXF8;
    return (gated ? 6600 : 3500) + waves * a.k_blocks * (bn == 256 ? (mx ? 440 : 330) : (mx ? 360 : 260));
}

// 256 x 4096 x 4096 bf16: 17.9 us for few (64 tokens, K in 2) against 20.4 and
// 24.4 in pairs; 512 x 4096 x 4096: 25 against 20.9 and 24.7; 1024 x 1024 x 8192:
// 25.5 against 34.5 and 40.9.
// GATED: the pairs' tiles have 128 channels of each product, and sum K in one accumulator.
template <bool GATED = false>
Choice choose(const MatmulArgs &a, int sms)
{
    const bool mx = a.in_dt == BIGEMM_MXF8, pieces = GATED ? a.seg_blocks < a.k_blocks : matmul_in_pieces(a);
    Choice c = {};
    long long least = -1;
    for (int bn = 16; bn <= 128; bn *= 2) {
        // running sums over pieces are in registers, of at most 64 tokens; smaller MXFP8 tiles
        // would start inside a block of scales
        if ((bn == 128 && pieces) || (mx && bn < 64 && a.M > bn)) continue;
        if (up(a.M, bn) > 65535) continue;     // the grid's second axis
        const long long tiles = up(a.N, GATED ? 64 : 128) * up(a.M, bn);
        // clusters of 5 to 7 CTAs leave SMs of their neighbourhood idle (300 x 1000 x 2048: 13.6 us in
        // 7, 8.9 in 4)
        for (int split : {1, 2, 3, 4, 8}) {
            if (split > 1 && (split * 4 > a.k_blocks || tiles * split > 2ll * sms)) break;
            // clusters of 3 and 8 CTAs that want an SM each do not fit the machine's groups of SMs (gated,
            // 80 x 3000 -> 3000 in 3: 20.0 us, 15.7 beside each other; 128 CTAs in 8: 1.3 to 1.6 times as long)
            const bool fits = split == 1 || split == 2 || split == 4;
            for (int alone = 0; alone <= (bn >= 64 && fits && tiles * split <= sms ? 1 : 0); ++alone) {
                const FewCut cut = {bn, split, alone != 0};
                const long long cost = few_cost<GATED>(a, sms, cut);
                if (least < 0 || cost <= least) c.few = cut, least = cost;
            }
        }
        if (bn >= a.M) break;                  // larger tiles hold no more
    }
    if (a.M > 128 && !(GATED && pieces))
        for (int bn = GATED ? 256 : 128; bn <= 256; bn += 128) {
            const long long cost = many_cost(a, sms, bn, GATED ? bn / 2 : bn, GATED);
            if (least < 0 || cost < least) c.many = true, c.bn = bn, least = cost;
        }
    return c;
}

// 128-byte pieces of a row that one tensor-memory accumulator sums where K is
// summed in pieces: 512 products of 16-bit operands (32 additions), 2048 of MXFP8 ones
// (64; their sums lose less per addition, and with one accumulator each hand-over
// costs 1 us per wave of tiles).  4096 x 8192 x 8192 MXFP8, error of the sums against
// 64 bits in the 2-norm and time to MXFP8 (graph replay): one sum 7.0e-7 and 182 us,
// pieces of 4096 3.3e-7 and 191, of 2048 1.5e-7 and 216, of 1024 1.0e-7 and 265; a
// plain fp32 product 1.5e-7.
int full_segment(bool mx) { return mx ? 16 : 8; }

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
    PackList k(workspace);
    k.add(a.w, a.ldw, a.N, a.K, es);
    k.add(a.x, a.ldx, a.M, a.K, es);
    return k.run(stream);
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

// A 16-bit output as boxes of 32 rows by 32 columns (if its rows are on the grid; true where none is needed).
bool put_map(CUtensorMap *map, bool vec, void *p, int dt, long long rows, long long cols, long long ld)
{
    return !p || !vec || box_map(map, p, dt, rows, cols, ld, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
}

uint64_t gated_workspace(const GatedArgs &a)
{
    return (uint64_t)((addressable(a.w, a.ldw, 2) ? 0 : packed_bytes(a.N, a.K, 2)) +
                      (addressable(a.w_up, a.ldw_up, 2) ? 0 : packed_bytes(a.N, a.K, 2)) +
                      (addressable(a.x, a.ldx, 2) ? 0 : packed_bytes(a.M, a.K, 2)));
}

bigemm_status gated(GatedArgs &a, void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (a.M < 0 || a.N < 1 || a.K < 1 || a.act < BIGEMM_ACT_NONE || a.act > BIGEMM_ACT_SILU) return BIGEMM_ERR_INVALID_ARG;
    if (a.M == 0) return BIGEMM_OK;
    if (a.M > kMaxSize || a.N > kMaxSize || a.K > kMaxSize) return BIGEMM_ERR_UNSUPPORTED;
    if (!a.x || !a.w || !a.w_up || !a.out) return BIGEMM_ERR_INVALID_ARG;
    if (a.ldx < a.K || a.ldw < a.K || a.ldw_up < a.K || a.ldo < a.N || (a.gate && a.ldgate < a.N) || (a.up && a.ldup < a.N))
        return BIGEMM_ERR_INVALID_ARG;
    if (!on_grid(a.x, 0, 1, 2) || !on_grid(a.w, 0, 1, 2) || !on_grid(a.w_up, 0, 1, 2) || !on_grid(a.out, 0, 1, 2) ||
        !on_grid(a.gate, 0, 1, 2) || !on_grid(a.up, 0, 1, 2) || !on_grid(a.bias, 0, 1, 4) || !on_grid(a.bias_up, 0, 1, 4))
        return BIGEMM_ERR_INVALID_ARG;
    if (!distinct({a.x, a.w, a.w_up, a.out, a.gate, a.up}, 3)) return BIGEMM_ERR_INVALID_ARG;
    const uint64_t space = gated_workspace(a);
    if (!on_grid(workspace, 0, 1, 16) || (space > 0 && (!workspace || workspace_bytes < space))) return BIGEMM_ERR_INVALID_ARG;
    DeviceState *ds = device_state();
    if (!ds) return BIGEMM_ERR_CUDA;
    const cudaStream_t s = (cudaStream_t)stream;
    a.vec_out = on_grid(a.out, a.ldo, 2, 16) && a.ldo * 2 < kFar;
    a.vec_gate = on_grid(a.gate, a.ldgate, 2, 16) && a.ldgate * 2 < kFar;
    a.vec_up = on_grid(a.up, a.ldup, 2, 16) && a.ldup * 2 < kFar;
    a.vec_bias = on_grid(a.bias, 0, 1, 16), a.vec_bias_up = on_grid(a.bias_up, 0, 1, 16);
    a.k_blocks = (int)up(a.K * 2ll, kRow);
    a.seg_blocks = a.K > kLongestSum ? full_segment(false) : a.k_blocks;
    a.timeout_ns = wait_timeout_ns();
    a.err = ds->err;
    PackList k(static_cast<uint8_t *>(workspace));
    k.add(a.w, a.ldw, a.N, a.K, 2);
    k.add(a.w_up, a.ldw_up, a.N, a.K, 2);
    k.add(a.x, a.ldx, a.M, a.K, 2);
    if (k.run(s) != cudaSuccess) return BIGEMM_ERR_CUDA;
    const Choice pick = choose<true>(a, ds->sm_count);
    if (pick.many) {
        const long long mt = up(a.M, kManyTokens), nt = up(a.N, 128);
        if (mt * nt > 0x7fffffff) return BIGEMM_ERR_UNSUPPORTED;
        a.m_tiles = (int)mt, a.n_tiles = (int)nt;
        GatedMaps maps = {};
        if (!operand_map(&maps.x, a.x, a.in_dt, a.M, a.K, a.ldx, 128) ||
            !operand_map(&maps.w[0], a.w, a.in_dt, a.N, a.K, a.ldw, 128) ||
            !operand_map(&maps.w[1], a.w_up, a.in_dt, a.N, a.K, a.ldw_up, 128) ||
            !put_map(&maps.out, a.vec_out, a.out, a.out_dt, a.M, a.N, a.ldo) ||
            !put_map(&maps.kept[0], a.vec_gate, a.gate, a.out_dt, a.M, a.N, a.ldgate) ||
            !put_map(&maps.kept[1], a.vec_up, a.up, a.out_dt, a.M, a.N, a.ldup))
            return BIGEMM_ERR_CUDA;
        return launch_gated_many(a, maps, ds->sm_count, s) == cudaSuccess ? BIGEMM_OK : BIGEMM_ERR_CUDA;
    }
    a.split = pick.few.split;
    CUtensorMap mg = {}, mu = {}, mxm = {};
    if (!operand_map(&mg, a.w, a.in_dt, a.N, a.K, a.ldw, 64) || !operand_map(&mu, a.w_up, a.in_dt, a.N, a.K, a.ldw_up, 64) ||
        !operand_map(&mxm, a.x, a.in_dt, a.M, a.K, a.ldx, pick.few.bn))
        return BIGEMM_ERR_CUDA;
    return launch_gated_few(a, pick.few, mg, mu, mxm, s) == cudaSuccess ? BIGEMM_OK : BIGEMM_ERR_CUDA;
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

uint64_t matmul_gated_workspace_bytes(int M, int N, int K, const void *x, int64_t ldx, const void *w_gate, int64_t ldw_gate,
                                      const void *w_up, int64_t ldw_up)
{
    if (M < 1 || N < 1 || K < 1) return 0;
    GatedArgs a = {};
    a.M = M, a.N = N, a.K = K, a.x = x, a.w = w_gate, a.w_up = w_up, a.ldx = ldx, a.ldw = ldw_gate, a.ldw_up = ldw_up;
    return gated_workspace(a);
}

bigemm_status matmul_gated_run(int M, int N, int K, bigemm_dtype dtype, const void *x, int64_t ldx, const void *w_gate,
                               int64_t ldw_gate, const void *w_up, int64_t ldw_up, const float *bias_gate,
                               const float *bias_up, int act, void *out, int64_t ldo, void *gate, int64_t ldgate, void *up,
                               int64_t ldup, void *workspace, uint64_t workspace_bytes, void *stream)
{
    if (dtype < BIGEMM_F32 || dtype > BIGEMM_BF16) return BIGEMM_ERR_INVALID_ARG;
    if (dtype == BIGEMM_F32) return BIGEMM_ERR_UNSUPPORTED;
    GatedArgs a = {};
    a.M = M, a.N = N, a.K = K, a.in_dt = a.out_dt = dtype, a.act = act;
    a.x = x, a.w = w_gate, a.w_up = w_up, a.ldx = ldx, a.ldw = ldw_gate, a.ldw_up = ldw_up;
    a.bias = bias_gate, a.bias_up = bias_up, a.out = out, a.ldo = ldo;
    a.gate = gate, a.ldgate = ldgate, a.up = up, a.ldup = ldup;
    return gated(a, workspace, workspace_bytes, stream);
}

}  // extern "C"
