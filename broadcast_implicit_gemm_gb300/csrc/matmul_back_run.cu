// matmul_back_run.cu -- entry points of the products' gradients (matmul_back.cuh): checks of
// arguments, tensor maps, the cut of dx and the place of everything in the workspace.
#include <algorithm>

#include "column_sums.cuh"
#include "matmul_back.cuh"
#include "matmul_host.cuh"

using namespace bigemm;

namespace {

constexpr int kPairs = 76;           // of the machine: what cuts and workspaces are made for

// A product's gradients, or (count 2) a gated layer's.
struct Problem {
    int M, N, K, dt, count, act;
    const void *dout, *x, *w[2], *gate, *up;
    long long ldd, ldx, ldw[2], ldg, ldu;
    void *dx, *dw[2];
    long long lddx, lddw[2];
    float *dbias[2];
};

// How many shares the units of dx and of dw are cut into along their summed axis.  In
// blocks' time (0.33 us): a unit takes its blocks and kUnitCost more, all units together
// what they take over the pairs, no less than the longest or the waves of the longer kind,
// and each result's shares are written and read again in fp32 (at about 5 TB/s from L2)
// and joined.  Fewer shares where it makes no difference.  dx, 100 x 4096 x 4096: 26.9 us
// whole, 21.3 in 2, 22.8 in 4, 24.6 in 8; 777 x 5001 x 1000: 37.2, 27.5, 27.3 and 30.8;
// 1024 x 4096 x 4096: 45.1 whole, 62.3 in 2.  dw, 8192 x 512 x 512: 40.2 whole, 18.1 in 4,
// 15.4 in 8, 18.5 in 16.  (kUnitCost 4, 5, 6: 1 x 4096 x 4096 25.1, 21.6, 21.7 us;
// 64 x 8192 x 8192 57.4, 58.7, 60.8.)  A dw unit whose rows are off the 16-byte grid, written
// by plain stores, counts kOffGridCost when the pairs share the units out (5, 10, 14, 20, 32:
// 32 x 8782 x 1845 51, 47, 42, 42 and 42; 16 x 5632 x 7449 109, 95, 94, 97 and 103).
constexpr int kUnitCost = 5, kOffGridCost = 14;
struct Cut {
    int dx, dw;
};
long long fewest_shares(long long blocks) { return std::min<long long>(kMostShares, up(blocks, kLongestSum / 64)); }
Cut cut_of(const Problem &p)
{
    const long long blocks = p.count * up(p.N, 64), m_blocks = up(p.M, 64);
    const long long tiles = up(p.M, 256) * up(p.K, 256), dw_tiles = p.count * up(p.N, 256) * up(p.K, 256);
    long long least = -1;
    Cut best = {1, 1};
    // sums that are longer than one accumulator takes (131072 tokens through 4096 x 4096 in 4 shares 4683 us, 4665 in
    // one; dx of 4096 tokens over 65536 channels in 2 2513, 2394)
    const long long s_least = fewest_shares(blocks), t_least = fewest_shares(m_blocks);
    // (no more units than two waves of pairs: what is chosen from stays short, it is done twice a call)
    for (int t_try : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
        const long long t = std::max<long long>(t_try, t_least);
        if (t_try > 1 && (t * 4 > m_blocks || t * dw_tiles > 2 * kPairs)) break;
        for (int s_try : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
            const long long s = std::max<long long>(s_try, s_least);
            if (s_try > 1 && (s * 4 > blocks || s * tiles > 2 * kPairs)) break;
            const long long unit = up(blocks, s) + kUnitCost, dw_unit = up(m_blocks, t) + kUnitCost;
            const long long waves = unit >= dw_unit ? up(tiles * s, kPairs) * unit : up(dw_tiles * t, kPairs) * dw_unit;
            const long long walk = std::max(up(tiles * s * unit + dw_tiles * t * dw_unit, kPairs), waves);
            long long moved = 0;
            if (s > 1) moved += 2 * s * p.M * p.K * 4;
            if (t > 1) moved += 2 * t * p.count * p.N * p.K * 4;
            const long long cost = walk + (s > 1 || t > 1 ? 8 : 0) + moved / 1650000;
            if (least < 0 || cost < least) least = cost, best = {(int)s, (int)t};
        }
    }
    return best;
}

// Runs of rows of the elementwise kernel: eight blocks per SM, of 32 rows at least, and
// no second wave that is not a whole one (777 x 5001: 22 runs, not 25).  Without sums 16
// rows, which a block's warps have in flight at once, where those make less than two waves
// (gated, 64 x 256 -> 704: 11.8 us with 32, 10.3 with 16; 1024 x 1024 -> 2816 31.0 and 31.9).
int gate_runs(const Problem &p, bool vec, bool sums)
{
    const long long across = up(p.N, kGateColumns), wave = 2ll * kPairs * kGateBeside(vec);
    const int rows = !sums && up(p.M, 16) * across < 2 * wave ? 16 : 32;
    const long long want = std::min(std::max<long long>(1, 8 * 2 * kPairs / across), up(p.M, rows));
    return (int)(want * across > wave && want * across < 2 * wave && across <= wave ? wave / across : want);
}

struct Space {
    uint64_t pitch, d, packed, part_pitch, part, dw_part, sums, total;   // pitches in elements, places in bytes
    int runs;
    Cut cut;
};

Space space_of(const Problem &p)
{
    Space s = {};
    s.cut = cut_of(p), s.runs = std::max(gate_runs(p, false, true), gate_runs(p, true, true));
    uint64_t at = 0;
    auto take = [&](uint64_t bytes) {
        const uint64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    if (p.count == 2) {
        s.pitch = (uint64_t)up(p.N, 8) * 8;
        s.d = take(2 * s.pitch * (uint64_t)p.M * 2);
    }
    uint64_t packed = 0;
    if (p.count == 1 && !addressable(p.dout, p.ldd, 2)) packed += packed_bytes(p.M, p.N, 2);
    if (!addressable(p.x, p.ldx, 2)) packed += packed_bytes(p.M, p.K, 2);
    for (int i = 0; i < p.count; ++i)
        if (!addressable(p.w[i], p.ldw[i], 2)) packed += packed_bytes(p.N, p.K, 2);
    s.packed = take(packed);
    s.part_pitch = (uint64_t)up(p.K, 4) * 4;
    s.part = take(s.cut.dx > 1 ? (uint64_t)s.cut.dx * p.M * s.part_pitch * 4 : 0);
    s.dw_part = take(s.cut.dw > 1 ? (uint64_t)s.cut.dw * p.count * p.N * s.part_pitch * 4 : 0);
    // (whether there are biases, and how they lie, is not known to who asks for the size)
    s.sums = take((uint64_t)p.count * s.runs * sum_pitch(p.N) * 4);
    s.total = at;
    return s;
}

bool sizes_fit(const Problem &p) { return p.M <= kMaxSize && p.N <= kMaxSize && p.K <= kMaxSize; }

bool reach(const void *p, long long ld, long long cols) { return p && ld >= cols && on_grid(p, 0, 1, 2); }

// Shares, [count][rows][K], as boxes of 32 rows by 128 bytes.
bool part_map(CUtensorMap *map, const void *p, int count, int rows, int K, const Space &s)
{
    const uint64_t dims[3] = {(uint64_t)K, (uint64_t)rows, (uint64_t)count};
    const uint64_t strides[2] = {s.part_pitch * 4, s.part_pitch * 4 * (uint64_t)rows};
    const uint32_t box[3] = {32, 32, 1}, ones[3] = {1, 1, 1};
    return encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, p, dims, strides, box, ones, CU_TENSOR_MAP_SWIZZLE_128B);
}

JoinResult join_result(const void *part, int split, int rows, void *out, long long ld)
{
    return {static_cast<const float *>(part), out, ld, rows, split, on_grid(out, ld, 2, 8)};
}

bigemm_status zero_gradients(const Problem &p, cudaStream_t s)
{
    for (int i = 0; i < p.count; ++i) {
        if (cudaMemset2DAsync(p.dw[i], (size_t)p.lddw[i] * 2, 0, (size_t)p.K * 2, (size_t)p.N, s) != cudaSuccess) return BIGEMM_ERR_CUDA;
        if (p.dbias[i] && cudaMemsetAsync(p.dbias[i], 0, (size_t)p.N * 4, s) != cudaSuccess) return BIGEMM_ERR_CUDA;
    }
    return BIGEMM_OK;
}

bigemm_status gradients(Problem &p, void *workspace, uint64_t bytes, void *stream)
{
    if (p.M < 0 || p.N < 1 || p.K < 1 || p.dt < BIGEMM_F32 || p.dt > BIGEMM_BF16) return BIGEMM_ERR_INVALID_ARG;
    if (p.act < BIGEMM_ACT_NONE || p.act > BIGEMM_ACT_SILU) return BIGEMM_ERR_INVALID_ARG;
    if (p.dt == BIGEMM_F32 || !sizes_fit(p)) return BIGEMM_ERR_UNSUPPORTED;
    for (int i = 0; i < p.count; ++i)
        if (!reach(p.dw[i], p.lddw[i], p.K) || !on_grid(p.dbias[i], 0, 1, 4)) return BIGEMM_ERR_INVALID_ARG;
    const cudaStream_t s = (cudaStream_t)stream;
    if (p.M == 0) return device_state() ? zero_gradients(p, s) : BIGEMM_ERR_CUDA;
    if (!reach(p.dout, p.ldd, p.N) || !reach(p.x, p.ldx, p.K) || !reach(p.dx, p.lddx, p.K)) return BIGEMM_ERR_INVALID_ARG;
    for (int i = 0; i < p.count; ++i)
        if (!reach(p.w[i], p.ldw[i], p.K)) return BIGEMM_ERR_INVALID_ARG;
    if (p.count == 2 && (!reach(p.gate, p.ldg, p.N) || !reach(p.up, p.ldu, p.N))) return BIGEMM_ERR_INVALID_ARG;
    if (!distinct({p.dout, p.x, p.w[0], p.w[1], p.gate, p.up, p.dx, p.dw[0], p.dw[1], p.dbias[0], p.dbias[1]}, 6))
        return BIGEMM_ERR_INVALID_ARG;
    const Space at = space_of(p);
    if (!on_grid(workspace, 0, 1, 16) || !workspace || bytes < at.total) return BIGEMM_ERR_INVALID_ARG;
    DeviceState *ds = device_state();
    if (!ds) return BIGEMM_ERR_CUDA;
    uint8_t *space = static_cast<uint8_t *>(workspace);
    const int pairs_of_all = ds->sm_count / 2;

    // the products' operands
    const void *d[2] = {p.dout, nullptr};
    long long ldd[2] = {p.ldd, 0};
    GateBackArgs g = {};
    const bool biases = p.dbias[0] || p.dbias[1];
    const bool vec = on_grid(p.dout, p.ldd, 2, 16) && (p.count == 1 || (on_grid(p.gate, p.ldg, 2, 16) && on_grid(p.up, p.ldu, 2, 16)));
    g.M = p.M, g.N = p.N, g.runs = gate_runs(p, vec, biases), g.act = -1;
    g.dout = p.dout, g.gate = p.gate, g.up = p.up, g.ldd = p.ldd, g.ldg = p.ldg, g.ldu = p.ldu;
    float *sums = reinterpret_cast<float *>(space + at.sums);
    for (int i = 0; i < p.count; ++i)        // (a single run's sums are the result)
        g.sums[i] = p.dbias[i] && g.runs > 1 ? sums + i * g.runs * sum_pitch(p.N) : p.dbias[i];
    if (p.count == 2) {
        g.act = p.act, g.pitch = (long long)at.pitch;
        g.dg = space + at.d, g.du = space + at.d + at.pitch * (uint64_t)p.M * 2;
        d[0] = g.dg, d[1] = g.du, ldd[0] = ldd[1] = g.pitch;
    }
    const bool beside = p.count == 1 && p.M <= kSumsBeside;
    if ((p.count == 2 || (biases && !beside)) && launch_gate_back(g, p.dt, vec, s) != cudaSuccess) return BIGEMM_ERR_CUDA;
    if (biases && !beside && g.runs > 1) {
        ColumnSums c = {};
        c.parts = g.runs, c.cols = p.N;
        for (int i = 0; i < p.count; ++i)
            if (p.dbias[i]) c.from[c.count] = g.sums[i], c.out[c.count++] = p.dbias[i];
        if (launch_column_sums(c, s) != cudaSuccess) return BIGEMM_ERR_CUDA;
    }
    PackList k(space + at.packed);
    if (p.count == 1) k.add(d[0], ldd[0], p.M, p.N, 2);
    k.add(p.x, p.ldx, p.M, p.K, 2);
    for (int i = 0; i < p.count; ++i) k.add(p.w[i], p.ldw[i], p.N, p.K, 2);
    if (k.run(s) != cudaSuccess) return BIGEMM_ERR_CUDA;

    BackArgs a = {};
    BackMaps maps = {};
    a.M = p.M, a.N = p.N, a.K = p.K, a.dt = p.dt, a.count = p.count;
    const long long dx_m = up(p.M, 256), dw_m = up(p.N, 256), n = up(p.K, 256);
    const long long dx_units = dx_m * n * at.cut.dx, dw_units = p.count * dw_m * n * at.cut.dw;
    if (dx_units + dw_units > 0x3fffffff) return BIGEMM_ERR_UNSUPPORTED;
    a.n_blocks = (int)up(p.N, 64), a.dw_m = (int)dw_m;
    a.to_dx = make_unit_grid((int)dx_m, (int)n, at.cut.dx, p.count * a.n_blocks);
    a.to_dw = make_unit_grid((int)(p.count * dw_m), (int)n, at.cut.dw, (int)up(p.M, 64));
    const int pairs = (int)std::min<long long>(pairs_of_all, dx_units + dw_units);
    bool dw_grid = true;
    for (int i = 0; i < p.count; ++i) {
        a.dw[i] = p.dw[i], a.lddw[i] = p.lddw[i], a.dw_rows[i] = addressable(p.dw[i], p.lddw[i], 2);
        dw_grid = dw_grid && (a.dw_rows[i] || at.cut.dw > 1);    // (shares are on the grid)
    }
    const long long dx_time = up(a.to_dx.blocks, at.cut.dx) + kUnitCost;
    const long long dw_time = up(a.to_dw.blocks, at.cut.dw) + (dw_grid ? kUnitCost : kOffGridCost);
    a.dw_first = dw_time > dx_time;
    a.walk = a.dw_first ? make_back_walk((int)dw_units, (int)dx_units, pairs, dw_time, dx_time)
                        : make_back_walk((int)dx_units, (int)dw_units, pairs, dx_time, dw_time);
    a.dx = p.dx, a.lddx = p.lddx, a.dx_rows = addressable(p.dx, p.lddx, 2);
    if (beside) a.dout = p.dout, a.ldd = p.ldd, a.sums = p.dbias[0];
    a.timeout_ns = wait_timeout_ns();
    a.err = ds->err;
    bool ok = operand_map(&maps.x, p.x, p.dt, p.M, p.K, p.ldx, 64);
    for (int i = 0; i < p.count; ++i) {
        ok = ok && operand_map(&maps.d[i], d[i], p.dt, p.M, p.N, ldd[i], 64) &&
             operand_map(&maps.w[i], p.w[i], p.dt, p.N, p.K, p.ldw[i], 64) &&
             (!a.dw_rows[i] || at.cut.dw > 1 || box_map(&maps.dw[i], p.dw[i], p.dt, p.N, p.K, p.lddw[i], 32, 64, CU_TENSOR_MAP_SWIZZLE_128B));
    }
    if (at.cut.dx == 1 && a.dx_rows) ok = ok && box_map(&maps.dx, p.dx, p.dt, p.M, p.K, p.lddx, 32, 64, CU_TENSOR_MAP_SWIZZLE_128B);
    JoinArgs join = {};
    join.cols = p.K, join.pitch = (long long)at.part_pitch;
    if (at.cut.dx > 1) {
        ok = ok && part_map(&maps.part[0], space + at.part, at.cut.dx, p.M, p.K, at);
        join.result[join.count++] = join_result(space + at.part, at.cut.dx, p.M, p.dx, p.lddx);
    }
    if (at.cut.dw > 1) {
        ok = ok && part_map(&maps.part[1], space + at.dw_part, p.count * at.cut.dw, p.N, p.K, at);
        for (int i = 0; i < p.count; ++i)
            join.result[join.count++] = join_result(space + at.dw_part + (uint64_t)i * at.cut.dw * p.N * at.part_pitch * 4, at.cut.dw,
                                                    p.N, p.dw[i], p.lddw[i]);
    }
    if (!ok || launch_matmul_back(a, maps, pairs, s) != cudaSuccess) return BIGEMM_ERR_CUDA;
    return join.count == 0 || launch_back_join(join, p.dt, s) == cudaSuccess ? BIGEMM_OK : BIGEMM_ERR_CUDA;
}

}  // namespace

extern "C" {

uint64_t matmul_backward_workspace_bytes(int M, int N, int K, const void *dout, int64_t lddout, const void *x, int64_t ldx,
                                         const void *w, int64_t ldw)
{
    Problem p = {};
    p.M = M, p.N = N, p.K = K, p.count = 1, p.dout = dout, p.ldd = lddout, p.x = x, p.ldx = ldx, p.w[0] = w, p.ldw[0] = ldw;
    return M < 1 || N < 1 || K < 1 || !sizes_fit(p) ? 0 : space_of(p).total;
}

bigemm_status matmul_backward_run(int M, int N, int K, bigemm_dtype dtype, const void *dout, int64_t lddout, const void *x,
                                  int64_t ldx, const void *w, int64_t ldw, void *dx, int64_t lddx, void *dw, int64_t lddw,
                                  float *dbias, void *workspace, uint64_t workspace_bytes, void *stream)
{
    Problem p = {};
    p.M = M, p.N = N, p.K = K, p.dt = dtype, p.count = 1, p.dout = dout, p.ldd = lddout, p.x = x, p.ldx = ldx;
    p.w[0] = w, p.ldw[0] = ldw, p.dx = dx, p.lddx = lddx, p.dw[0] = dw, p.lddw[0] = lddw, p.dbias[0] = dbias;
    return gradients(p, workspace, workspace_bytes, stream);
}

uint64_t matmul_gated_backward_workspace_bytes(int M, int N, int K, const void *x, int64_t ldx, const void *w_gate,
                                               int64_t ldw_gate, const void *w_up, int64_t ldw_up)
{
    Problem p = {};
    p.M = M, p.N = N, p.K = K, p.count = 2, p.x = x, p.ldx = ldx;
    p.w[0] = w_gate, p.ldw[0] = ldw_gate, p.w[1] = w_up, p.ldw[1] = ldw_up;
    return M < 1 || N < 1 || K < 1 || !sizes_fit(p) ? 0 : space_of(p).total;
}

bigemm_status matmul_gated_backward_run(int M, int N, int K, bigemm_dtype dtype, const void *dout, int64_t lddout,
                                        const void *x, int64_t ldx, const void *w_gate, int64_t ldw_gate, const void *w_up,
                                        int64_t ldw_up, const void *gate, int64_t ldgate, const void *up, int64_t ldup,
                                        int act, void *dx, int64_t lddx, void *dw_gate, int64_t lddw_gate, void *dw_up,
                                        int64_t lddw_up, float *dbias_gate, float *dbias_up, void *workspace,
                                        uint64_t workspace_bytes, void *stream)
{
    Problem p = {};
    p.M = M, p.N = N, p.K = K, p.dt = dtype, p.count = 2, p.act = act, p.dout = dout, p.ldd = lddout, p.x = x, p.ldx = ldx;
    p.w[0] = w_gate, p.ldw[0] = ldw_gate, p.w[1] = w_up, p.ldw[1] = ldw_up;
    p.gate = gate, p.ldg = ldgate, p.up = up, p.ldu = ldup, p.dx = dx, p.lddx = lddx;
    p.dw[0] = dw_gate, p.lddw[0] = lddw_gate, p.dw[1] = dw_up, p.lddw[1] = lddw_up;
    p.dbias[0] = dbias_gate, p.dbias[1] = dbias_up;
    return gradients(p, workspace, workspace_bytes, stream);
}

}  // extern "C"
