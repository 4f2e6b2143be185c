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
// dsum and writes dx.  A block (a cluster of them where rows are long, a warp where they
// are short) walks over its rows with the next ones on their way into shared memory; a
// thread keeps the same columns all the way, so it adds up its part of the weights'
// gradients in registers.  Each block leaves one row of partial sums (152 rows of 8192
// columns against 8192 rows), which a second launch adds in their order: the result does
// not depend on timing.
#pragma once
#include "column_sums.cuh"
#include "norm.cuh"

namespace bigemm {

struct NormBackArgs {
    int cols;
    long long rows, ldd, ldx, lds, ldo;
    const void *dout, *x, *dsum;      // dsum: or null
    const float *weight, *mean, *rstd;
    float eps, inv_cols;
    void *dx;
    float *dweight, *dbias;           // a row per block or cluster, sum_pitch(cols) apart
    // one-pass kernels: rows that a walk moves on by, and the same in bytes of each matrix
    unsigned step;
    long long step_d, step_x, step_s, step_o;
    unsigned long long timeout_ns;
    int *err;
};

constexpr int kBackSms = 152;         // of the machine: one wave of blocks
constexpr int kBackCtaCols = 8192;    // of a block
constexpr int kBackMaxCols = 8 * kBackCtaCols;   // of the one-pass kernels: of a cluster

// Blocks of the one-pass kernels: at most 1024 threads per SM.
struct BackGrid {
    int threads, rows, cluster;       // rows: that a block takes at once; cluster: blocks on a row
    int parts;                        // rows of partial sums, at most: one per block or cluster
};

// Clusters of so many blocks, each with an SM to itself, that run at once on the current
// device: 36 of 4 and 15 of 8, not 38 and 19, since a cluster's SMs are neighbours (4096 x
// 40000 bf16 layer 720 us with 19, whose last four begin when others have done all their rows,
// and 462 with 15; 4096 x 20000 358 with 38, 197 with 36).  0: not known.
int back_clusters(int cluster);

inline BackGrid back_grid(long long rows, int cols)
{
    const int pieces = (cols + kPiece - 1) / kPiece;
    BackGrid g;
    g.cluster = 1;
    while (g.cluster < 8 && cols > g.cluster * kBackCtaCols) g.cluster *= 2;
    g.threads = pieces <= 32 ? 128 : ((pieces + g.cluster - 1) / g.cluster + 31) / 32 * 32;
    g.rows = pieces <= 32 ? 4 : 1;
    // a block beside another on its SM is worth its row of sums where each has four turns (2000 x 1000 f16 layer:
    // 12.0 us with as many as fit, 10.2 so, 11.6 with eight turns)
    const long long fits = 1024 / g.threads, worth = rows / (g.rows * 4ll * kBackSms);
    const long long beside = worth < 1 ? 1 : worth < fits ? worth : fits;
    const long long need = (rows + g.rows - 1) / g.rows, most = kBackSms * beside / g.cluster;
    g.parts = (int)(need < most ? need : most);
    return g;
}

namespace {

// Two fp32 values, for the instructions that take them together.
struct Pair {
    unsigned long long v;
};
__device__ __forceinline__ Pair pair(float a, float b)
{
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p.v) : "f"(a), "f"(b));
    return p;
}
__device__ __forceinline__ float2 both(Pair p)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p.v));
    return f;
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b)
{
    Pair p;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
    return p;
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b)
{
    Pair p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p.v) : "l"(a.v), "l"(b.v));
    return p;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c)
{
    Pair p;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return p;
}
constexpr int kPairs = kPiece / 2;

__device__ __forceinline__ void pairs_of(const float (&v)[kPiece], Pair (&p)[kPairs])
{
#pragma unroll
    for (int i = 0; i < kPairs; ++i) p[i] = pair(v[2 * i], v[2 * i + 1]);
}

// 8 elements as they lie in memory.
template <typename T>
__device__ __forceinline__ void pairs_of(const Raw<T> &r, Pair (&p)[kPairs])
{
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        const uint32_t q[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
        for (int i = 0; i < kPairs; ++i) p[i] = pair(__uint_as_float(q[i] << 16), __uint_as_float(q[i] & 0xffff0000u));
    } else {
        float f[kPiece];
        unpack<T>(r, f);
        pairs_of(f, p);
    }
}

// Two values as 16-bit ones.
template <typename T>
__device__ __forceinline__ uint32_t word_of(Pair p)
{
    const float2 f = both(p);
    if constexpr (std::is_same_v<T, __half>) {
        const __half2 h = __floats2half2_rn(f.x, f.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

// Where a thread's 8 elements of a row lie, the same in every row: on the 16-byte grid 16
// bytes each of its warp's next ones (8 in a row of 16 bits, twice 4 of 32); off it pairs,
// one of each 64.  A warp's loads and stores cover consecutive elements.
template <typename T, bool VEC>
struct Columns {
    static constexpr int run = VEC ? 16 / (int)sizeof(T) : 2;   // consecutive ones
    int c0;
    bool whole;                      // all of the warp's inside the row
    // thread t of the columns from base on
    __device__ __forceinline__ Columns(int t, int base, int cols)
    {
        const int warp = base + t / 32 * 32 * kPiece;
        c0 = warp + t % 32 * run;
        whole = warp + 32 * kPiece <= cols;
    }
    static __device__ __forceinline__ int off(int i) { return i / run * (32 * run) + i % run; }
    __device__ __forceinline__ int at(int i) const { return c0 + off(i); }
};

// A thread's elements of a row in memory; zeros past it.
template <typename T, bool VEC>
__device__ __forceinline__ void values_at(const T *row, const Columns<T, VEC> &c, int cols, float (&v)[kPiece])
{
    if (VEC && c.whole) {
        Raw<T> r;
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = *reinterpret_cast<const uint4 *>(row + c.at(i * c.run));
        unpack<T>(r, v);
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) v[i] = c.whole || c.at(i) < cols ? to_f32<T>(row[c.at(i)]) : 0.f;
    }
}

// The same to memory.
template <typename T, bool VEC>
__device__ __forceinline__ void put(T *row, const Columns<T, VEC> &c, int cols, const Pair (&p)[kPairs])
{
    if (c.whole) {
        if constexpr (sizeof(T) == 2) {
            uint32_t w[kPairs];
#pragma unroll
            for (int i = 0; i < kPairs; ++i) w[i] = word_of<T>(p[i]);
            if (VEC) {
                *reinterpret_cast<uint4 *>(row + c.c0) = make_uint4(w[0], w[1], w[2], w[3]);
            } else if (reinterpret_cast<uintptr_t>(row) % 4 == 0) {
#pragma unroll
                for (int i = 0; i < kPairs; ++i) *reinterpret_cast<uint32_t *>(row + c.at(2 * i)) = w[i];
            } else {
                // words of a lane's first and its neighbour's second element; the warp's ends by themselves
                const int lane = threadIdx.x & 31;
                uint16_t *e = reinterpret_cast<uint16_t *>(row) + c.c0;
#pragma unroll
                for (int i = 0; i < kPairs; ++i, e += 64) {
                    const uint32_t before = __shfl_up_sync(0xffffffffu, w[i], 1);
                    if (lane > 0) *reinterpret_cast<uint32_t *>(e - 1) = __funnelshift_r(before, w[i], 16);
                    if (lane == 0) e[0] = (uint16_t)w[i];
                    if (lane == 31) e[1] = (uint16_t)(w[i] >> 16);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                const float2 f = both(p[i]);
                if (VEC) {
                    const float2 g = both(p[i ^ 1]);
                    if (i % 2 == 0) *reinterpret_cast<float4 *>(row + c.at(2 * i)) = make_float4(f.x, f.y, g.x, g.y);
                } else {
                    row[c.at(2 * i)] = f.x, row[c.at(2 * i) + 1] = f.y;
                }
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const float2 f = both(p[i]);
        if (c.at(2 * i) < cols) row[c.at(2 * i)] = from_f32<T>(f.x);
        if (c.at(2 * i) + 1 < cols) row[c.at(2 * i) + 1] = from_f32<T>(f.y);
    }
}

// A thread's sums to a row of them, in words of its consecutive columns (one by one they
// touch each 32 bytes eight times: 500 x 2048 bf16 layer with dsum 18.5 us).
template <typename T, bool VEC>
__device__ __forceinline__ void put_sums(float *row, const Columns<T, VEC> &c, int cols, const float (&v)[kPiece])
{
    if (c.whole && reinterpret_cast<uintptr_t>(row) % 16 == 0) {
#pragma unroll
        for (int i = 0; i < kPiece; i += VEC ? 4 : 2) {
            if constexpr (VEC) *reinterpret_cast<float4 *>(row + c.at(i)) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            else *reinterpret_cast<float2 *>(row + c.at(i)) = make_float2(v[i], v[i + 1]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
        if (c.at(i) < cols) row[c.at(i)] = v[i];
}

template <typename T, bool VEC>
__device__ __forceinline__ void weights(const NormBackArgs &a, const Columns<T, VEC> &c, float (&g)[kPiece])
{
#pragma unroll
    for (int i = 0; i < kPiece; ++i) g[i] = a.weight && c.at(i) < a.cols ? a.weight[c.at(i)] : 1.f;
}

// Rows come through a ring in shared memory, three of dout, x and dsum (two of 32 bits).  On the
// 16-byte grid a thread copies what it reads itself, so the ring needs no barrier; off it a
// row's threads copy the 16-byte words that the row touches, and wait for each other.  The
// rows in flight take no registers either way.  (Held in registers, one row ahead: 8192 x
// 8192 bf16 with dsum 185 us, 97 so.  Longer rings are no faster: 16384 x 4096 f16 with
// dsum, RMS: 88, 84 and 92 us with two, three and four rows.)
template <typename T, bool SUM>
struct Ring {
    static constexpr int streams = SUM ? 3 : 2, q = (int)sizeof(T) / 2;      // 16-byte words of a piece
    static constexpr int stages = q == 1 ? 3 : 2;
    // words of one stream in a stage: off the grid a row touches one more than it has pieces' words
    static constexpr int words(bool vec, int threads) { return q * threads + (vec ? 0 : 1); }
    static constexpr int bytes(bool vec, int threads) { return stages * streams * words(vec, threads) * 16; }
};

// Shared memory by address.
__device__ __forceinline__ uint4 ld_shared16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_shared4(uint32_t at)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
template <typename T>
__device__ __forceinline__ T ld_shared_element(uint32_t at)
{
    if constexpr (sizeof(T) == 4) {
        float v;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
        return v;
    } else {
        uint16_t v;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
        return *reinterpret_cast<T *>(&v);
    }
}
template <typename T>
__device__ __forceinline__ void st_shared_element(uint32_t at, T v)
{
    if constexpr (sizeof(T) == 4) asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
    else asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"(*reinterpret_cast<const uint16_t *>(&v)) : "memory");
}

// A thread's piece of a row to shared memory: its words are 512 bytes apart, the ring's `by`;
// bytes: of each word, inside the row.
template <typename T>
__device__ __forceinline__ void copy_piece(uint32_t to, uint32_t by, const uint8_t *from, const int (&bytes)[2], bool there)
{
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) cp_async16_part(to + i * by, from + i * 512, there ? bytes[i] : 0);
}

template <typename T>
__device__ __forceinline__ void ring_piece(uint32_t from, uint32_t by, Pair (&p)[kPairs])
{
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.q[i] = ld_shared16(from + i * by);
    pairs_of<T>(r, p);
}

// Thread t of tpr's share of the words that `count` elements from `from` on touch.  `edge`:
// the matrix's first or last row, whose words may reach past it and come by elements then.
template <typename T>
__device__ __forceinline__ void copy_words(uint32_t to, const T *from, int count, int t, int tpr, bool edge, const Span &span)
{
    const int skew = (int)(reinterpret_cast<uintptr_t>(from) & 15), words = (skew + count * (int)sizeof(T) + 15) >> 4;
    const uint8_t *first = reinterpret_cast<const uint8_t *>(from) - skew;
    if (!edge) {
#pragma unroll
        for (int k = 0; k <= (int)sizeof(T) / 2; ++k) {
            const int w = t + k * tpr;
            cp_async16_part(to + w * 16, first + 16 * w, w < words ? 16 : 0);
        }
        return;
    }
#pragma unroll 1
    for (int w = t; w < words; w += tpr) {
        const uint8_t *at = first + 16 * w;
        if (at >= span.begin && at + 16 <= span.end) {
            cp_async16_part(to + w * 16, at, 16);
        } else {
            for (int i = 0; i < 16 / (int)sizeof(T); ++i) {
                const T *e = reinterpret_cast<const T *>(at) + i;
                if (e >= from && e < from + count) st_shared_element(to + w * 16 + i * (int)sizeof(T), *e);
            }
        }
    }
}

// A thread's elements of those words; zeros past the row.
template <typename T>
__device__ __forceinline__ void word_values(uint32_t words, const uint8_t *from, int base, const Columns<T, false> &c, int cols,
                                            Pair (&p)[kPairs])
{
    const uint32_t at = words + (uint32_t)(reinterpret_cast<uintptr_t>(from) & 15) + (uint32_t)(c.c0 - base) * (uint32_t)sizeof(T);
    float v[kPiece];
    if constexpr (sizeof(T) == 2) {
        if (c.whole) {
            uint32_t w[kPairs];
#pragma unroll
            for (int i = 0; i < kPairs; ++i)         // (an even start needs one of the two: no branch)
                w[i] = __funnelshift_r(ld_shared4((at & ~3u) + 128 * i), ld_shared4((at & ~3u) + 4 + 128 * i), (at & 2) * 8);
            Raw<T> r;
            r.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
            pairs_of<T>(r, p);
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < kPiece; ++i)
        v[i] = c.whole || c.at(i) < cols ? to_f32<T>(ld_shared_element<T>(at + (uint32_t)c.off(i) * (uint32_t)sizeof(T))) : 0.f;
    pairs_of(v, p);
}

// A warp's sum to the same place in every block of the cluster, counted on that block's
// barrier.  (A store and a barrier of the cluster wait for the rows written before, too:
// 8192 x 8192 in clusters of two 162 us.)
__device__ __forceinline__ void send_sum(float *at, uint64_t *bar, float v, int ranks)
{
    const uint32_t here = smem_u32(at), mine = smem_u32(bar);
    for (int k = 0; k < ranks; ++k)
        asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                         mapa_shared(here, (uint32_t)k)),
                     "r"(__float_as_uint(v)), "r"(mapa_shared(mine, (uint32_t)k))
                     : "memory");
}

// Sums of two values over the warp: lanes below 16 get x's, the others y's.
__device__ __forceinline__ float half_sums(float x, float y)
{
    const bool low = (threadIdx.x & 16) == 0;
    float v = (low ? x : y) + __shfl_xor_sync(0xffffffffu, low ? y : x, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// TPR: most threads of a row (a warp of four, or the block).  WIDE: the row has a cluster.
template <typename T, bool LAYER, bool SUM, int TPR, bool VEC, bool WIDE>
__global__ void __launch_bounds__(norm_threads(TPR), 1024 / norm_threads(TPR)) norm_back_kernel(const NormBackArgs a, int cluster)
{
    griddep_enter();
    static_assert(!WIDE || TPR > 32, "a cluster of whole blocks");
    constexpr int THREADS = norm_threads(TPR), ROWS = THREADS / TPR;
    using R = Ring<T, SUM>;
    constexpr int S = R::stages;
    extern __shared__ uint4 ring[];      // [stages][streams][words]; of ROWS rows, side by side
    __shared__ float part[2][2][32];     // by turn: the warps' sums of one kind, of the other
    __shared__ float wide[2][2][8];      // WIDE: the blocks' sums, and whether all are there
    __shared__ uint64_t sent[2];
    __shared__ volatile int abort_flag;
    const int warp = (int)threadIdx.x >> 5, lane = (int)threadIdx.x & 31, threads = (int)blockDim.x;
    const int tpr = TPR == 32 ? 32 : threads, t = TPR == 32 ? lane : (int)threadIdx.x;
    const int rank = WIDE ? (int)cluster_ctarank() : 0, mine = WIDE ? (int)blockIdx.x / cluster : (int)blockIdx.x;
    const int base = rank * threads * kPiece, columns = min(a.cols - base, tpr * kPiece);     // of this block
    const Columns<T, VEC> c(t, base, a.cols);
    // rows are below 2^31: so are r and what is a few steps ahead of it, unsigned
    const unsigned rows = (unsigned)a.rows;
    unsigned r = (unsigned)mine * ROWS + (TPR == 32 ? warp : 0), ahead = r;
    const Span d_span = span_of(a.dout, a.rows, a.ldd, a.cols, sizeof(T)), x_span = span_of(a.x, a.rows, a.ldx, a.cols, sizeof(T));
    const Span s_span = SUM ? span_of(a.dsum, a.rows, a.lds, a.cols, sizeof(T)) : d_span;
    // the next row to ask for, from this thread's first column on, or this block's
    const int first = VEC ? c.c0 : base, left = (a.cols - c.c0) * (int)sizeof(T);
    const int inside[2] = {max(0, min(16, left)), max(0, min(16, left - 512))};
    auto start = [&](const void *p, long long ld) { return static_cast<const uint8_t *>(p) + ((long long)r * ld + first) * (int)sizeof(T); };
    const uint8_t *next_d = start(a.dout, a.ldd), *next_x = start(a.x, a.ldx), *next_s = SUM ? start(a.dsum, a.lds) : nullptr;
    T *out = static_cast<T *>(a.dx) + (long long)r * a.ldo;
    // off the grid: where the present row starts within its first word
    const uint8_t *now_d = next_d, *now_x = next_x, *now_s = next_s;
    // the ring: a stage's words of each stream are `apart` bytes from the next stream's
    const uint32_t by = (uint32_t)threads * 16u, apart = (VEC ? R::q * threads : R::words(false, tpr)) * 16u;
    const uint32_t turn_bytes = apart * R::streams;
    const uint32_t ring0 = smem_u32(ring) + (VEC ? (uint32_t)threadIdx.x * 16u : ROWS > 1 ? (uint32_t)warp * S * turn_bytes : 0u);
    const uint32_t ring1 = ring0 + S * turn_bytes;
    uint32_t now = ring0, fill = ring0;
    auto fetch = [&]() {
        const bool there = ahead < rows;
        if constexpr (VEC) {
            copy_piece<T>(fill, by, next_d, inside, there);
            copy_piece<T>(fill + apart, by, next_x, inside, there);
            if (SUM) copy_piece<T>(fill + 2 * apart, by, next_s, inside, there);
        } else if (there) {
            const bool edge = ahead == 0 || ahead == rows - 1 || a.cols * (int)sizeof(T) < 16;
            copy_words<T>(fill, reinterpret_cast<const T *>(next_d), columns, t, tpr, edge, d_span);
            copy_words<T>(fill + apart, reinterpret_cast<const T *>(next_x), columns, t, tpr, edge, x_span);
            if (SUM) copy_words<T>(fill + 2 * apart, reinterpret_cast<const T *>(next_s), columns, t, tpr, edge, s_span);
        }
        ahead += a.step, next_d += a.step_d, next_x += a.step_x;
        if (SUM) next_s += a.step_s;
        fill += turn_bytes;
        if (fill == ring1) fill = ring0;
        cp_async_commit();
    };
    if (VEC && left <= (R::q - 1) * 512) {
        // words past the row: zeros, once
        for (uint32_t i = ring0; i != ring1; i += apart)
            for (int k = 0; k < R::q; ++k)
                if (inside[k] == 0)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(i + k * by), "r"(0) : "memory");
    }
    Pair dw[kPairs], db[LAYER ? kPairs : 1], w[kPairs];
    {
        float f[kPiece];
        weights<T, VEC>(a, c, f);
        pairs_of(f, w);
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) dw[i] = db[LAYER ? i : 0] = pair(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fetch();
    // statistics of 32 rows of the walk at a time, a lane's each
    float mean = 0.f, root = 0.f;
    if (WIDE) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < 2; ++i) mbar_init(&sent[i], 1);
            abort_flag = 0;
            fence_mbar_init();
        }
        cluster_sync_all();              // every block of the cluster runs, and its barriers are there
    }
    bool ok = true;
    // the loop's condition is the block's first row, so that no warp leaves another at the barrier or in a shuffle
    for (int n = 0; r - (ROWS > 1 ? warp : 0) < rows; ++n, r += a.step) {
        const bool live = r < rows;
        const int turn = n & 1;
        if (LAYER && (n & 31) == 0) {
            const unsigned at = r + lane * a.step;
            if (at < rows) mean = a.mean[at], root = a.rstd[at];
        }
        Pair d[kPairs], x[kPairs];
        cp_async_wait<S - 2>();
        if constexpr (VEC) {
            ring_piece<T>(now, by, d);
            ring_piece<T>(now + apart, by, x);
        } else {
            // the row's words of all its threads; and all have done with the stage before
            if (TPR == 32) __syncwarp();
            else __syncthreads();
            word_values<T>(now, now_d, base, c, a.cols, d);
            word_values<T>(now + apart, now_x, base, c, a.cols, x);
        }
        if (ROWS > 1 && !live) {             // a warp past the last row: what its words hold is nothing's
#pragma unroll
            for (int i = 0; i < kPairs; ++i) d[i] = x[i] = pair(0.f, 0.f);
        }
        fetch();
        float rstd = LAYER ? __shfl_sync(0xffffffffu, root, n & 31) : 0.f;
        // sums over the row: of g xh and g; of g x and x x
        Pair s0 = pair(0.f, 0.f), s1 = s0;
        if (LAYER) {
            const float m0 = -__shfl_sync(0xffffffffu, mean, n & 31);
            const Pair m = pair(m0, m0), scale = pair(rstd, rstd);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                x[i] = (x[i] + m) * scale;                       // (outside the row d is 0)
                dw[i] = fma(d[i], x[i], dw[i]);
                db[LAYER ? i : 0] = db[LAYER ? i : 0] + d[i];
                d[i] = d[i] * w[i];                              // g from here on
                s0 = fma(d[i], x[i], s0);
                s1 = s1 + d[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                s0 = fma(d[i] * w[i], x[i], s0);
                s1 = fma(x[i], x[i], s1);
            }
        }
        const float2 f0 = both(s0), f1 = both(s1);
        float sum = half_sums(f0.x + f0.y, f1.x + f1.y);
        if (TPR > 32) {
            const int warps = threads >> 5, kind = lane >> 4;
            float(&places)[2][32] = part[turn];
            if ((lane & 15) == 0) places[kind][warp] = sum;
            __syncthreads();
            if (!WIDE || warp == 0) {
                sum = (lane & 15) < warps ? places[kind][lane & 15] : 0.f;
                if ((lane & 15) + 16 < warps) sum += places[kind][(lane & 15) + 16];
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            }
            if (WIDE) {
                // the block's sums to every block of the cluster.  A place is written again two turns on, by a block
                // that has had this one's sums of the turn between, which went when all warps here had read the place.
                // (the wait is at the cluster's scope, where the stores come from: 8192 x 12288 201 us, 228 at the block's)
                if (threadIdx.x == 0) mbar_arrive_expect_tx(&sent[turn], (uint32_t)cluster * 8u);
                if (warp == 0 && (lane & 15) == 0) send_sum(&wide[turn][kind][rank], &sent[turn], sum, cluster);
                ok = ok && mbar_wait_warp<true>(&sent[turn], (uint32_t)(n >> 1) & 1u, a.timeout_ns, &abort_flag, a.err);
                sum = (lane & 15) < cluster ? wide[turn][kind][lane & 15] : 0.f;
#pragma unroll
                for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            }
        }
        const float sum0 = __shfl_sync(0xffffffffu, sum, 0), sum1 = __shfl_sync(0xffffffffu, sum, 16);
        if (live && ok) {
            Pair level, slope, o[kPairs];
            if (LAYER) {
                slope = pair(-sum0 * a.inv_cols, -sum0 * a.inv_cols), level = pair(-sum1 * a.inv_cols, -sum1 * a.inv_cols);
            } else {
                rstd = rsqrtf(sum1 * a.inv_cols + a.eps);
                const float f = -rstd * rstd * (sum0 * a.inv_cols);
                slope = pair(f, f);
            }
            const Pair scale = pair(rstd, rstd);
            Pair s[kPairs];
            if constexpr (SUM && VEC) ring_piece<T>(now + 2 * apart, by, s);
            if constexpr (SUM && !VEC) word_values<T>(now + 2 * apart, now_s, base, c, a.cols, s);
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                Pair v;
                if (LAYER) {
                    v = fma(x[i], slope, d[i] + level);
                } else {
                    v = fma(x[i], slope, d[i] * w[i]);
                    dw[i] = fma(d[i] * scale, x[i], dw[i]);
                }
                o[i] = SUM ? fma(v, scale, s[i]) : v * scale;
            }
            put<T, VEC>(out, c, a.cols, o);
        }
        out = reinterpret_cast<T *>(reinterpret_cast<uint8_t *>(out) + a.step_o);
        if (!VEC) {
            now_d += a.step_d, now_x += a.step_x;
            if (SUM) now_s += a.step_s;
        }
        now += turn_bytes;
        if (now == ring1) now = ring0;
    }
    if (WIDE) cluster_sync_all();        // no block leaves while sums are on their way to it
    if (!ok) return;
    float *to_w = a.dweight + mine * sum_pitch(a.cols), *to_b = LAYER ? a.dbias + mine * sum_pitch(a.cols) : nullptr;
    float fw[kPiece], fb[LAYER ? kPiece : 1];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const float2 f = both(dw[i]);
        fw[2 * i] = f.x, fw[2 * i + 1] = f.y;
        if constexpr (LAYER) {
            const float2 g = both(db[i]);
            fb[2 * i] = g.x, fb[2 * i + 1] = g.y;
        }
    }
    if (ROWS > 1) {
        // four warps, the same columns; over the ring, which nothing more is on its way to
        float *total = reinterpret_cast<float *>(ring);
        cp_async_wait<0>();
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
            total[(warp * 2) * 32 * kPiece + i * 32 + lane] = fw[i];
            if (LAYER) total[(warp * 2 + 1) * 32 * kPiece + i * 32 + lane] = fb[LAYER ? i : 0];
        }
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
#pragma unroll
            for (int k = 1; k < ROWS; ++k) {
                fw[i] += total[(k * 2) * 32 * kPiece + i * 32 + lane];
                if (LAYER) fb[LAYER ? i : 0] += total[(k * 2 + 1) * 32 * kPiece + i * 32 + lane];
            }
    }
    put_sums(to_w, c, a.cols, fw);
    if constexpr (LAYER) put_sums(to_b, c, a.cols, fb);
}

// Rows of more columns than a cluster of eight holds take two kernels.  The first adds up the weights'
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
    // pieces of a run by themselves, so that no sum has more than some hundred additions behind it (up to
    // some hundred thousand rows)
    constexpr int kPieceRows = 256;
    float dw = 0.f, db = 0.f;
    for (long long r = r0; r < r1;) {
        const long long end = min(r + kPieceRows, r1);
        float pw = 0.f, pb = 0.f;
#pragma unroll 4
        for (; r < end; ++r) {
            const float dv = to_f32<T>(d[r * a.ldd]), xv = to_f32<T>(x[r * a.ldx]);
            pw = fmaf(dv, LAYER ? (xv - a.mean[r]) * rstds[r] : xv * rstds[r], pw);
            if (LAYER) pb += dv;
        }
        dw += pw, db += pb;
    }
    a.dweight[blockIdx.y * sum_pitch(a.cols) + c] = dw;
    if (LAYER) a.dbias[blockIdx.y * sum_pitch(a.cols) + c] = db;
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
    auto row_at = [&](int s, Columns<T, VEC> &c, float (&g)[kPiece], float (&xh)[kPiece]) {
        c = Columns<T, VEC>((int)threadIdx.x, s * 512 * kPiece, a.cols);
        float d[kPiece], x[kPiece];
        values_at<T, VEC>(dr, c, a.cols, d);
        values_at<T, VEC>(xr, c, a.cols, x);
        weights<T, VEC>(a, c, g);
#pragma unroll
        for (int i = 0; i < kPiece; ++i) g[i] *= d[i], xh[i] = (x[i] - m) * rstd;
    };
    Columns<T, VEC> c(0, 0, 0);
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
            float v[kPiece];
            values_at<T, VEC>(sr, c, a.cols, v);
#pragma unroll
            for (int i = 0; i < kPiece; ++i) o[i] += v[i];
        }
        Pair p[kPairs];
        pairs_of(o, p);
        put<T, VEC>(to, c, a.cols, p);
    }
}

template <typename T, bool LAYER, bool SUM, int TPR, bool VEC, bool WIDE = false>
cudaError_t launch_back_tpr(NormBackArgs a, const BackGrid &g, cudaStream_t s)
{
    auto kern = norm_back_kernel<T, LAYER, SUM, TPR, VEC, WIDE>;
    using R = Ring<T, SUM>;
    constexpr int rows = norm_threads(TPR) / TPR, most = rows * R::bytes(VEC, TPR);
    static std::atomic<unsigned long long> attr_set{0};   // bit per device: smem opt-in done
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev >= 64 || !(attr_set >> dev & 1ull)) {
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e != cudaSuccess) return e;
        if (dev < 64) attr_set |= 1ull << dev;
    }
    a.step = (unsigned)(g.parts * rows);
    const long long es = (long long)sizeof(T);
    a.step_d = a.step * a.ldd * es, a.step_x = a.step * a.ldx * es, a.step_s = a.step * a.lds * es, a.step_o = a.step * a.ldo * es;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(g.parts * g.cluster));
    cfg.blockDim = dim3((unsigned)g.threads);
    cfg.dynamicSmemBytes = (size_t)(rows > 1 ? most : R::bytes(VEC, g.threads));
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)g.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = WIDE ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, g.cluster);
}

template <typename T, bool LAYER, bool SUM, bool VEC>
cudaError_t launch_back_rows(const NormBackArgs &a, int parts, cudaStream_t s)
{
    BackGrid g = back_grid(a.rows, a.cols);
    g.parts = parts;
    if (g.rows > 1) return launch_back_tpr<T, LAYER, SUM, 32, VEC>(a, g, s);
    if (g.cluster > 1)
        return launch_back_tpr<T, LAYER, SUM, kBackCtaCols / kPiece, VEC, true>(a, g, s);
    if (g.threads <= 256) return launch_back_tpr<T, LAYER, SUM, 256, VEC>(a, g, s);
    if (g.threads <= 512) return launch_back_tpr<T, LAYER, SUM, 512, VEC>(a, g, s);
    return launch_back_tpr<T, LAYER, SUM, 1024, VEC>(a, g, s);
}

template <typename T, bool LAYER, bool VEC>
cudaError_t launch_back_vec(const NormBackArgs &a, float *rstds, int parts, cudaStream_t s)
{
    ProfScope prof(LAYER ? "layernorm_backward" : "rmsnorm_backward", s);
    if (a.cols <= kBackMaxCols)
        return a.dsum ? launch_back_rows<T, LAYER, true, VEC>(a, parts, s) : launch_back_rows<T, LAYER, false, VEC>(a, parts, s);
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
// a.dbias; rstds: [rows] for the roots of long RMS rows; parts: rows of partial sums.
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
