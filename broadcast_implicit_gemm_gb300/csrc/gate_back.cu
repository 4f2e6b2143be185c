// gate_back.cu -- the elementwise part of a gated layer's gradients (matmul_back.cuh):
//
//   d_g = dout u act'(g),  d_u = dout act(g)
//
// rounded once to the operands' type, which is what the tensor core takes (a separate
// multiplication would round them too; two 16-bit parts of each would keep 22 bits for
// twice the products, which take 1.2 of 1.4 ms of 4096 x 4096 -> 16384.  dx and dw are off by 0.0024
// in the 2-norm so, bf16, by 0.0017 with unrounded ones), and their sums over the tokens,
// of the fp32 values before that.  Bound by memory: 10 bytes per element of 16-bit matrices.  A
// warp takes 256 columns, 8 a lane, of every eighth row of its block's run, so that a
// lane's sums stay in registers; two rows' loads are in flight.
#include "column_sums.cuh"
#include "matmul_back.cuh"
#include "norm.cuh"

namespace bigemm {

namespace {

// act(z) and its slope.  With p = 1 / (1 + 2^-t):
//   silu  z p,     p (1 + z (1 - p))
//   gelu  z Phi,   Phi + z phi                      (Phi as in mm_gelu)
//   tanh  z p,     p + z p (1 - p) t'(z) / log2(e),  t as in mm_act
template <int ACT>
__device__ __forceinline__ void act_slope(float z, float &a, float &s)
{
    constexpr float kLog2e = 1.4426950408889634f;
    a = z, s = 1.f;
    if (ACT == BIGEMM_ACT_RELU) a = z < 0.f ? 0.f : z, s = z > 0.f ? 1.f : 0.f;
    if (ACT == BIGEMM_ACT_GELU) {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * z * (-0.5f * kLog2e)));
        const float p = mm_normal_below(z, e);
        a = z * p;
        s = fmaf(z * e, 0.39894228040143268f, p);
    }
    if (ACT == BIGEMM_ACT_GELU_TANH) {
        constexpr float c = 2.f * 0.79788456080286536f;      // 2 sqrt(2/pi)
        const float p = mm_sigmoid2(1.f, z * (c * kLog2e + c * kLog2e * 0.044715f * (z * z)));
        // p (1 - p) is 0 long before z^2 = 400, and z^2 may overflow
        const float zz = fminf(z * z, 400.f);
        a = z * p;
        s = fmaf(z * p * (1.f - p), c + c * 3.f * 0.044715f * zz, p);
    }
    if (ACT == BIGEMM_ACT_SILU) {
        const float p = mm_sigmoid2(1.f, kLog2e * z);
        a = z * p;
        s = p * fmaf(z, 1.f - p, 1.f);
    }
}

template <int ACT>
__device__ __forceinline__ void slopes(const float (&d)[kPiece], float (&g)[kPiece], float (&u)[kPiece])
{
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
        float a, s;
        act_slope<ACT>(g[i], a, s);
        g[i] = d[i] * u[i] * s;
        u[i] = d[i] * a;
    }
}

// g and u become d_g and d_u.
__device__ __forceinline__ void slopes_of(int act, const float (&d)[kPiece], float (&g)[kPiece], float (&u)[kPiece])
{
    switch (act) {
    case BIGEMM_ACT_RELU: slopes<BIGEMM_ACT_RELU>(d, g, u); break;
    case BIGEMM_ACT_GELU: slopes<BIGEMM_ACT_GELU>(d, g, u); break;
    case BIGEMM_ACT_GELU_TANH: slopes<BIGEMM_ACT_GELU_TANH>(d, g, u); break;
    case BIGEMM_ACT_SILU: slopes<BIGEMM_ACT_SILU>(d, g, u); break;
    default: slopes<BIGEMM_ACT_NONE>(d, g, u); break;
    }
}

// A lane's 8 of a block's 256 columns: consecutive ones on the 16-byte grid; off it one
// of each 32, so that a warp's plain loads cover consecutive elements (lanes with 8
// consecutive ones, in two aligned loads and a shift: 777 x 5001 f16 gelu 27 us; with
// pairs 18).
template <bool VEC>
__device__ __forceinline__ int gate_column(int lane, int i) { return VEC ? lane * kPiece + i : i * 32 + lane; }

template <typename T, bool VEC>
struct GateRaw {
    std::conditional_t<VEC, Raw<T>, T[kPiece]> d;

    __device__ __forceinline__ void load(const T *row, int c0, int lane, int cols)
    {
        if constexpr (VEC) {
            const int c = c0 + lane * kPiece;
            if (c + kPiece <= cols) {
                d.q[0] = *reinterpret_cast<const uint4 *>(row + c);
                return;
            }
            T *e = reinterpret_cast<T *>(&d);
#pragma unroll
            for (int i = 0; i < kPiece; ++i) e[i] = c + i < cols ? row[c + i] : from_f32<T>(0.f);
        } else {
            const T *e = row + c0 + lane;
#pragma unroll
            for (int i = 0; i < kPiece; ++i) d[i] = c0 + i * 32 + lane < cols ? e[i * 32] : from_f32<T>(0.f);
        }
    }
    __device__ __forceinline__ void values(float (&v)[kPiece]) const
    {
        if constexpr (VEC) {
            unpack<T>(d, v);
        } else {
#pragma unroll
            for (int i = 0; i < kPiece; ++i) v[i] = to_f32<T>(d[i]);
        }
    }
};

// Rows of d_g and d_u start on the 16-byte grid.
template <typename T, bool VEC>
__device__ __forceinline__ void gate_store(T *row, int c0, int lane, int cols, const float (&v)[kPiece])
{
    if constexpr (VEC) {
        store_piece<T, true>(row, c0 + lane * kPiece, cols, v);
    } else {
        T *e = row + c0 + lane;
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (c0 + i * 32 + lane < cols) e[i * 32] = from_f32<T>(v[i]);
    }
}

// GATED: d_g and d_u; SUMS: the sums over the run's rows (else of dout alone).
template <typename T, bool VEC, bool GATED, bool SUMS>
__global__ void __launch_bounds__(256, kGateBeside(VEC)) gate_back_kernel(const GateBackArgs a)
{
    griddep_enter();
    static_assert(GATED || SUMS, "something to do");
    __shared__ float total[SUMS ? (GATED ? 2 : 1) * 8 * kGateColumns : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = (int)blockIdx.x * kGateColumns;
    const long long r0 = (long long)a.M * blockIdx.y / a.runs, r1 = (long long)a.M * (blockIdx.y + 1) / a.runs;
    const T *dout = static_cast<const T *>(a.dout), *gate = static_cast<const T *>(a.gate), *up = static_cast<const T *>(a.up);
    float sg[SUMS ? kPiece : 1], su[SUMS && GATED ? kPiece : 1];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) sg[SUMS ? i : 0] = 0.f, su[SUMS && GATED ? i : 0] = 0.f;
    constexpr int U = !GATED ? (VEC ? 8 : 4) : VEC ? 2 : 1;       // rows whose loads leave together
    for (long long r = r0 + warp; r < r1; r += 8 * U) {
        GateRaw<T, VEC> d[U], g[GATED ? U : 1], u[GATED ? U : 1];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const long long row = r + 8 * k;
            if (row >= r1) break;
            d[k].load(dout + row * a.ldd, c0, lane, a.N);
            if (GATED) {
                g[GATED ? k : 0].load(gate + row * a.ldg, c0, lane, a.N);
                u[GATED ? k : 0].load(up + row * a.ldu, c0, lane, a.N);
            }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const long long row = r + 8 * k;
            if (row >= r1) break;
            float dv[kPiece];
            d[k].values(dv);
            if constexpr (GATED) {
                float gv[kPiece], uv[kPiece];
                g[k].values(gv);
                u[k].values(uv);
                slopes_of(a.act, dv, gv, uv);
                gate_store<T, VEC>(static_cast<T *>(a.dg) + row * a.pitch, c0, lane, a.N, gv);
                gate_store<T, VEC>(static_cast<T *>(a.du) + row * a.pitch, c0, lane, a.N, uv);
                if (SUMS) {
#pragma unroll
                    for (int i = 0; i < kPiece; ++i) sg[SUMS ? i : 0] += gv[i], su[SUMS ? i : 0] += uv[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < kPiece; ++i) sg[SUMS ? i : 0] += dv[i];
            }
        }
    }
    if constexpr (SUMS) {
        // a thread adds what one lane of each warp has of one of its columns
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
            total[warp * kGateColumns + i * 32 + lane] = sg[i];
            if constexpr (GATED) total[(8 + warp) * kGateColumns + i * 32 + lane] = su[i];
        }
        __syncthreads();
        const int i = (int)threadIdx.x >> 5, col = c0 + gate_column<VEC>(lane, i);
        if (col >= a.N) return;
#pragma unroll
        for (int o = 0; o < (GATED ? 2 : 1); ++o) {
            if (!a.sums[o]) continue;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) v += total[(o * 8 + w) * kGateColumns + i * 32 + lane];
            a.sums[o][blockIdx.y * sum_pitch(a.N) + col] = v;
        }
    }
}

template <typename T, bool VEC>
cudaError_t launch_gate_type(const GateBackArgs &a, cudaStream_t s)
{
    const dim3 grid((unsigned)((a.N + kGateColumns - 1ll) / kGateColumns), (unsigned)a.runs), block(256);
    if (a.act < 0) return launch_pdl(gate_back_kernel<T, VEC, false, true>, grid, block, 0, s, a);
    return a.sums[0] || a.sums[1] ? launch_pdl(gate_back_kernel<T, VEC, true, true>, grid, block, 0, s, a)
                                  : launch_pdl(gate_back_kernel<T, VEC, true, false>, grid, block, 0, s, a);
}

}  // namespace

cudaError_t launch_gate_back(const GateBackArgs &a, int dt, bool vec, cudaStream_t stream)
{
    ProfScope prof("gate_back", stream);
    if (dt == BIGEMM_F16) return vec ? launch_gate_type<__half, true>(a, stream) : launch_gate_type<__half, false>(a, stream);
    return vec ? launch_gate_type<__nv_bfloat16, true>(a, stream) : launch_gate_type<__nv_bfloat16, false>(a, stream);
}

}  // namespace bigemm
