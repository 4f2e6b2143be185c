// gate_back.cu -- the elementwise part of a gated layer's gradients (matmul_back.cuh):
//
//   d_g = dout u act'(g),  d_u = dout act(g)
//
// rounded once to the operands' type, which is what the tensor core takes (a separate
// multiplication would round them too), and their sums over the tokens, of the fp32
// values before that.  Bound by memory: 10 bytes per element of 16-bit matrices.  A
// warp takes 256 columns, 8 a lane, of every eighth row of its block's run, so that a
// lane's sums stay in registers; two rows' loads are in flight.
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

// GATED: d_g and d_u; SUMS: the sums over the run's rows (else of dout alone).
template <typename T, bool VEC, bool GATED, bool SUMS>
__global__ void __launch_bounds__(256) gate_back_kernel(const GateBackArgs a)
{
    griddep_enter();
    static_assert(GATED || SUMS, "something to do");
    __shared__ float total[SUMS ? (GATED ? 2 : 1) * 8 * kGateColumns : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = ((int)blockIdx.x * 32 + lane) * kPiece;
    const long long r0 = (long long)a.M * blockIdx.y / a.runs, r1 = (long long)a.M * (blockIdx.y + 1) / a.runs;
    const Span d_span = span_of(a.dout, a.M, a.ldd, a.N, sizeof(T));
    const Span g_span = GATED ? span_of(a.gate, a.M, a.ldg, a.N, sizeof(T)) : d_span;
    const Span u_span = GATED ? span_of(a.up, a.M, a.ldu, a.N, sizeof(T)) : d_span;
    float sg[SUMS ? kPiece : 1], su[SUMS && GATED ? kPiece : 1];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) sg[SUMS ? i : 0] = 0.f, su[SUMS && GATED ? i : 0] = 0.f;
    if (c < a.N) {
        constexpr int U = 2;
        for (long long r = r0 + warp; r < r1; r += 8 * U) {
            Held<T, VEC> d[U], g[GATED ? U : 1], u[GATED ? U : 1];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const long long row = r + 8 * k;
                if (row >= r1) break;
                hold<T, VEC>(static_cast<const T *>(a.dout) + row * a.ldd, c, a.N, d_span, d[k]);
                if (GATED) {
                    hold<T, VEC>(static_cast<const T *>(a.gate) + row * a.ldg, c, a.N, g_span, g[GATED ? k : 0]);
                    hold<T, VEC>(static_cast<const T *>(a.up) + row * a.ldu, c, a.N, u_span, u[GATED ? k : 0]);
                }
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const long long row = r + 8 * k;
                if (row >= r1) break;
                float dv[kPiece];
                take<T, VEC>(d[k], c, a.N, dv);
                if constexpr (GATED) {
                    float gv[kPiece], uv[kPiece];
                    take<T, VEC>(g[k], c, a.N, gv);
                    take<T, VEC>(u[k], c, a.N, uv);
                    slopes_of(a.act, dv, gv, uv);
                    store_piece<T, true>(static_cast<T *>(a.dg) + row * a.pitch, c, a.N, gv);
                    store_piece<T, true>(static_cast<T *>(a.du) + row * a.pitch, c, a.N, uv);
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
    }
    if constexpr (SUMS) {
#pragma unroll
        for (int i = 0; i < kPiece; ++i) {
            total[warp * kGateColumns + i * 32 + lane] = sg[i];
            if constexpr (GATED) total[(8 + warp) * kGateColumns + i * 32 + lane] = su[i];
        }
        __syncthreads();
        // a thread a column: column 8 l + i of the block is at i * 32 + l
        const int l = (int)threadIdx.x >> 3, i = (int)threadIdx.x & 7, col = (int)blockIdx.x * kGateColumns + (int)threadIdx.x;
        if (col >= a.N) return;
#pragma unroll
        for (int o = 0; o < (GATED ? 2 : 1); ++o) {
            if (!a.sums[o]) continue;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) v += total[(o * 8 + w) * kGateColumns + i * 32 + l];
            a.sums[o][(long long)blockIdx.y * a.N + col] = v;
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
