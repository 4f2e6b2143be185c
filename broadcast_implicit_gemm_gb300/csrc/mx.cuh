// mx.cuh -- MXFP8: e4m3 elements with one power-of-two scale per 32 elements
// of a row, shared by the kernels that write it (norm.cu, the matrix products).
//
// The scale of a group is the smallest power of two s with amax <= 448 s (448
// is e4m3's largest value), so no element saturates; it is stored as the byte
// code with s = 2^(code - 127) (E8M0).  A group that holds a NaN or an infinity
// gets code 255, E8M0's NaN, and NaN elements.
#pragma once
#include <cstdint>
#include <cuda_fp8.h>

#include "mx_layout.h"

namespace bigemm {

// The scale's code from a group's largest magnitude: its exponent less 8, one
// more where the fraction exceeds 448's (1.75, fraction bits 0x600000: adding
// 0x1fffff then carries into the exponent); at least 0 (2^-127).
__device__ __forceinline__ uint32_t mx_scale_code(float amax)
{
    const uint32_t b = __float_as_uint(amax);
    const int code = max((int)((b + 0x1fffffu) >> 23) - 8, 0);
    return b >= 0x7f800000u ? 255u : (uint32_t)code;
}

// 1 / s = 2^(127 - code), exact (codes of finite groups are at most 248); NaN
// for 255.
__device__ __forceinline__ float mx_inv_scale(uint32_t code)
{
    return __uint_as_float(code == 255u ? 0x7fffffffu : (254u - code) << 23);
}

// The largest magnitude of two values, NaN if either is.
__device__ __forceinline__ float mx_amax(float a, float b)
{
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(fabsf(a)), "f"(fabsf(b)));
    return m;
}

// Four floats, already divided by the scale, as e4m3 (nearest even), the first
// in the low byte.
__device__ __forceinline__ uint32_t mx_pack4(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

}  // namespace bigemm
