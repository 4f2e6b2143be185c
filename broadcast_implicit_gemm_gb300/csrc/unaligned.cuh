// unaligned.cuh -- 16 bytes of a row that does not start on a 16-byte boundary,
// in two aligned 16-byte loads and a shift.  Nothing outside the matrix's span
// (its first row's first byte to its last row's last) is read: the one or two
// pieces whose aligned words would reach past it go byte by byte.  What the
// words hold of neighbouring rows is masked off.
#pragma once
#include <cstdint>

namespace bigemm {

struct Span {
    const uint8_t *begin, *end;
};

// A piece as loaded; its bytes start at byte `by` of the words.
struct Wide {
    uint4 a, b;
    uint32_t by;
};

// Bytes first .. last - 1 (0 <= first, last <= 16) of the 16 at `at` lie in the
// row; the loads' results are not touched here, so that several are in flight.
__device__ __forceinline__ Wide wide_load(const uint8_t *at, int first, int last, const Span &s)
{
    Wide w;
    w.a = w.b = make_uint4(0, 0, 0, 0);
    w.by = 0;
    if (first >= last) return w;
    const uintptr_t p = reinterpret_cast<uintptr_t>(at);
    const uint8_t *lo = reinterpret_cast<const uint8_t *>(p & ~(uintptr_t)15);
    const int by = (int)(p & 15);
    const bool need_a = by + first < 16, need_b = by + last > 16;
    if ((!need_a || lo >= s.begin) && (need_a || lo + 16 >= s.begin) && (!need_b || lo + 32 <= s.end) &&
        (need_b || lo + 16 <= s.end)) {
        w.by = (uint32_t)by;
        if (need_a) w.a = *reinterpret_cast<const uint4 *>(lo);
        if (need_b) w.b = *reinterpret_cast<const uint4 *>(lo + 16);
    } else {
        uint32_t q[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i >= first && i < last) q[i >> 2] |= (uint32_t)at[i] << (8 * (i & 3));
        w.a = make_uint4(q[0], q[1], q[2], q[3]);
    }
    return w;
}

__device__ __forceinline__ uint32_t keep_bytes(uint32_t v, int first, int last)   // of a word's four
{
    const uint32_t lo = first <= 0 ? 0xffffffffu : first >= 4 ? 0u : 0xffffffffu << (8 * first);
    const uint32_t hi = last >= 4 ? 0xffffffffu : last <= 0 ? 0u : 0xffffffffu >> (8 * (4 - last));
    return v & lo & hi;
}

// The 16 bytes, zeros outside first .. last - 1.
__device__ __forceinline__ uint4 wide_take(const Wide &w, int first, int last)
{
    uint32_t q[8] = {w.a.x, w.a.y, w.a.z, w.a.w, w.b.x, w.b.y, w.b.z, w.b.w};
    if (w.by & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) q[i] = q[i + 2];
    }
    if (w.by & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) q[i] = q[i + 1];
    }
    const uint32_t sh = (w.by & 3) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = __funnelshift_r(q[i], q[i + 1], sh);
    if (first > 0 || last < 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = keep_bytes(q[i], first - 4 * i, last - 4 * i);
    }
    return make_uint4(q[0], q[1], q[2], q[3]);
}

}  // namespace bigemm
