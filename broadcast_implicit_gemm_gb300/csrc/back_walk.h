// back_walk.h -- which unit of the gradients' products (matmul_back.cu) a pair of CTAs
// takes at each turn.
//
// There are long units, 0 to dx - 1, and short ones, dx to dx + dw - 1 (where dw's units
// are the longer ones they come first).  The pairs take the long ones in turn; the `late`
// ones that get one fewer take `ahead` short units each meanwhile, and then all walk the
// rest in turn, the late ones first: each unit goes to the pair that is free first.
//
// No CUDA dependency on the host side, so that a plain C++ test can check it.
#pragma once

#if defined(__CUDACC__)
#define BIGEMM_BW_HD __host__ __device__ __forceinline__
#else
#define BIGEMM_BW_HD inline
#endif

namespace bigemm {

struct BackWalk {
    int dx, dw;                      // long and short units
    int late, ahead;
    int whole, extra;                // long ones of every pair, and pairs that have one more
};

// dx_time, dw_time: a unit's, in the same measure.
BIGEMM_BW_HD BackWalk make_back_walk(int dx, int dw, int pairs, long long dx_time, long long dw_time)
{
    BackWalk w = {dx, dw, 0, 0, dx / pairs, dx % pairs};
    if (dx % pairs) {
        w.late = pairs - dx % pairs;
        const long long fit = dx_time / dw_time, most = dw / w.late;
        w.ahead = (int)(fit < most ? fit : most);
    }
    return w;
}

// The pair's unit of a turn; -1: none left.
BIGEMM_BW_HD int back_unit(const BackWalk &w, int turn, int pair, int pairs)
{
    const int i = turn * pairs + pair;
    if (i < w.dx) return i;
    const int first = pairs - w.late, behind = w.whole + (pair < w.extra ? 1 : 0);
    int j = turn - behind;           // turns since this pair's last dx unit
    int k;
    if (pair >= first && j < w.ahead) {
        k = j * w.late + (pair - first);
    } else if (pair >= first) {
        k = w.ahead * w.late + (j - w.ahead) * pairs + (pair - first);
    } else {
        k = w.ahead * w.late + j * pairs + w.late + pair;
    }
    return k < w.dw ? w.dx + k : -1;
}

}  // namespace bigemm
