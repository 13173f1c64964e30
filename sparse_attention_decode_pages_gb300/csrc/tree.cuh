// tree.cuh -- which nodes of a tree of drafted tokens a node sees.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace spd {

// By one warp: bits of node v and its ancestors, or 0 for what is no node, from parents [T], T <= 64, for nodes
// v = lane (m[0]) and v = lane + 32 (m[1]); the paths double six times.  False where a parent is
// out of range.
__device__ __forceinline__ bool tree_masks(const int32_t* parents, int T, unsigned long long (&m)[2]) {
    const int lane = threadIdx.x & 31;
    int up[2];
    bool gone[2], bad = false;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int v = lane + 32 * i, p = v < T ? parents[v] : -2;
        m[i] = 1ull << v;
        up[i] = p >= 0 && p < v ? p : -1;
        gone[i] = p < -1 || p >= v;
        bad |= p < -2 || p >= v;
    }
#pragma unroll
    for (int step = 0; step < 6; ++step) {
        unsigned long long m2[2];
        int up2[2];
        bool gone2[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // both nodes' values before either changes
            const int at = up[i] < 0 ? 0 : up[i];
            const unsigned long long ma = __shfl_sync(0xffffffffu, m[0], at & 31), mb = __shfl_sync(0xffffffffu, m[1], at & 31);
            const int ua = __shfl_sync(0xffffffffu, up[0], at & 31), ub = __shfl_sync(0xffffffffu, up[1], at & 31);
            const bool ga = __shfl_sync(0xffffffffu, (int)gone[0], at & 31), gb = __shfl_sync(0xffffffffu, (int)gone[1], at & 31);
            m2[i] = at < 32 ? ma : mb;
            up2[i] = at < 32 ? ua : ub;
            gone2[i] = at < 32 ? ga : gb;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (up[i] >= 0) {
                m[i] |= m2[i];
                gone[i] |= gone2[i];
                up[i] = up2[i];
            }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) m[i] = gone[i] ? 0ull : m[i];
    return !__any_sync(0xffffffffu, bad);
}

}  // namespace spd
