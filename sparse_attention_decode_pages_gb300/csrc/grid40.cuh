// grid40.cuh -- probabilities as whole numbers on a 2^-40 grid, whose sums are exact in any
// order, and the exact floor of a random number times such a sum.
#pragma once

#include "common.cuh"

namespace spd {

typedef unsigned long long u64;

// floor(2^40 v) from the float's bits, in integer operations only (a 64-bit
// float-to-integer conversion is a slow instruction): for a normal v < 1,
// v = mant * 2^(E - 150), so 2^40 v = (mant << 40) >> (150 - E), a shift the
// PTX shr clamps to 0 past 64.  v >= 1 (and +inf) counts as 1; v <= 0, NaN and
// subnormals (far below the grid) give 0.
__device__ __forceinline__ u64 fixed40(float v) {
    const unsigned bits = __float_as_uint(v);
    const unsigned E = bits >> 23;  // with the sign bit: negative values give E >= 256
    const u64 x = (u64)((bits & 0x7fffffu) | 0x800000u) << 40;
    u64 w;
    asm("shr.b64 %0, %1, %2;" : "=l"(w) : "l"(x), "r"(150u - E));
    if (E - 1u >= 126u) {  // not a normal value in (0, 1)
        const bool one = E >= 127u && E <= 255u && !(E == 255u && (bits & 0x7fffffu));
        w = one ? (1ull << 40) : 0ull;
    }
    return w;
}

// floor(2^40 v) when it lies below 2^32: v * 2^40 is exact in fp32 (a power-of-two
// scaling that neither overflows nor leaves the normal range for a normal v below 2^-8),
// and the float-to-uint32 conversion truncates it, i.e. floors it.  The conversion
// saturates: 0 for a negative v or a NaN (as fixed40), 2^32 - 1 for a v of 2^-8 or more
// or +inf, so a result below 2^30 is always the exact floor(2^40 v).
__device__ __forceinline__ unsigned fixed40_u32(float v) { return __float2uint_rz(v * 1099511627776.0f); }

// floor(u * total) for a float u in [0, 1), exactly: u = m * 2^-shift
__device__ __forceinline__ u64 scaled_floor(float u, u64 total) {
    const unsigned bits = __float_as_uint(u);
    const unsigned E = (bits >> 23) & 0xffu;
    u64 m;
    int shift;
    if (E == 0) {
        m = bits & 0x7fffffu;
        shift = 149;
    } else {
        m = (bits & 0x7fffffu) | 0x800000u;
        shift = 150 - (int)E;
    }
    if (shift <= 0) return ~0ull;  // u >= 2^23: past any total
    const u64 lo = m * total, hi = __umul64hi(m, total);
    if (shift >= 128) return 0ull;
    if (shift >= 64) return hi >> (shift - 64);
    return (lo >> shift) | (hi << (64 - shift));
}

}  // namespace spd
