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

// floor(u * total) for a float u >= 0, exactly: u = m * 2^-shift.  2^64 and more: 2^64 - 1, past any total.
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
    if (hi >> shift) return ~0ull;
    return (lo >> shift) | (hi << (64 - shift));
}

// Sums of floor(2^40 v) of many values of any size, at four multiply-adds for two of them and no conversion:
// with t = v 2^20 + 2^23 rounded towards zero, t - 2^23 is floor(2^20 v) and also lies in t's low bits; what it leaves of
// v is exact, and its next 20 bits are found the same way.  Values above 1 count as 1, negative ones and NaN as
// 0.  take() is good for 4,095 values before total() (4,096 ones are 2^32).
struct GridSum {
    unsigned hi = 0, lo = 0, n = 0;
    __device__ __forceinline__ void take(float2 v) {
        v.x = fminf(fmaxf(v.x, 0.f), 1.f);
        v.y = fminf(fmaxf(v.y, 0.f), 1.f);
        const float2 one = make_float2(8388608.f, 8388608.f);  // 2^23
        const float2 t = fma2_rz(v, make_float2(1048576.f, 1048576.f), one);
        const float2 h = add2(t, make_float2(-8388608.f, -8388608.f));
        const float2 r = fma2(h, make_float2(-9.5367431640625e-7f, -9.5367431640625e-7f), v);  // - 2^-20 h: exact
        const float2 l = fma2_rz(r, make_float2(1099511627776.f, 1099511627776.f), one);
        hi += __float_as_uint(t.x) + __float_as_uint(t.y);
        lo += __float_as_uint(l.x) + __float_as_uint(l.y);
        n += 2;
    }
    __device__ __forceinline__ u64 total() const {  // (2^23's bits are 0x4b000000; the differences fit 32 bits)
        return ((u64)(hi - n * 0x4b000000u) << 20) + (lo - n * 0x4b000000u);
    }
};

}  // namespace spd
