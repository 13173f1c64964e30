// attn4.cuh -- what the two kernels of attention over the 4-bit cache share: constants of
// their softmax, the queries' scaling, and the join of a row's splits.
#pragma once

#include "kernels.h"
#include "kv4.cuh"

namespace spd {

// Online softmax in fp32 in base 2.  A row's reference moves only when a logit exceeds it by
// kHead4, and weights carry a factor 2^kBias4, so that what fp16 drops of a weight lies
// 2^-32 below the reference and the largest weight, 2^(kHead4 + kBias4), is within fp16.
constexpr float kHead4 = 8.f, kBias4 = 7.f;
constexpr float kMost4 = 32768.f;   // 2^(kHead4 + kBias4)
constexpr float kLow4 = -3.0e38f;   // a row's reference before its first visible token

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// The exponent e of a query row, its lanes' largest magnitudes given: 2^-e brings the row's
// largest channel into [1, 2), so that fp16 keeps its channels to 2^-25 of that.
__device__ __forceinline__ int query_exponent(float amax) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    const int e = (int)(__float_as_uint(amax) >> 23) - 127;
    return amax == 0.f ? 0 : e > 126 ? 126 : e < -126 ? -126 : e;
}

// A CTA whose wait ran out still waits for its own copies and products in flight, whatever limit
// the caller has set: the memory that they write is another CTA's after it.
__device__ __forceinline__ unsigned long long drain_limit(const Attn4Args& a) {
    return a.wait_ns > 2000000000ull ? a.wait_ns : 2000000000ull;
}

// Called by every thread of the CTA behind its partials' stores: whether this was the last of the
// row's nsplit units to finish (its ticket is then reset for the next call).
__device__ __forceinline__ bool last_split(const Attn4Args& a, int row, int nsplit, int* s_last) {
    __syncthreads();
    if (threadIdx.x == 0) {
        fence_acq_rel_gpu();
        const int done = atomic_add_acq_rel(a.counters + row, 1);
        *s_last = done == nsplit - 1;
        if (*s_last) a.counters[row] = 0;
        fence_acq_rel_gpu();
    }
    __syncthreads();
    return *s_last != 0;
}

// The R query rows of a row from its nsplit partials, by the log-sum-exp rule: sixteen
// partials' loads in flight at a time, the sums rescaled when a group's maximum is larger
// (76 partials one after the other took 13 us).
template <int D, int THREADS, typename OutIndex>
__device__ __forceinline__ void join_splits(const Attn4Args& a, int row, int nsplit, int R, OutIndex out_index) {
    constexpr int BATCH = 16;
    const float NEG_INF = __int_as_float(0xff800000);
    for (int i = threadIdx.x; i < R * (D / 4); i += THREADS) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        const long long at = (long long)row * a.num_splits * R + r;
        float top = NEG_INF, sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < nsplit; k0 += BATCH) {
            float pl[BATCH];
            float4 x[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                pl[k] = NEG_INF;
                x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + k < nsplit) {
                    pl[k] = __ldcg(a.part_lse + at + (long long)(k0 + k) * R);
                    x[k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + (at + (long long)(k0 + k) * R) * D + d));
                }
            }
            float m = top;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) m = fmaxf(m, pl[k]);
            const float f = top == NEG_INF ? 0.f : fast_exp2((top - m) * kLog2e);
            sum *= f;
            o.x *= f;
            o.y *= f;
            o.z *= f;
            o.w *= f;
            top = m;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const float w = pl[k] == NEG_INF ? 0.f : fast_exp2((pl[k] - top) * kLog2e);
                sum += w;
                o.x = fmaf(w, x[k].x, o.x);
                o.y = fmaf(w, x[k].y, o.y);
                o.z = fmaf(w, x[k].z, o.z);
                o.w = fmaf(w, x[k].w, o.w);
            }
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const long long oi = out_index(r);
        *reinterpret_cast<uint2*>(a.o + oi * D + d) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (d == 0 && a.lse) a.lse[oi] = sum == 0.f ? NEG_INF : top + log2f(sum) * kLn2;
    }
}

}  // namespace spd
