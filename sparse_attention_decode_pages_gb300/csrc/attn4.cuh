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
// n to take this ticket (which is then reset for the next call).
__device__ __forceinline__ bool last_of(int* ticket, int n, int* s_last) {
    __syncthreads();
    if (threadIdx.x == 0) {
        fence_acq_rel_gpu();
        const int done = atomic_add_acq_rel(ticket, 1);
        *s_last = done == n - 1;
        if (*s_last) *ticket = 0;
        fence_acq_rel_gpu();
    }
    __syncthreads();
    return *s_last != 0;
}

// The R query rows of a row from n partials, the first at `first`, by the log-sum-exp rule,
// sink(r, d, o, lse): BATCH partials' loads in flight at a time, the sums rescaled when a batch's
// maximum is larger (76 partials one after the other took 13 us).
template <int D, int THREADS, int BATCH, typename Sink>
__device__ __forceinline__ void join_parts(const Attn4Args& a, long long first, int n, int R, Sink sink) {
    const float NEG_INF = __int_as_float(0xff800000);
    for (int i = threadIdx.x; i < R * (D / 4); i += THREADS) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        const long long at = first * R + r;
        float top = NEG_INF, sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < n; k0 += BATCH) {
            float pl[BATCH];
            float4 x[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                pl[k] = NEG_INF;
                x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k0 + k < n) {
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
        sink(r, d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv), sum == 0.f ? NEG_INF : top + log2f(sum) * kLn2);
    }
}

// The output row of query row r of a row (sequence b, KV head h).
__device__ __forceinline__ long long output_row(const Attn4Args& a, int b, int h, int r) {
    const int G = a.H_q / a.H_kv, t = r / G;
    return ((long long)b * a.T + t) * a.H_q + h * G + (r - t * G);
}

// The join in two steps: the last unit of each group joins the group, beside the others, and the
// last group the groups.
template <int D, int THREADS, int BATCH>
__device__ __forceinline__ void join_groups(const Attn4Args& a, int row, int split, int nsplit, int R, int* s_last) {
    const long long base = (long long)row * a.parts;
    const int group = split / a.group, b = row / a.H_kv, h = row - b * a.H_kv;
    // (one loop for the two steps: code that runs once costs its fetching)
#pragma unroll 1
    for (int step = 0; step < 2; ++step) {
        const long long first = base + (step == 0 ? group * a.group : a.num_splits);
        const int n = step == 0 ? min(a.group, nsplit - group * a.group) : (nsplit + a.group - 1) / a.group;
        if (!last_of(a.counters + (step == 0 ? a.B * a.H_kv + row * (a.parts - a.num_splits) + group : row), n, s_last)) return;
        join_parts<D, THREADS, BATCH>(a, first, n, R, [&](int r, int d, const float4& o, float lse) {
            if (step == 0) {
                const long long at = (base + a.num_splits + group) * R + r;
                *reinterpret_cast<float4*>(a.part_o + at * D + d) = o;
                if (d == 0) a.part_lse[at] = lse;
            } else {
                const long long oi = output_row(a, b, h, r);
                *reinterpret_cast<uint2*>(a.o + oi * D + d) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
                if (d == 0 && a.lse) a.lse[oi] = lse;
            }
        });
    }
}

template <int D, int THREADS>
__device__ __noinline__ void join_groups_apart(const Attn4Args& a, int row, int split, int nsplit, int R, int* s_last) {
    join_groups<D, THREADS, 8>(a, row, split, nsplit, R, s_last);  // (16 spill: 96 -> 136 us for 304 splits of 64 rows)
}

// A unit's end: the last of a row's nsplit units joins them, or, where that would be much for one
// CTA, they are joined in groups.  APART: by code apart from the kernel's (within it, it costs the
// verification registers that it spills, 334 -> 345 us where nothing is joined in groups; the
// decode kernel has them, and is 5 us faster for one KV head's 131,072 tokens).
template <int D, int THREADS, bool APART, typename OutIndex>
__device__ __forceinline__ void join_splits(const Attn4Args& a, int row, int split, int nsplit, int R, int* s_last,
                                            OutIndex out_index) {
    if (nsplit == 1) return;
    if (nsplit > a.group) {
        if constexpr (APART) join_groups_apart<D, THREADS>(a, row, split, nsplit, R, s_last);
        else join_groups<D, THREADS, 16>(a, row, split, nsplit, R, s_last);
        return;
    }
    if (!last_of(a.counters + row, nsplit, s_last)) return;
    join_parts<D, THREADS, 16>(a, (long long)row * a.parts, nsplit, R, [&](int r, int d, const float4& o, float lse) {
        const long long oi = out_index(r);
        *reinterpret_cast<uint2*>(a.o + oi * D + d) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
        if (d == 0 && a.lse) a.lse[oi] = lse;
    });
}

}  // namespace spd
