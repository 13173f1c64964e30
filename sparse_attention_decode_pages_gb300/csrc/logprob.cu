// logprob.cu -- log probabilities of given tokens with the entropy of their
// distributions and the most likely alternatives (token_logprobs), in one pass over
// the logits.
//
// With M = max x, d = (x - M) * inv_t, S = sum exp d, T = sum d exp d:
//   lse = M * inv_t + log S,  logprob = (x[target] - M) * inv_t - log S,
//   entropy = log S - T / S        (d is taken from raw logits, so a mask of the type's
//                                   lowest value overflows nothing)
// and M, S, T of two parts of a row join by shifting the smaller M's sums.
//
// A row is cut into parts that fit the registers of one CTA: every thread issues all
// of its 16-byte loads at once and keeps the values, so the exact maximum is known
// before the sums (no running rescale) and the alternatives need no second read.
// The part's K-th largest of the 256 thread maxima bounds its K-th largest logit from
// below; only threads whose maximum reaches that bound scan their values, and the few
// dozen survivors are ranked by counting.  (Should more survive than the list holds --
// rows of equal logits -- the K largest are taken one by one instead.)  The last part
// of a row to finish (an atomic ticket; nothing waits) joins the parts.
#include "common.cuh"
#include "kernels.h"

namespace spd {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpList = 1024;  // survivors a CTA can hold
typedef unsigned long long u64;

// The order of the alternatives as a whole number: the larger logit first (-0 as 0), the
// lower token first among equals; 0 for what is never one (-inf, NaN).
__device__ __forceinline__ unsigned lp_order(float x) {
    return x > __int_as_float(0xff800000) ? float_key(x + 0.f) : 0u;
}

__device__ __forceinline__ u64 lp_key(unsigned order, int i) { return (u64)order << 32 | (0xffffffffu - (unsigned)i); }

__device__ __forceinline__ float lp_key_value(u64 key) {
    const unsigned u = (unsigned)(key >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

template <bool BF16>
__device__ __forceinline__ float lp_at(const void* p, long long i) {
    return BF16 ? __bfloat162float(reinterpret_cast<const bf16*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
}

// Element j of a 16-byte vector.
template <bool BF16>
__device__ __forceinline__ float lp_elem(const uint4& v, int j) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (!BF16) return __uint_as_float(w[j]);
    return __uint_as_float(j & 1 ? w[j >> 1] & 0xffff0000u : w[j >> 1] << 16);
}

__device__ __forceinline__ uint4 lp_load(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

struct LpStat {
    float M, S, T, pad;  // T in base 2: sum of d * log2(e) * exp(d)
};

struct LpPlan {
    int nv;     // 16-byte vectors a thread holds
    int parts;  // of a row
    int vecs;   // of a part
};

// Rows are cut into the largest parts that still give every SM two CTAs, else into
// parts a quarter as large: a single row of 151,936 fp32 logits takes 38 CTAs.
inline LpPlan lp_plan(long long rows, int n, bool bf16, int sms) {
    const int ve = bf16 ? 8 : 4;
    const int nvec = (n + 2 * ve - 2) / ve;  // a row that starts inside a vector touches one more
    LpPlan p;
    p.nv = 16;
    p.parts = (nvec + p.nv * kLpThreads - 1) / (p.nv * kLpThreads);
    if (rows * p.parts < 2LL * sms) {
        p.nv = 4;
        p.parts = (nvec + p.nv * kLpThreads - 1) / (p.nv * kLpThreads);
    }
    p.vecs = (nvec + p.parts - 1) / p.parts;
    return p;
}

struct LpWs {
    int* tickets;  // [rows], zero on entry and on exit
    LpStat* stats;  // [rows][parts]
    u64* keys;      // [rows][parts][top_k]
};

__host__ __device__ inline size_t lp_align(size_t x) { return (x + 255) & ~size_t(255); }

inline size_t lp_ws_layout(void* ws, long long rows, int parts, int top_k, LpWs* w) {
    const size_t o1 = lp_align((size_t)rows * sizeof(int)), o2 = lp_align(o1 + (size_t)rows * parts * sizeof(LpStat));
    if (w) {
        w->tickets = static_cast<int*>(ws);
        w->stats = reinterpret_cast<LpStat*>(static_cast<char*>(ws) + o1);
        w->keys = reinterpret_cast<u64*>(static_cast<char*>(ws) + o2);
    }
    return o2 + (size_t)rows * parts * top_k * sizeof(u64);
}

struct LpShared {
    u64 list[kLpList];
    u64 top[32];
    unsigned tmax[kLpThreads];
    float a[kLpWarps], b[kLpWarps];
    u64 best[kLpWarps];
    int count, flag;
    unsigned bound;
};

// The K largest of the s.count keys of s.list, in order, into s.top (0 where there are
// fewer); the keys differ from one another.
__device__ __forceinline__ void lp_rank(LpShared& s, int K) {
    for (int i = threadIdx.x; i < s.count; i += kLpThreads) {
        const u64 mine = s.list[i];
        int r = 0;
        for (int j = 0; j < s.count; ++j) r += s.list[j] > mine;
        if (r < K) s.top[r] = mine;
    }
}

template <bool BF16, int NV>
__global__ void __launch_bounds__(kLpThreads, NV >= 16 ? 2 : 3) logprob_kernel(const LogprobArgs a, const LpPlan plan, const LpWs w) {
    constexpr int VE = BF16 ? 8 : 4;
    __shared__ LpShared s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x / plan.parts;
    const int part = blockIdx.x % plan.parts;
    const int K = a.top_k;
    const float NEG_INF = __int_as_float(0xff800000);
    const char* rowp = static_cast<const char*>(a.logits) + row * a.row_stride * (BF16 ? 2 : 4);
    const int lead = (int)(reinterpret_cast<uintptr_t>(rowp) & 15) / (BF16 ? 2 : 4);  // elements before the row in its first vector
    const uint4* vecs = reinterpret_cast<const uint4*>(rowp - lead * (BF16 ? 2 : 4));
    const int v0 = part * plan.vecs, v1 = min(v0 + plan.vecs, (lead + a.n + VE - 1) / VE);
    if (tid == 0) s.count = 0;
    if (tid < 32) s.top[tid] = 0ull;
    pdl_wait();
    pdl_trigger();

    // all loads, then the thread's largest value
    uint4 x[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int v = v0 + tid + j * kLpThreads;
        const int i0 = v * VE - lead;  // token of the vector's first element
        constexpr uint32_t kNone = BF16 ? 0xff80ff80u : 0xff800000u;  // -inf
        x[j] = make_uint4(kNone, kNone, kNone, kNone);
        if (v < v1) {
            if (i0 >= 0 && i0 + VE <= a.n) {
                x[j] = lp_load(vecs + v);
            } else {  // a vector that the row fills in part
                uint32_t t[4] = {kNone, kNone, kNone, kNone};
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    if (i0 + e >= 0 && i0 + e < a.n) {
                        if (BF16) {
                            const uint32_t h = reinterpret_cast<const uint16_t*>(rowp)[i0 + e];
                            t[e >> 1] = e & 1 ? (t[e >> 1] & 0xffffu) | h << 16 : (t[e >> 1] & 0xffff0000u) | h;
                        } else {
                            t[e & 3] = reinterpret_cast<const uint32_t*>(rowp)[i0 + e];
                        }
                    }
                x[j] = make_uint4(t[0], t[1], t[2], t[3]);
            }
        }
    }
    float m = NEG_INF;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VE; ++e) m = fmaxf(m, lp_elem<BF16>(x[j], e));
    const unsigned mine = lp_order(m);
    s.tmax[tid] = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane == 0) s.a[warp] = m;
    __syncthreads();
    float M = s.a[0];
#pragma unroll
    for (int i = 1; i < kLpWarps; ++i) M = fmaxf(M, s.a[i]);
    __syncthreads();

    // the bound: the K-th largest thread maximum, its low bits cleared (one warp, a bit at a
    // time from the highest in which the maxima can differ), while the others sum
    if (K > 0 && warp == 0) {
        unsigned t[kLpThreads / 32];
        unsigned lo = 0xffffffffu;
#pragma unroll
        for (int i = 0; i < kLpThreads / 32; ++i) {
            t[i] = s.tmax[lane + 32 * i];
            lo = min(lo, t[i]);
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        const unsigned hi = lp_order(M);
        unsigned bound = 0;
        if (hi != 0) {
            const int top = hi == lo ? 0 : 32 - __clz(hi ^ lo);  // bits that differ: below 2^top
            bound = top >= 32 ? 0u : hi >> top << top;
            for (int bit = top - 1; bit >= max(0, top - 12); --bit) {
                const unsigned cand = bound | 1u << bit;
                int c = 0;
#pragma unroll
                for (int i = 0; i < kLpThreads / 32; ++i) c += t[i] >= cand;
                if ((int)__reduce_add_sync(0xffffffffu, (unsigned)c) >= K) bound = cand;
            }
        }
        if (lane == 0) s.bound = bound;
    }

    const float c2 = a.inv_t * kLog2e;
    const float ref = M == NEG_INF ? 0.f : M;
    float S = 0.f, T = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const float d = (lp_elem<BF16>(x[j], e) - ref) * c2;
            const float p = fast_exp2(d);
            S += p;
            T = fmaf(p, fmaxf(d, -1e30f), T);
        }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        S += __shfl_xor_sync(0xffffffffu, S, off);
        T += __shfl_xor_sync(0xffffffffu, T, off);
    }
    if (lane == 0) {
        s.a[warp] = S;
        s.b[warp] = T;
    }
    __syncthreads();
    S = T = 0.f;
#pragma unroll
    for (int i = 0; i < kLpWarps; ++i) {
        S += s.a[i];
        T += s.b[i];
    }

    if (K > 0) {
        const unsigned bound = max(s.bound, 1u);
        if (mine >= bound) {
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const unsigned o = lp_order(lp_elem<BF16>(x[j], e));
                    if (o >= bound) {
                        const int at = atomicAdd(&s.count, 1);
                        if (at < kLpList) s.list[at] = lp_key(o, (v0 + tid + j * kLpThreads) * VE - lead + e);
                    }
                }
        }
        __syncthreads();
        if (s.count <= kLpList) {
            lp_rank(s, K);
        } else {  // one by one: each the largest below the last
            u64 last = ~0ull;
            for (int k = 0; k < K; ++k) {
                u64 best = 0ull;
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const unsigned o = lp_order(lp_elem<BF16>(x[j], e));
                        const u64 key = lp_key(o, (v0 + tid + j * kLpThreads) * VE - lead + e);
                        if (o != 0 && key < last && key > best) best = key;
                    }
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const u64 y = __shfl_xor_sync(0xffffffffu, best, off);
                    best = y > best ? y : best;
                }
                if (lane == 0) s.best[warp] = best;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < kLpWarps; ++i) best = s.best[i] > best ? s.best[i] : best;
                if (tid == 0) s.top[k] = best;
                last = best;
                __syncthreads();
            }
        }
        __syncthreads();
    }

    if (plan.parts > 1) {
        const long long at = row * plan.parts + part;
        if (tid == 0) *reinterpret_cast<float4*>(w.stats + at) = make_float4(M, S, T, 0.f);
        if (tid < K) w.keys[at * K + tid] = s.top[tid];
        __syncthreads();
        if (tid == 0) {
            fence_acq_rel_gpu();
            const int done = atomic_add_acq_rel(w.tickets + row, 1);
            s.flag = done == plan.parts - 1;
            if (s.flag) w.tickets[row] = 0;
            fence_acq_rel_gpu();
            s.count = 0;
            s.bound = 0;
        }
        __syncthreads();
        if (!s.flag) return;
        // join: every thread takes some parts' sums, relative to the row's maximum
        const float4* st = reinterpret_cast<const float4*>(w.stats + row * plan.parts);
        float mm = NEG_INF;
        for (int p = tid; p < plan.parts; p += kLpThreads) mm = fmaxf(mm, __ldcg(st + p).x);
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, off));
        if (lane == 0) s.a[warp] = mm;
        __syncthreads();
        M = s.a[0];
#pragma unroll
        for (int i = 1; i < kLpWarps; ++i) M = fmaxf(M, s.a[i]);
        __syncthreads();
        S = T = 0.f;
        for (int p = tid; p < plan.parts; p += kLpThreads) {
            const float4 y = __ldcg(st + p);
            if (y.x == NEG_INF) {
                S += y.y;  // 0, or NaN where the part holds one
            } else {
                const float d = (y.x - M) * c2, f = fast_exp2(d);
                S += f * y.y;
                T += f * fmaf(fmaxf(d, -1e30f), y.y, y.z);
            }
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            S += __shfl_xor_sync(0xffffffffu, S, off);
            T += __shfl_xor_sync(0xffffffffu, T, off);
        }
        if (lane == 0) {
            s.a[warp] = S;
            s.b[warp] = T;
        }
        if (tid < 32) s.top[tid] = 0ull;
        const u64* keys = w.keys + row * plan.parts * K;
        if (K > 0) {
            // the K-th key of any part bounds the row's K-th from below
            unsigned bound = 0;
            for (int p = tid; p < plan.parts; p += kLpThreads)
                bound = max(bound, (unsigned)(__ldcg(keys + (long long)p * K + K - 1) >> 32));
            bound = __reduce_max_sync(0xffffffffu, bound);
            if (lane == 0) atomicMax(&s.bound, bound);
        }
        __syncthreads();
        S = T = 0.f;
#pragma unroll
        for (int i = 0; i < kLpWarps; ++i) {
            S += s.a[i];
            T += s.b[i];
        }
        if (K > 0) {
            const unsigned bound = max(s.bound, 1u);
            for (int i = tid; i < plan.parts * K; i += kLpThreads) {
                const u64 key = __ldcg(keys + i);
                if ((unsigned)(key >> 32) >= bound) {
                    const int at = atomicAdd(&s.count, 1);
                    if (at < kLpList) s.list[at] = key;
                }
            }
            __syncthreads();
            if (s.count <= kLpList) {
                lp_rank(s, K);
            } else {
                u64 last = ~0ull;
                for (int k = 0; k < K; ++k) {
                    u64 best = 0ull;
                    for (int i = tid; i < plan.parts * K; i += kLpThreads) {
                        const u64 key = __ldcg(keys + i);
                        if (key < last && key > best) best = key;
                    }
#pragma unroll
                    for (int off = 1; off < 32; off <<= 1) {
                        const u64 y = __shfl_xor_sync(0xffffffffu, best, off);
                        best = y > best ? y : best;
                    }
                    if (lane == 0) s.best[warp] = best;
                    __syncthreads();
#pragma unroll
                    for (int i = 0; i < kLpWarps; ++i) best = s.best[i] > best ? s.best[i] : best;
                    if (tid == 0) s.top[k] = best;
                    last = best;
                    __syncthreads();
                }
            }
            __syncthreads();
        }
    }

    // outputs: S is NaN where the row holds a NaN or +inf; a row with nothing above -inf has S = 0
    const bool empty = S == 0.f;
    const float logS = logf(S);
    const float lse = empty ? NEG_INF : M * a.inv_t + logS;
    if (tid == 0) {
        if (a.logprob) {
            const int t = a.targets[row];
            if (t < -1 || t >= a.n) raise_status(a.status, SPD_DEV_BAD_TOKEN);
            float lp = 0.f;
            if (t >= 0 && t < a.n) lp = empty ? NEG_INF : (lp_at<BF16>(rowp, t) - M) * a.inv_t - logS;
            a.logprob[row] = lp;
        }
        if (a.entropy) a.entropy[row] = empty ? 0.f : logS - kLn2 * (T / S);
        if (a.lse) a.lse[row] = lse;
    }
    if (tid < K) {
        const u64 key = s.top[tid];
        a.top_ids[row * K + tid] = key ? (int)(0xffffffffu - (unsigned)key) : -1;
        a.top_logprobs[row * K + tid] = key ? (lp_key_value(key) - M) * a.inv_t - logS : NEG_INF;
    }
}

size_t token_logprobs_ws(long long rows, int n, int top_k, int num_sms) {
    size_t need = 16;
    for (int bf = 0; bf < 2; ++bf) {
        const LpPlan p = lp_plan(rows, n, bf != 0, num_sms);
        const size_t b = p.parts > 1 ? lp_ws_layout(nullptr, rows, p.parts, top_k, nullptr) : 16;
        need = b > need ? b : need;
    }
    return need;
}

cudaError_t launch_token_logprobs(const LogprobArgs& a, int num_sms, cudaStream_t st) {
    const LpPlan p = lp_plan(a.rows, a.n, a.bf16, num_sms);
    LpWs w;
    lp_ws_layout(a.ws, a.rows, p.parts, a.top_k, &w);
    const dim3 grid((unsigned)(a.rows * p.parts)), block(kLpThreads);
    if (a.bf16)
        return p.nv == 16 ? launch_pdl(logprob_kernel<true, 16>, grid, block, 0, st, a, p, w)
                          : launch_pdl(logprob_kernel<true, 4>, grid, block, 0, st, a, p, w);
    return p.nv == 16 ? launch_pdl(logprob_kernel<false, 16>, grid, block, 0, st, a, p, w)
                      : launch_pdl(logprob_kernel<false, 4>, grid, block, 0, st, a, p, w);
}

}  // namespace spd
