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
// A CTA streams one part of a row, a tile of 256 threads x 4 vectors at a time, the
// next tile's loads in flight while it works on one.  Each thread keeps S and T
// relative to a reference of its own, which moves only when a value exceeds it by
// kLpHead, so nothing is exchanged per tile.  For the alternatives the CTA keeps a
// list of candidates and a bound that at least K values reach: first the K-th largest
// of the 256 thread maxima of the first tile, then, after 2, 4, 8, ... tiles, the K-th
// largest of the list, which is cut to K at the same time; a thread looks at its
// single values only where its tile's maximum reaches the bound.  (Should more values
// pass than the list holds -- ascending rows, rows of equal logits -- the part's K
// largest are taken one by one from memory instead.)  The last part of a row to
// finish (an atomic ticket; nothing waits) joins the parts.
//
// Bound by memory: 448 rows of 151,936 fp32 logits, 8 alternatives: 46.3 us, 5.9 TB/s, 87 % of
// the measured copy peak.  Of bf16 logits 39 us, 52 %: about eight instructions a value (unpacking, maximum,
// difference, exponential, sum, clamp, multiply-add, comparison) for two bytes.  One bf16 row, 20
// alternatives: 9.2 us, the latency of a part's first bound and of the join of 19 parts.  Where the list
// overflows, K passes over the part: 448 rows of equal or ascending fp32 logits, 8 / 32
// alternatives: 1.1 / 2.7 ms, against 47 / 53 us of usual ones (bf16: 0.9 / 2.4 ms, 40 / 49 us).
#include "common.cuh"
#include "kernels.h"

namespace spd {

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpList = 1024;  // survivors a CTA can hold
constexpr int kLpU = 4;        // 16-byte vectors of a thread in a tile
constexpr int kLpTile = kLpThreads * kLpU;
constexpr float kLpHead = 6.f;  // log2 headroom before a thread's reference moves
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
    int parts;  // of a row
    int vecs;   // 16-byte vectors of a part
};

// Parts of a row: the number whose CTAs, run kLpOcc to an SM, take the least time by
// waves * (tiles of a part + kLpFixed).  kLpFixed stands for what a CTA does besides
// streaming (the first bound, the joins), in tiles.  448 rows of 151,936 fp32 logits:
// whole rows, one wave, 46 us; halves, two waves, 57 us; fifths 76 us.  One row: a part
// for each tile.
constexpr int kLpOcc = 3;
constexpr int kLpFixed = 6;

inline LpPlan lp_plan(long long rows, int n, bool bf16, int sms) {
    const int nvec = n / (bf16 ? 8 : 4) + 1;
    const int most = (nvec + kLpTile - 1) / kLpTile;
    const long long slots = (long long)kLpOcc * sms;
    LpPlan p = {1, nvec};
    if (rows > kTickets) return p;  // many times the rows that fill the GPU
    long long best = -1;
    for (int parts = 1; parts <= most; ++parts) {
        const int vecs = (nvec + parts - 1) / parts;
        const long long cost = (rows * parts + slots - 1) / slots * ((vecs + kLpTile - 1) / kLpTile + kLpFixed);
        if (best < 0 || cost < best) {
            best = cost;
            p.parts = parts;
            p.vecs = vecs;
        }
    }
    return p;
}

struct LpWs {
    int* tickets;   // [kTickets], zero on entry and on exit: no call's other data lie on another's
    LpStat* stats;  // [rows][parts]
    u64* keys;      // [rows][parts][top_k]
};

__host__ __device__ inline size_t lp_align(size_t x) { return (x + 255) & ~size_t(255); }

inline size_t lp_ws_layout(void* ws, long long rows, int parts, int top_k, LpWs* w) {
    const size_t o1 = kTicketBytes, o2 = lp_align(o1 + (size_t)rows * parts * sizeof(LpStat));
    if (w) {
        w->tickets = static_cast<int*>(ws) + 4;
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
    int count, flag, over;
    float bound;
    unsigned join_bound;
};

// The K largest of the first n keys of s.list, in order, into s.top (whose entries from
// n on stay as they are); the keys differ from one another.
__device__ __forceinline__ void lp_rank(LpShared& s, int n, int K) {
    for (int i = threadIdx.x; i < n; i += kLpThreads) {
        const u64 mine = s.list[i];
        int r = 0;
        for (int j = 0; j < n; ++j) r += s.list[j] > mine;
        if (r < K) s.top[r] = mine;
    }
}

// Adds a candidate to the list.
__device__ __forceinline__ void lp_push(LpShared& s, float x, int token) {
    const int at = atomicAdd(&s.count, 1);
    if (at < kLpList) s.list[at] = lp_key(lp_order(x), token);
}

// Cuts the list to its K largest and raises the bound to the last of them.  By all threads.
__device__ __forceinline__ void lp_raise(LpShared& s, int K) {
    __syncthreads();
    const int n = min(s.count, kLpList);
    if (n > K) lp_rank(s, n, K);
    __syncthreads();
    if (n > K) {
        if (threadIdx.x < K) s.list[threadIdx.x] = s.top[threadIdx.x];
        if (threadIdx.x == 0) {
            if (s.count > kLpList) s.over = 1;
            s.count = K;
            s.bound = lp_key_value(s.top[K - 1]);
        }
    }
    __syncthreads();
}

// One tile's kept values.
struct LpRegs {
    uint4 x[kLpU];
};

template <bool BF16>
__global__ void __launch_bounds__(kLpThreads, kLpOcc) logprob_kernel(const LogprobArgs a, const LpPlan plan, const LpWs w) {
    constexpr int VE = BF16 ? 8 : 4, SZ = BF16 ? 2 : 4;
    constexpr uint32_t kNone = BF16 ? 0xff80ff80u : 0xff800000u;  // -inf
    __shared__ LpShared s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x / plan.parts;
    const int part = blockIdx.x % plan.parts;
    const int K = a.top_k;
    const float NEG_INF = __int_as_float(0xff800000);
    const char* rowp = static_cast<const char*>(a.logits) + row * a.row_stride * SZ;
    // whole vectors of the row, and the tokens before and behind them
    const int head = min(a.n, (int)((16 - (reinterpret_cast<uintptr_t>(rowp) & 15)) & 15) / SZ);
    const uint4* vecs = reinterpret_cast<const uint4*>(rowp + head * SZ);
    const int nvec = (a.n - head) / VE;
    const int v0 = min(part * plan.vecs, nvec), v1 = part == plan.parts - 1 ? nvec : min(v0 + plan.vecs, nvec);
    if (tid == 0) {
        s.count = 0;
        s.over = 0;
    }
    if (tid < 32) s.top[tid] = 0ull;
    pdl_wait();
    pdl_trigger();

    auto load = [&](int tile) {
        LpRegs r;
#pragma unroll
        for (int j = 0; j < kLpU; ++j) {
            const int v = v0 + tile * kLpTile + tid + j * kLpThreads;
            r.x[j] = v < v1 ? lp_load(vecs + v) : make_uint4(kNone, kNone, kNone, kNone);
        }
        return r;
    };
    const float c2 = a.inv_t * kLog2e;
    float ref = NEG_INF, S = 0.f, T = 0.f;
    // sums of one tile; returns the thread's largest value in it
    auto sums = [&](const LpRegs& r) {
        float m = NEG_INF;
#pragma unroll
        for (int j = 0; j < kLpU; ++j)
#pragma unroll
            for (int e = 0; e < VE; ++e) m = fmaxf(m, lp_elem<BF16>(r.x[j], e));
        if ((m - ref) * c2 > kLpHead || (ref == NEG_INF && m > NEG_INF)) {
            if (ref > NEG_INF) {
                const float d = (ref - m) * c2, f = fast_exp2(d);
                T = f * fmaf(fmaxf(d, -1e30f), S, T);
                S *= f;
            }
            ref = m;
        }
        const float base = ref == NEG_INF ? 0.f : ref;
#pragma unroll
        for (int j = 0; j < kLpU; ++j)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float d = (lp_elem<BF16>(r.x[j], e) - base) * c2;
                const float p = fast_exp2(d);
                S += p;
                T = fmaf(p, fmaxf(d, -1e30f), T);
            }
        return m;
    };
    auto scan = [&](const LpRegs& r, int tile, float bound) {
#pragma unroll
        for (int j = 0; j < kLpU; ++j)
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float x = lp_elem<BF16>(r.x[j], e);
                if (x >= bound) lp_push(s, x, head + (v0 + tile * kLpTile + tid + j * kLpThreads) * VE + e);
            }
    };

    const int tiles = (v1 - v0 + kLpTile - 1) / kLpTile;
    LpRegs cur = load(0);
    // the tokens outside the row's whole vectors: a thread each, of the first and the last part
    float edge = NEG_INF;
    int edge_token = 0;
    {
        const int tail0 = head + nvec * VE;
        if (part == 0 && tid < head) {
            edge_token = tid;
            edge = lp_at<BF16>(rowp, tid);
        } else if (part == plan.parts - 1 && tid >= 32 && tid - 32 < a.n - tail0) {
            edge_token = tail0 + tid - 32;
            edge = lp_at<BF16>(rowp, edge_token);
        }
    }
    // (one loop for the first tile and the others: straight code that runs once costs its fetching)
    int raise = 1;
#pragma unroll 1
    for (int t = 0; t == 0 || t < tiles; ++t) {
        LpRegs next = load(t + 1);
        if (K > 0 && t == raise) {
            lp_raise(s, K);
            raise *= 2;
        }
        const float m = sums(cur);
        if (K > 0) {
            if (t == 0) {
                // the first bound: the K-th largest thread maximum with its low bits cleared, found a
                // bit at a time from the highest in which the maxima differ
                s.tmax[tid] = lp_order(fmaxf(m, edge));
                __syncthreads();
                if (warp == 0) {
                    unsigned v[kLpThreads / 32];
                    unsigned lo = 0xffffffffu, hi = 0;
#pragma unroll
                    for (int i = 0; i < kLpThreads / 32; ++i) {
                        v[i] = s.tmax[lane + 32 * i];
                        lo = min(lo, v[i]);
                        hi = max(hi, v[i]);
                    }
                    lo = __reduce_min_sync(0xffffffffu, lo);
                    hi = __reduce_max_sync(0xffffffffu, hi);
                    const int top = hi == lo ? 0 : 32 - __clz(hi ^ lo);  // the bits that differ lie below 2^top
                    unsigned bound = top >= 32 ? 0u : hi >> top << top;
                    for (int bit = top - 1; bit >= max(0, top - 12); --bit) {
                        const unsigned cand = bound | 1u << bit;
                        int c = 0;
#pragma unroll
                        for (int i = 0; i < kLpThreads / 32; ++i) c += v[i] >= cand;
                        if ((int)__reduce_add_sync(0xffffffffu, (unsigned)c) >= K) bound = cand;
                    }
                    // at least the lowest finite value, so that nothing at -inf passes
                    const unsigned least = float_key(-3.402823466e+38f);
                    if (lane == 0) s.bound = lp_key_value((u64)max(bound, least) << 32);
                }
                __syncthreads();
                if (edge >= s.bound) lp_push(s, edge, edge_token);
            }
            const float bound = s.bound;
            if (m >= bound) scan(cur, t, bound);
        }
        cur = next;
    }
    if (!(edge == NEG_INF)) {  // the thread's single token, NaN too
        const float m = fmaxf(ref, edge);
        // (d bounded as everywhere: f is 0 far above the bound, and 0 times an infinite product would be NaN)
        const float d = ref == NEG_INF ? -1e30f : fmaxf((ref - m) * c2, -1e30f), f = fast_exp2(d);
        const float de = (edge - m) * c2, fe = fast_exp2(de);
        T = fmaf(f, fmaf(d, S, T), fe * fmaxf(de, -1e30f));
        S = fmaf(f, S, fe);
        ref = m;
    }

    // the threads' sums relative to the part's largest reference
    float M = ref;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if (lane == 0) s.a[warp] = M;
    __syncthreads();
    M = s.a[0];
#pragma unroll
    for (int i = 1; i < kLpWarps; ++i) M = fmaxf(M, s.a[i]);
    if (ref > NEG_INF) {
        const float d = (ref - M) * c2, f = fast_exp2(d);
        T = f * fmaf(fmaxf(d, -1e30f), S, T);
        S *= f;
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        S += __shfl_xor_sync(0xffffffffu, S, off);
        T += __shfl_xor_sync(0xffffffffu, T, off);
    }
    __syncthreads();
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
        const int n = s.count;
        if (n <= kLpList && !s.over) {
            lp_rank(s, n, K);
        } else {  // one by one from memory: each the largest below the last
            const int t0 = part == 0 ? 0 : head + v0 * VE, t1 = part == plan.parts - 1 ? a.n : head + v1 * VE;
            u64 last = ~0ull;
            for (int k = 0; k < K; ++k) {
                u64 best = 0ull;
                for (int i = t0 + tid; i < t1; i += kLpThreads) {
                    const unsigned o = lp_order(lp_at<BF16>(rowp, i));
                    const u64 key = lp_key(o, i);
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
            s.join_bound = 0;
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
            // a bound that at least K keys reach: the m-th largest of the parts' j-th keys, m * j >= K
            // (with more parts than threads the largest of their K-th keys)
            if (plan.parts <= kLpThreads) {
                const int j = (K + plan.parts - 1) / plan.parts, m = (K + j - 1) / j;
                if (tid < plan.parts) s.list[tid] = __ldcg(keys + (long long)tid * K + j - 1) & ~0xffffffffull | (unsigned)tid;
                __syncthreads();
                if (tid < plan.parts) {
                    const u64 mine = s.list[tid];
                    int rank = 0;
                    for (int p = 0; p < plan.parts; ++p) rank += s.list[p] > mine;
                    if (rank == m - 1) s.join_bound = (unsigned)(mine >> 32);
                }
            } else {
                unsigned bound = 0;
                for (int p = tid; p < plan.parts; p += kLpThreads)
                    bound = max(bound, (unsigned)(__ldcg(keys + (long long)p * K + K - 1) >> 32));
                bound = __reduce_max_sync(0xffffffffu, bound);
                if (lane == 0) atomicMax(&s.join_bound, bound);
            }
        }
        __syncthreads();
        S = T = 0.f;
#pragma unroll
        for (int i = 0; i < kLpWarps; ++i) {
            S += s.a[i];
            T += s.b[i];
        }
        if (K > 0) {
            const unsigned bound = max(s.join_bound, 1u);
            for (int i = tid; i < plan.parts * K; i += kLpThreads) {
                const u64 key = __ldcg(keys + i);
                if ((unsigned)(key >> 32) >= bound) {
                    const int at = atomicAdd(&s.count, 1);
                    if (at < kLpList) s.list[at] = key;
                }
            }
            __syncthreads();
            if (s.count <= kLpList) {
                lp_rank(s, s.count, K);
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
    return a.bf16 ? launch_pdl(logprob_kernel<true>, grid, block, 0, st, a, p, w)
                  : launch_pdl(logprob_kernel<false>, grid, block, 0, st, a, p, w);
}

}  // namespace spd
