// logprob.cu -- log probabilities of given tokens with the entropy of their
// distributions and the most likely alternatives (token_logprobs).
//
//   z = inv_t * x,  lse = log sum exp z,  logprob = z[target] - lse,
//   entropy = lse - sum p z = log S - T / S,  S = sum exp(z - m),  T = sum (z - m) exp(z - m)
//
// One CTA per row: the maximum, then S and T, then one pass for each alternative.
#include "common.cuh"
#include "kernels.h"

namespace spd {

constexpr int kLogprobThreads = 512;
typedef unsigned long long u64;

__device__ __forceinline__ float lp_value(const LogprobArgs& a, long long at) {
    return a.bf16 ? __bfloat162float(reinterpret_cast<const bf16*>(a.logits)[at])
                  : reinterpret_cast<const float*>(a.logits)[at];
}

// A whole number in the order of the alternatives: the larger logit first, the lower
// token first among equals; 0 for a logit that is never one (-inf, NaN).
__device__ __forceinline__ u64 lp_key(float x, int i) {
    if (!(x > __int_as_float(0xff800000))) return 0ull;
    return (u64)float_key(x + 0.f) << 32 | (0xffffffffu - (unsigned)i);
}

__device__ __forceinline__ float lp_key_value(u64 key) {
    const unsigned u = (unsigned)(key >> 32);
    return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}

__global__ void __launch_bounds__(kLogprobThreads) logprob_kernel(const LogprobArgs a) {
    __shared__ u64 s_key[kLogprobThreads / 32];
    __shared__ float s_a[kLogprobThreads / 32], s_b[kLogprobThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x, base = row * a.row_stride;
    const float NEG_INF = __int_as_float(0xff800000);
    pdl_wait();
    pdl_trigger();
    float m = NEG_INF;
    bool nan = false;
    for (int i = tid; i < a.n; i += kLogprobThreads) {
        const float z = lp_value(a, base + i) * a.inv_t;
        m = fmaxf(m, z);
        nan |= !(z == z);
    }
    for (int off = 1; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    if (lane == 0) s_a[warp] = m;
    nan = __syncthreads_or(nan);
    for (int i = 0; i < kLogprobThreads / 32; ++i) m = fmaxf(m, s_a[i]);
    __syncthreads();
    float S = 0.f, T = 0.f;
    for (int i = tid; i < a.n; i += kLogprobThreads) {
        const float d = lp_value(a, base + i) * a.inv_t - m;
        if (d > NEG_INF) {
            const float e = exp2f(d * kLog2e);
            S += e;
            T += d * e;
        }
    }
    for (int off = 1; off < 32; off <<= 1) {
        S += __shfl_xor_sync(0xffffffffu, S, off);
        T += __shfl_xor_sync(0xffffffffu, T, off);
    }
    if (lane == 0) {
        s_a[warp] = S;
        s_b[warp] = T;
    }
    __syncthreads();
    S = T = 0.f;
    for (int i = 0; i < kLogprobThreads / 32; ++i) {
        S += s_a[i];
        T += s_b[i];
    }
    const float NAN_ = __int_as_float(0x7fffffff);
    const bool empty = m == NEG_INF && !nan;
    const float lse = nan ? NAN_ : empty ? NEG_INF : m + logf(S);
    if (tid == 0) {
        const int t = a.logprob ? a.targets[row] : -1;
        if (t < -1 || t >= a.n) raise_status(a.status, SPD_DEV_BAD_TOKEN);
        if (a.logprob) a.logprob[row] = t < 0 || t >= a.n ? 0.f : empty ? NEG_INF : lp_value(a, base + t) * a.inv_t - lse;
        if (a.entropy) a.entropy[row] = nan ? NAN_ : empty ? 0.f : logf(S) - T / S;
        if (a.lse) a.lse[row] = lse;
    }
    u64 last = ~0ull;
    for (int k = 0; k < a.top_k; ++k) {
        u64 best = 0ull;
        for (int i = tid; i < a.n; i += kLogprobThreads) {
            const u64 key = lp_key(lp_value(a, base + i), i);
            if (key < last && key > best) best = key;
        }
        for (int off = 1; off < 32; off <<= 1) {
            const u64 o = __shfl_xor_sync(0xffffffffu, best, off);
            best = o > best ? o : best;
        }
        __syncthreads();
        if (lane == 0) s_key[warp] = best;
        __syncthreads();
        for (int i = 0; i < kLogprobThreads / 32; ++i) best = s_key[i] > best ? s_key[i] : best;
        if (tid == 0) {
            a.top_ids[row * a.top_k + k] = best ? (int)(0xffffffffu - (unsigned)best) : -1;
            a.top_logprobs[row * a.top_k + k] = best ? lp_key_value(best) * a.inv_t - lse : NEG_INF;
        }
        last = best;  // 0 when nothing is left: every later round finds nothing
    }
}

size_t token_logprobs_ws(long long rows, int n, int top_k, int num_sms) { return 16; }

cudaError_t launch_token_logprobs(const LogprobArgs& a, int num_sms, cudaStream_t st) {
    return launch_pdl(logprob_kernel, dim3((unsigned)a.rows), dim3(kLogprobThreads), 0, st, a);
}

}  // namespace spd
