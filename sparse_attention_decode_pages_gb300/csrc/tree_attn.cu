// tree_attn.cu -- attention of the nodes of a tree of drafted tokens over the paged cache, their
// ancestors and themselves: the plain form, a warp a query row, a token a lane, one pass with the running
// maximum and sum of the softmax.
#include "common.cuh"
#include "kernels.h"
#include "tree.cuh"

namespace spd {
namespace {

constexpr int kWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) tree_attn_kernel(const TreeAttnArgs a) {
    __shared__ unsigned long long s_mask[kTreeMax];
    __shared__ float s_q[kWarps][D];
    __shared__ float s_p[kWarps][32];
    __shared__ const bf16* s_v[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const float NEG_INF = __int_as_float(0xff800000);
    const int b = blockIdx.x / a.T, t = blockIdx.x % a.T;
    const int G = a.H_q / a.H_kv;
    pdl_wait();
    pdl_trigger();
    if (warp == 0 && !tree_masks(a.parents + (long long)b * a.T, a.T, s_mask) && lane == 0) raise_status(a.status, SPD_DEV_BAD_TREE);
    __syncthreads();
    int len = a.seq_lens[b];
    unsigned long long mask = s_mask[t];
    if (seq_pages(len, a.ps, a.max_pages) < 0) {
        if (threadIdx.x == 0) raise_status(a.status, SPD_DEV_BAD_LEN);
        mask = 0;
    }
    if (mask == 0) len = 0;
    const bf16* K = reinterpret_cast<const bf16*>(a.K);
    const bf16* V = reinterpret_cast<const bf16*>(a.V);
    for (int hq = warp; hq < a.H_q; hq += kWarps) {
        const int h = hq / G;
        const bf16* q = reinterpret_cast<const bf16*>(a.q) + ((long long)b * a.T + t) * a.q_stride + (long long)hq * D;
        __syncwarp();
        for (int d = lane; d < D; d += 32) s_q[warp][d] = __bfloat162float(q[d]);
        __syncwarp();
        float m = NEG_INF, l = 0.f, o[D / 32] = {};
        for (int t0 = 0; t0 < len + a.T; t0 += 32) {
            const int i = t0 + lane;
            const bf16 *k = nullptr, *v = nullptr;
            if (i < len) {
                const int p = a.page_table[(long long)b * a.max_pages + i / a.ps];
                if (p < 0 || p >= a.num_phys) {
                    raise_status(a.status, SPD_DEV_BAD_PAGE);
                } else {
                    const long long row = ((long long)p * a.H_kv + h) * a.ps + i % a.ps;
                    k = K + row * D;
                    v = V + row * D;
                }
            } else if (i < len + a.T && (mask >> (i - len) & 1)) {
                const long long row = (long long)b * a.T + (i - len);
                k = reinterpret_cast<const bf16*>(a.k_tree) + row * a.k_stride + h * D;
                v = reinterpret_cast<const bf16*>(a.v_tree) + row * a.v_stride + h * D;
            }
            float s = NEG_INF;
            if (k) {
                s = 0.f;
                for (int d = 0; d < D; ++d) s = fmaf(s_q[warp][d], __bfloat162float(k[d]), s);
                s *= a.scale_log2;
            }
            float top = s;
            for (int off = 16; off; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            const float now = fmaxf(m, top);
            if (now == NEG_INF) continue;
            const float corr = fast_exp2(m - now);
            const float p = k ? fast_exp2(s - now) : 0.f;
            float sum = p;
            for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            l = l * corr + sum;
            m = now;
            s_p[warp][lane] = p;
            s_v[warp][lane] = v;
            __syncwarp();
            for (int j = 0; j < D / 32; ++j) o[j] *= corr;
            for (int i2 = 0; i2 < 32; ++i2) {
                const bf16* vv = s_v[warp][i2];
                if (!vv) continue;
                for (int j = 0; j < D / 32; ++j) o[j] = fmaf(s_p[warp][i2], __bfloat162float(vv[lane + 32 * j]), o[j]);
            }
            __syncwarp();
        }
        const long long at = ((long long)b * a.T + t) * a.H_q + hq;
        for (int j = 0; j < D / 32; ++j) reinterpret_cast<bf16*>(a.o)[at * D + lane + 32 * j] = __float2bfloat16_rn(l != 0.f ? o[j] / l : 0.f);
        if (lane == 0 && a.lse) a.lse[at] = l != 0.f ? (m + log2f(l)) * kLn2 : NEG_INF;
    }
}

}  // namespace

size_t tree_attn_ws(int B, int H_kv, int G, int T, int D, int num_sms) { return 256; }

cudaError_t launch_tree_attn(const TreeAttnArgs& a, cudaStream_t st) {
    return launch_pdl(a.D == 128 ? tree_attn_kernel<128> : tree_attn_kernel<64>, dim3((unsigned)a.B * a.T), dim3(32 * kWarps), 0, st, a);
}

}  // namespace spd
