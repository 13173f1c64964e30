// spec_tree.cu -- the accepted path through a tree of drafted tokens.
//
// At a node with target row q the children are tried in order.  With the whole weights
// W(x) = floor(2^40 q(x)) and their sum R, child c with token x is taken when
// floor(u R) < W(x), that is with probability W(x) / R (to u's resolution); a child that is
// not taken leaves the distribution behind it without its token: R -= W(x), W(x) = 0.  The last
// token is drawn from what is left, so what comes out is distributed as q whatever was tried.
//
// What a step needs from the row is its sum, so a step reads one row once and the
// children's weights, which are loaded for all nodes at the start.  A cluster walks one
// sequence: warp w of the cluster's W sums the w-th run of the row, the CTAs' sums go to
// every CTA through distributed shared memory (two sets in turn, one cluster barrier a step), and
// every CTA takes the same decision.  The rows of nodes off the path are never read.  At
// the end the runs' sums tell which warp holds the drawn token; it reads its run once more.
#include <cooperative_groups.h>

#include "common.cuh"
#include "grid40.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace spd {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kStep = 128;   // elements of a warp's load
constexpr int kUnroll = 8;   // loads in flight

// Four elements of a row from x, 0 behind `end`.
template <bool VEC>
__device__ __forceinline__ float4 load4(const float* row, long long x, long long end) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (VEC) {
        if (x < end) v = __ldg(reinterpret_cast<const float4*>(row + x));
    } else {
        if (x < end) v.x = __ldg(row + x);
        if (x + 1 < end) v.y = __ldg(row + x + 1);
        if (x + 2 < end) v.z = __ldg(row + x + 2);
        if (x + 3 < end) v.w = __ldg(row + x + 3);
    }
    return v;
}

// The sum of four weights: in 32 bits where each is below 2^30 (probabilities below 2^-10,
// nearly all), else in 64.
__device__ __forceinline__ u64 sum4(const float4& v) {
    const unsigned a = fixed40_u32(v.x), b = fixed40_u32(v.y), c = fixed40_u32(v.z), d = fixed40_u32(v.w);
    if ((a | b | c | d) < (1u << 30)) return a + b + c + d;
    return fixed40(v.x) + fixed40(v.y) + fixed40(v.z) + fixed40(v.w);
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads) accept_tree_kernel(TreeAcceptArgs a) {
    __shared__ u64 s_share[2][kMaxCluster];  // the CTAs' sums of a row, in turn
    __shared__ u64 s_warp[kWarps];
    __shared__ u64 s_w[kTreeMax];            // a node's weight in its parent's row
    __shared__ float s_u[kTreeMax];
    __shared__ int s_parent[kTreeMax], s_token[kTreeMax], s_tried[kTreeMax], s_path[kTreeMax];
    __shared__ int s_next, s_ntried, s_cross;
    __shared__ u64 s_left, s_before;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / size, T = a.T;
    const long long n = a.n;
    // elements of a warp's run: whole loads
    const long long run = ((n + (long long)size * kWarps - 1) / ((long long)size * kWarps) + kStep - 1) / kStep * kStep;
    const long long first = (long long)(rank * kWarps + warp) * run;
    const long long last = min(n, first + run);
    pdl_wait();
    pdl_trigger();

    if (tid < T) {
        const int parent = a.parents[(long long)b * T + tid];
        const int token = a.draft[(long long)b * T + tid];
        s_parent[tid] = parent;
        s_token[tid] = token;
        s_u[tid] = a.u_acc[(long long)b * T + tid];
        if (rank == 0 && (parent < -2 || parent >= tid)) raise_status(a.status, SPD_DEV_BAD_TREE);
        u64 w = 0;
        if (parent >= 0 && parent < tid && token >= 0 && token < n) w = fixed40(__ldg(a.q + ((long long)b * T + parent) * n + token));
        s_w[tid] = w;
    }
    __syncthreads();
    if (tid > 0 && tid < T) {  // a token that an earlier sibling has is no weight any more when it is tried
        bool again = false;
        for (int u = 1; u < tid; ++u) again |= s_parent[u] == s_parent[tid] && s_token[u] == s_token[tid];
        if (again) s_w[tid] = 0;
    }
    const bool root = s_parent[0] == -1;
    cluster.sync();  // the other CTAs' shared memory is there
    if (!root) {     // the same for the whole cluster
        if (rank == 0 && tid < T) {
            a.path[(long long)b * T + tid] = -1;
            a.tokens[(long long)b * T + tid] = -1;
            if (tid == 0) a.n_path[b] = 0;
        }
        return;
    }

    int node = 0, count = 0;
    const float* row;
    while (true) {
        row = a.q + ((long long)b * T + node) * n;
        u64 sum = 0;
        for (long long x = first + lane * 4; x < last; x += kUnroll * kStep) {
            float4 v[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) v[i] = load4<VEC>(row, x + i * kStep, last);
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) sum += sum4(v[i]);
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) s_warp[warp] = sum;
        __syncthreads();
        u64* share = s_share[count & 1];
        if (warp == 0) {
            u64 mine = lane < kWarps ? s_warp[lane] : 0;
#pragma unroll
            for (int off = kWarps / 2; off; off >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, off);
            mine = __shfl_sync(0xffffffffu, mine, 0);
            if (lane < size) *cluster.map_shared_rank(share + rank, lane) = mine;
        }
        cluster.sync();
        if (tid == 0) {
            u64 left = 0;
            for (int r = 0; r < size; ++r) left += share[r];
            int next = -1, tried = 0;
            for (int c = node + 1; c < T; ++c) {
                if (s_parent[c] != node) continue;
                const int token = s_token[c];
                if (token < 0 || token >= n) {
                    if (rank == 0) raise_status(a.status, SPD_DEV_BAD_TOKEN);
                    continue;
                }
                if (scaled_floor(s_u[c], left) < s_w[c]) {
                    next = c;
                    break;
                }
                left -= s_w[c];
                s_tried[tried++] = c;
            }
            s_path[count] = node;
            s_next = next;
            s_ntried = tried;
            s_left = left;
        }
        __syncthreads();
        ++count;
        if (s_next < 0) break;
        node = s_next;
        __syncthreads();  // s_next has been read
    }

    const u64 left = s_left;
    const int tried = s_ntried;
    if (rank == 0 && tid < T) {
        a.path[(long long)b * T + tid] = tid < count ? s_path[tid] : -1;
        if (tid != count - 1 || left == 0) a.tokens[(long long)b * T + tid] = tid < count - 1 ? s_token[s_path[tid + 1]] : -1;
        if (tid == 0) a.n_path[b] = count;
    }
    if (left == 0) return;
    const u64 target = min(scaled_floor(a.u_res[b], left), left - 1);
    if (tid == 0) {  // the run that holds it, without the tokens tried
        u64* share = s_share[(count - 1) & 1];
        for (int i = 0; i < tried; ++i) {
            const int c = s_tried[i];
            const int at = (int)(s_token[c] / run);
            share[at / kWarps] -= s_w[c];
            if (at / kWarps == rank) s_warp[at % kWarps] -= s_w[c];
        }
        u64 before = 0;
        for (int r = 0; r < rank; ++r) before += share[r];
        int cross = -1;
        if (before <= target && target - before < share[rank]) {
            cross = 0;
            while (target - before >= s_warp[cross]) before += s_warp[cross++];
        }
        s_cross = cross;
        s_before = before;
    }
    __syncthreads();
    if (warp != s_cross) return;
    u64 before = s_before;
    for (long long x0 = first; x0 < last; x0 += kUnroll * kStep) {
        float4 v[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) v[i] = load4<VEC>(row, x0 + i * kStep + lane * 4, last);
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const long long x = x0 + i * kStep + lane * 4;
            u64 w[4] = {fixed40(v[i].x), fixed40(v[i].y), fixed40(v[i].z), fixed40(v[i].w)};
            for (int k = 0; k < tried; ++k) {
                const long long at = s_token[s_tried[k]] - x;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (at == j) w[j] = 0;
            }
            const u64 mine = w[0] + w[1] + w[2] + w[3];
            u64 incl = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const u64 y = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += y;
            }
            u64 r = before + incl - mine;
            int hit = -1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                r += w[j];
                if (hit < 0 && r > target) hit = j;
            }
            const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0);
            if (hits) {
                if (lane == __ffs((int)hits) - 1) a.tokens[(long long)b * T + count - 1] = (int)x + hit;
                return;
            }
            before += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
}

}  // namespace

cudaError_t launch_spec_accept_tree(const TreeAcceptArgs& a, int num_sms, cudaStream_t st) {
    if (a.B <= 0) return cudaSuccess;
    (void)num_sms;
    const unsigned cluster = 8;
    return launch_pdl_cluster(a.n % 4 == 0 ? accept_tree_kernel<true> : accept_tree_kernel<false>,
                              dim3((unsigned)a.B * cluster), dim3(kThreads), 0, cluster, st, a);
}

}  // namespace spd
