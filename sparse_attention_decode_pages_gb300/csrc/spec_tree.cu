// spec_tree.cu -- the accepted path through a tree of drafted tokens.
//
// At a node with target row q the children are tried in order.  With the whole weights
// W(x) = floor(2^40 q(x)) and their sum R, child c with token x is taken when
// floor(u R) < W(x), that is with probability W(x) / R (to u's resolution); a child that is
// not taken leaves the distribution behind it without its token: R -= W(x), W(x) = 0.  The last
// token is drawn from what is left, so what comes out is distributed as q whatever was tried.
//
// What a step needs from the row is its sum, so a step reads one row once, and the
// children's weights, which are loaded for all nodes at the start.  The rows of nodes off the
// path are never read.  A walk is a chain of such steps, and what bounds it is a step's latency.  So a
// cluster of CTAs walks one sequence, and nothing in a step waits for more than the step's data: warp w of the
// cluster's W sums the w-th run of the row and sends its sum to every CTA (an asynchronous store that a barrier
// there counts), every warp adds up the W sums and tries the children, a lane each, all warps alike, and goes on to
// the next row.  Two sets of sums in turn suffice: a warp sends those of step k + 2 when it has every warp's of step k + 1,
// which that warp sent after it had read step k's.  At the end the runs' sums tell which warp holds the drawn
// token; it reads its run once more.  (64 sequences of 151,936 tokens, inputs that are not in the L2: one node, that is one row's sum and the
// draw, 19 us; trees of 8 nodes, longest walks of 4 or 5, 34; of 31 nodes, longest walks of 5 to 11, 43: the start is nearly half, a
// further step 2 to 5 us.  One sequence, 8 nodes: 8.1 us, 9.6 cold.)
#include <cooperative_groups.h>

#include <atomic>

#include "common.cuh"
#include "grid40.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace spd {
namespace {

// CTAs of eight warps, four an SM: with sixteen a row is read by half as many SMs.
constexpr int kThreads = 256, kWarps = kThreads / 32, kCtas = 4;
constexpr int kMaxCluster = 16, kMaxWarps = kMaxCluster * kWarps;
constexpr int kStep = 128;   // elements of a warp's load
constexpr int kUnroll = 8;   // loads in flight where they go to registers
// Rows whose length is a multiple of 4 come by bulk copies, each warp with a ring of its own: 48 KB a CTA in flight, and the
// first chunks of the likeliest next row, that of the first child, while the sums of this one are on their way.
constexpr int kChunk = 4 * kStep, kStages = 3;
constexpr size_t kRingBytes = (size_t)kWarps * kStages * kChunk * sizeof(float);

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

// The sum of the lanes' numbers below 2^62: 22 bits at a time, each by one reduction; top: what their bits from 44 on add up to.
__device__ __forceinline__ u64 warp_sum(u64 v, unsigned& top) {
    const unsigned m = (1u << 22) - 1u;
    const unsigned a = __reduce_add_sync(0xffffffffu, (unsigned)v & m), b = __reduce_add_sync(0xffffffffu, (unsigned)(v >> 22) & m);
    top = __reduce_add_sync(0xffffffffu, (unsigned)(v >> 44));
    return a + ((u64)b << 22) + ((u64)top << 44);
}
__device__ __forceinline__ u64 warp_sum(u64 v) {
    unsigned top;
    return warp_sum(v, top);
}

// What a warp sends that has no sum, because its copies were late.  A row's sum is at most 2^61, so a total above that (by its
// bits from 44 on) has one in it; a lane adds up four at most, 2^64 - 2^62.
constexpr u64 kNoSum = 3ull << 60;
constexpr unsigned kMostTop = 1u << 17;
static_assert(kMaxWarps / 32 <= 4, "a lane's sums");

// The sum of the lanes up to this one.
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v += y;
    }
    return v;
}

// The address of this CTA's shared memory in another CTA of the cluster.
__device__ __forceinline__ uint32_t remote(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// Stores 8 bytes to a CTA's shared memory and counts them on its barrier.
__device__ __forceinline__ void send(uint32_t addr, u64 v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u64 [%0], %1, [%2];" ::"r"(addr), "l"(v), "r"(bar) : "memory");
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads, kCtas) accept_tree_kernel(TreeAcceptArgs a) {
    extern __shared__ __align__(128) float ring_all[];
    __shared__ uint64_t s_full[kWarps][kStages];
    __shared__ u64 s_sums[2][kMaxWarps];  // the runs' sums of a row, in turn
    __shared__ uint64_t s_bar[2];
    __shared__ u64 s_w[kTreeMax];         // a node's weight in its parent's row
    __shared__ float s_u[kTreeMax];
    __shared__ int s_parent[kTreeMax], s_token[kTreeMax];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / size, T = a.T, W = size * kWarps, me = rank * kWarps + warp;
    const int n = (int)a.n;
    // elements of a warp's run: whole loads
    const int run = ((n + W - 1) / W + kStep - 1) / kStep * kStep;
    const int first = me * run, last = min(n, first + run);
    auto limit = [&]() { return a.wait_ns > kDefaultWaitNs ? a.wait_ns : kDefaultWaitNs; };
    if (tid < 2) mbar_init(s_bar + tid, 1);
    if (VEC && lane < kStages) mbar_init(&s_full[warp][lane], 1);
    mbar_fence_init();
    __syncwarp();
    pdl_wait();
    pdl_trigger();

    bool ok = true;
    int flying = 0;  // chunks that were asked for and that no sum waits for, from the ring's slot on
    const int chunks = VEC && last > first ? (last - first + kChunk - 1) / kChunk : 0;
    float* ring = ring_all + warp * (kStages * kChunk);
    int slot = 0;  // of the ring's next chunk
    uint32_t parity = 0;
    const float* rows = a.q + (long long)b * T * n;
    // lane 0 asks for chunk c of a node's row
    auto ask = [&](int node, int c, int to) {
        const int x = first + c * kChunk;
        const uint32_t bytes = (uint32_t)min(kChunk, last - x) * sizeof(float);
        mbar_arrive_expect_tx(&s_full[warp][to], bytes);
        bulk_load(ring + to * kChunk, rows + (long long)node * n + x, bytes, &s_full[warp][to]);
    };
    auto ask_first = [&](int node) {
        if (VEC && lane == 0)
            for (int c = 0; c < min(kStages, chunks); ++c) ask(node, c, (slot + c) % kStages);
    };
    auto next_chunk = [&]() {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s_full[warp][slot], parity, a.status, a.wait_ns));
        return ok;
    };
    auto advance = [&]() {
        if (++slot == kStages) {
            slot = 0;
            parity ^= 1u;
        }
    };
    // copies land before their memory is given back, also those that nobody reads
    auto drain = [&]() {
        for (; flying > 0; --flying) {
            mbar_wait_bounded(&s_full[warp][slot], parity, a.status, limit());
            advance();
        }
    };
    // this warp's part of a row's sum; the first chunks have been asked for
    auto run_sum = [&](int node) {
        u64 sum = 0;
        if (VEC) {
            for (int c = 0; c < chunks; ++c) {
                if (!next_chunk()) {
                    flying = min(kStages, chunks - c);
                    break;
                }
                const int left = last - first - c * kChunk;
                float4 v[kChunk / kStep];
#pragma unroll
                for (int i = 0; i < kChunk / kStep; ++i) {
                    v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (i * kStep + lane * 4 < left) v[i] = *reinterpret_cast<const float4*>(ring + slot * kChunk + i * kStep + lane * 4);
                }
                __syncwarp();  // the chunk has been read
                if (lane == 0 && c + kStages < chunks) ask(node, c + kStages, slot);
                GridSum g;
#pragma unroll
                for (int i = 0; i < kChunk / kStep; ++i) {
                    g.take(make_float2(v[i].x, v[i].y));
                    g.take(make_float2(v[i].z, v[i].w));
                }
                sum += g.total();
                advance();
            }
        } else {
            const float* row = rows + (long long)node * n;
            for (int x = first + lane * 4; x < last; x += kUnroll * kStep) {
                float4 v[kUnroll];
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) v[i] = load4<VEC>(row, x + i * kStep, last);
                GridSum g;
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) {
                    g.take(make_float2(v[i].x, v[i].y));
                    g.take(make_float2(v[i].z, v[i].w));
                }
                sum += g.total();
            }
        }
        return warp_sum(sum);
    };

    // the nodes, and their weights, asked for before the first row's sum
    ask_first(0);
    int parent = -2, token = -1;
    float u = 0.f, q = 0.f;
    if (tid < T) {
        parent = a.parents[(long long)b * T + tid];
        token = a.draft[(long long)b * T + tid];
        u = a.u_acc[(long long)b * T + tid];
        if (rank == 0 && (parent < -2 || parent >= tid)) raise_status(a.status, SPD_DEV_BAD_TREE);
        if (parent >= 0 && parent < tid && token >= 0 && token < n) q = __ldg(rows + (long long)parent * n + token);
    }
    u64 sum = run_sum(0);
    if (tid < kTreeMax) {
        s_parent[tid] = parent;
        s_token[tid] = token;
        s_u[tid] = u;
        s_w[tid] = fixed40(q);
    }
    cluster.sync();  // the nodes are there, and every CTA's barriers
    if (s_parent[0] != -1) {  // no root: the same for the whole cluster
        if (rank == 0 && tid < T) {
            a.path[(long long)b * T + tid] = -1;
            a.tokens[(long long)b * T + tid] = -1;
            if (tid == 0) a.n_path[b] = 0;
        }
        drain();
        return;
    }

    int node = 0, count = 0;
    int my_path[2] = {-1, -1};  // lane i: the walk's nodes i and i + 32
    u64 left;                   // what the children leave of the row's sum
    unsigned tried[2];          // the last node's children that were tried: nodes 0 to 31 and 32 to 63
    u64 w2[2];                  // this lane's two nodes' weights in the row (0: no child, or a token tried before)
    while (true) {
        const int turn = count & 1;
        const uint32_t bar = smem_u32(s_bar + turn);
        if (tid == 0) mbar_arrive_expect_tx(s_bar + turn, W * 8);
        if (lane < size) send(remote(smem_u32(s_sums[turn] + me), lane), ok ? sum : kNoSum, remote(bar, lane));
        // while the sums are on their way: this lane's two nodes, if they are children of the node
        int tk[2];
        unsigned kids[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = lane + 32 * i;
            const bool child = c > node && s_parent[c] == node;
            tk[i] = s_token[c];
            if (child && (tk[i] < 0 || tk[i] >= n)) tk[i] = -1 - c;  // no token: a weight of 0 that equals no other's
            kids[i] = __ballot_sync(0xffffffffu, child);
            w2[i] = child && tk[i] >= 0 ? s_w[c] : 0;
        }
        const int guess = kids[0] ? __ffs((int)kids[0]) - 1 : kids[1] ? __ffs((int)kids[1]) + 31 : -1;
        if (ok && guess >= 0 && count > 0) {  // (the first rows of all sequences have the memory to themselves)
            ask_first(guess);
            flying = min(kStages, chunks);
        }
        for (unsigned k = kids[0]; k; k &= k - 1) {
            const int c = __ffs((int)k) - 1, x = __shfl_sync(0xffffffffu, tk[0], c);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (lane + 32 * i > c && tk[i] == x) w2[i] = 0;
        }
        for (unsigned k = kids[1]; k; k &= k - 1) {
            const int c = __ffs((int)k) + 31, x = __shfl_sync(0xffffffffu, tk[1], c - 32);
            if (lane + 32 > c && tk[1] == x) w2[1] = 0;
        }
        // what the children before each one take, and all of them
        u64 pre[2] = {warp_scan(w2[0], lane) - w2[0], 0}, all = __shfl_sync(0xffffffffu, pre[0] + w2[0], 31);
        if (kids[1]) {
            const u64 in = warp_scan(w2[1], lane);
            pre[1] = all + in - w2[1];
            all += __shfl_sync(0xffffffffu, in, 31);
        }
        // (never a shorter limit than the usual one: a sum that is on its way to a CTA lands before it ends)
        ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(s_bar + turn, (uint32_t)count >> 1 & 1u, a.status, limit()));
        if (!ok) break;
        u64 total = 0;
        for (int i = lane; i < W; i += 32) total += s_sums[turn][i];
        unsigned top;
        total = warp_sum(total, top);
        ok = top <= kMostTop;  // (the same for all warps of the cluster)
        if (!ok) break;
        // the children in order: each is tried on what the earlier ones leave
        const unsigned p0 = __ballot_sync(0xffffffffu, w2[0] && scaled_floor(s_u[lane], total - pre[0]) < w2[0]);
        unsigned p1 = 0;
        if (kids[1]) p1 = __ballot_sync(0xffffffffu, w2[1] && scaled_floor(s_u[lane + 32], total - pre[1]) < w2[1]);
        const int next = p0 ? __ffs((int)p0) - 1 : p1 ? __ffs((int)p1) + 31 : -1;
        tried[0] = kids[0] & (next < 0 || next >= 32 ? ~0u : (1u << next) - 1u);
        tried[1] = kids[1] & (next < 0 ? ~0u : next < 32 ? 0u : (1u << (next - 32)) - 1u);
        if (rank == 0 && warp == 0) {
            const bool bad = ((tried[0] >> lane & 1u) && tk[0] < 0) || ((tried[1] >> lane & 1u) && tk[1] < 0);
            if (bad) raise_status(a.status, SPD_DEV_BAD_TOKEN);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (lane + 32 * i == count) my_path[i] = node;
        ++count;
        left = total - all;
        if (next < 0) break;
        if (next != guess)  // what was asked for in vain
            for (; flying > 0 && next_chunk(); --flying) advance();
        node = next;
        if (ok) {
            flying = 0;
            if (next != guess || count == 1) ask_first(next);
            sum = run_sum(next);
        }
    }

    if (ok && rank == 0 && warp == 0) {
        // lane i writes entries i and i + 32; a node's token is that of the next one on the path
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = lane + 32 * i;
            const int after0 = __shfl_down_sync(0xffffffffu, my_path[i], 1), wrap = __shfl_sync(0xffffffffu, my_path[1], 0);
            const int after = lane < 31 ? after0 : i ? -1 : wrap;
            if (e < T) {
                a.path[(long long)b * T + e] = my_path[i];
                if (e != count - 1 || left == 0) a.tokens[(long long)b * T + e] = e < count - 1 ? s_token[after] : -1;
            }
        }
        if (lane == 0) a.n_path[b] = count;
    }
    if (ok && left != 0) {
        // the run that holds the drawn token: the runs' sums, without the tokens tried, up to this warp's
        const u64 target = min(scaled_floor(a.u_res[b], left), left - 1);
        const u64* sums = s_sums[(count - 1) & 1];
        u64 before = 0;
        for (int i = lane; i < me; i += 32) before += sums[i];
        u64 mine = 0, gone = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool out = tried[i] >> lane & 1u;
            const int at = out ? s_token[lane + 32 * i] : -1;
            if (at >= 0 && at < first) gone += w2[i];
            if (at >= first && at < last) mine += w2[i];
        }
        before = warp_sum(before) - warp_sum(gone);
        mine = sums[me] - warp_sum(mine);
        if (before <= target && target - before < mine) {
            const float* row = rows + (long long)node * n;
            for (int x0 = first; x0 < last; x0 += kUnroll * kStep) {
                float4 v[kUnroll];
                u64 part[kUnroll];
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) v[i] = load4<VEC>(row, x0 + i * kStep + lane * 4, last);
                // a token that was tried has no weight
                for (int k = 0; k < 2; ++k)
                    for (unsigned m = tried[k]; m; m &= m - 1) {
                        const int at = s_token[__ffs((int)m) - 1 + 32 * k] - x0 - lane * 4;
#pragma unroll
                        for (int i = 0; i < kUnroll; ++i) {
                            if (at == i * kStep) v[i].x = 0.f;
                            if (at == i * kStep + 1) v[i].y = 0.f;
                            if (at == i * kStep + 2) v[i].z = 0.f;
                            if (at == i * kStep + 3) v[i].w = 0.f;
                        }
                    }
                float4 y = v[0];
                int at = -1;
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) {
                    GridSum g;
                    g.take(make_float2(v[i].x, v[i].y));
                    g.take(make_float2(v[i].z, v[i].w));
                    part[i] = warp_sum(g.total());
                }
#pragma unroll
                for (int i = 0; i < kUnroll; ++i) {
                    if (at < 0 && target - before < part[i]) {
                        at = i;
                        y = v[i];
                    }
                    if (at < 0) before += part[i];
                }
                if (at < 0) continue;
                const u64 w[4] = {fixed40(y.x), fixed40(y.y), fixed40(y.z), fixed40(y.w)};
                const u64 four = w[0] + w[1] + w[2] + w[3];
                u64 r = before + warp_scan(four, lane) - four;
                int hit = -1;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    r += w[j];
                    if (hit < 0 && r > target) hit = j;
                }
                const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0);
                if (lane == __ffs((int)hits) - 1) a.tokens[(long long)b * T + count - 1] = x0 + at * kStep + lane * 4 + hit;
                break;
            }
        }
    }
    drain();
    cluster.sync();  // no CTA ends while another may still send to it
}

}  // namespace

// CTAs of a cluster: as many as let every sequence's cluster run at once, up to 16.  One sequence of a 151,936-token
// vocabulary, 4 / 8 / 16 CTAs: 13.9 / 10.9 / 9.5 us; 19: 22.3 / 16.8 / 19.6; 64, trees of 31 nodes: 47.1 / 45.7 / 43.0; 150: 2 / 4 / 8 CTAs
// 63.9 / 70.0 / 55.5; 400 sequences, 32,000 tokens: 1 / 2 / 4 CTAs 47.8 / 35.7 / 38.9.  (So twice as many would be the better rule for
// most batches, by up to a quarter.)
cudaError_t launch_spec_accept_tree(const TreeAcceptArgs& a, int num_sms, cudaStream_t st) {
    static std::atomic<bool> known[64][2];
    if (a.B <= 0) return cudaSuccess;
    unsigned cluster = kMaxCluster;
    while (cluster > 1 && (long long)cluster * a.B > kCtas * num_sms) cluster /= 2;
    const bool vec = a.n % 4 == 0;
    auto* kern = vec ? accept_tree_kernel<true> : accept_tree_kernel<false>;
    const size_t smem = vec ? kRingBytes : 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !known[dev][vec].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingBytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) known[dev][vec].store(true, std::memory_order_release);
    }
    return launch_pdl_cluster(kern, dim3((unsigned)a.B * cluster), dim3(kThreads), smem, cluster, st, a);
}

}  // namespace spd
