// evict.cu -- shortens the cache to the tokens of the largest attention weights.
//
// Two kernels.  The first chooses: of a (sequence, KV head)'s tokens the first n_sink, the newest n_recent, and the
// others of the largest weights.  A weight becomes a 32-bit key in the order of the numbers (above all numbers for the
// tokens that always stay); the largest key that `budget` tokens reach is found by counting, as the keys come in, those with each
// of the 2,048 values of their upper 11 bits, then two bits at a time by counting those that reach each of three candidates, until
// few keys are left in the range; those go on alone, one a thread, a bit and a barrier that counts at a time.  Tokens with a larger key stay, and of those with that very key the lowest positions.  A warp
// has consecutive tokens, so one scan of the warps' counts and ballots give every kept token its place.
// What bounds it is a count's latency: three CTAs an SM where rows are many, clusters of up to eight CTAs a row, their counts joined
// through distributed shared memory, where rows are few or long (the choice for 512 rows of 8K-16K tokens: 33 us, 8 rows of 65,521:
// 12; without the count of the upper bits 52 and 21, with keys in registers, one CTA of 1,024 threads an SM, 89 and 32).  The keys stay in shared memory; rows beyond
// 8 x 49,152 tokens are read anew for each count.  (Clusters and room follow the page table's width, not the lengths: 512 rows of 8K-16K
// tokens in a table for 131,072 tokens take eight CTAs each, the whole call 512 us in place of 390.)
//
// The second moves: a warp takes a new page of a KV head, 16 tokens at a time, all their keys' and values' rows in flight at
// once, and forms the page's minima and maxima on the way.  It is bound by memory: each kept row is read once and written
// once (512 heads' 4,096 tokens, 2.2 GB: 357 us, 91 % of the measured copy peak).
#include <cooperative_groups.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace spd {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kHeld = 49152, kHeldMany = 16384;  // tokens that a CTA holds: alone on an SM, and three on an SM
constexpr int kFew = kThreads;                   // keys that one CTA goes on with, one a thread
constexpr int kBinShift = 21, kBins = 1 << (32 - kBinShift);  // of the first count: keys' sign, exponent and two bits
static_assert(kBins == 4 * kThreads, "four bins a thread");

// Larger weight, larger key; -0 as 0; NaN below every number.  (No token: 0; one that stays whatever its weight: kAlways.)
constexpr uint32_t kAlways = 0xffffffffu;
__device__ __forceinline__ uint32_t weight_key(float w) { return w != w ? 1u : float_key(w + 0.f); }

// HELD: the cluster's shared memory holds the row's keys, `room` tokens a CTA.  Otherwise its CTAs go over parts of the row again
// and again.
template <bool HELD>
__global__ void __launch_bounds__(kThreads) choose_kernel(const EvictArgs a) {
    extern __shared__ __align__(16) uint32_t s_key[];
    __shared__ unsigned s_warp[2][kWarps][3];           // the warps' counts, in turn
    __shared__ unsigned s_count[2][kMaxCluster][3];     // the CTAs' counts, in turn
    __shared__ uint32_t s_few[kFew];                    // (the first CTA's) the keys that are left
    __shared__ __align__(16) unsigned s_bin[kBins];     // (in descending order of their keys)
    __shared__ unsigned s_cut[3];                       // the bin of the largest key wanted, keys from it on, keys above it
    __shared__ unsigned s_nfew;
    __shared__ uint32_t s_found;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), size = (int)cluster.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x / size, b = row / a.H_kv;
    if (tid == 0) s_nfew = 0;
    pdl_trigger();
    const int len = a.seq_lens[b];
    const bool head = rank == 0 && tid == 0 && row == b * a.H_kv;
    if (seq_pages(len, a.ps, a.max_pages) < 0) {  // the same for the whole cluster
        if (head) {
            raise_status(a.status, SPD_DEV_BAD_LEN);
            a.new_lens[b] = 0;
        }
        return;
    }
    if (head) a.new_lens[b] = min(len, a.budget);
    int32_t* kept = a.kept + (long long)row * a.budget;
    if (len <= a.budget) {  // all of them
        for (long long i = (long long)rank * kThreads + tid; i < len; i += (long long)size * kThreads) kept[i] = (int)i;
        return;
    }
    const unsigned k = (unsigned)a.budget;
    const float* w = a.w + (long long)row * a.max_pages * a.ps;

    // this warp's tokens: `per` (a multiple of four) times 32 consecutive ones
    const int warps = size * kWarps;
    const int per = ((len + 32 * warps - 1) / (32 * warps) + 3) & ~3;
    const int base = (rank * kWarps + warp) * per * 32 + lane;
    auto key_of = [&](int t, float x) { return t >= len ? 0u : t < a.n_sink || t >= len - a.n_recent ? kAlways : weight_key(x); };
    auto weight_at = [&](int t) { return __ldg(w + min(t, len - 1)); };
    uint32_t* keys = s_key + warp * per * 32;
    auto count_bin = [&](uint32_t x) {
        if (x) atomicAdd(s_bin + (kBins - 1 - (x >> kBinShift)), 1u);
    };
    reinterpret_cast<uint4*>(s_bin)[tid] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    if (HELD) {
        // 128 tokens at a time, four a lane (a row's room is a multiple of 16, so none lies past its end)
        const bool vec = (reinterpret_cast<uintptr_t>(a.w) & 15) == 0;
        const int first = (rank * kWarps + warp) * per * 32 + 4 * lane, last = a.max_pages * a.ps - 4;
        for (int i = 0; i < per; i += 16) {
            float4 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float* from = w + min(first + 32 * i + 128 * j, last);
                x[j] = vec ? __ldg(reinterpret_cast<const float4*>(from)) : make_float4(__ldg(from), __ldg(from + 1), __ldg(from + 2), __ldg(from + 3));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = first + 32 * i + 128 * j;
                if (i + 4 * j >= per) break;
                uint4 y;
                if (__all_sync(0xffffffffu, t >= a.n_sink && t + 3 < len - a.n_recent)) {
                    y = make_uint4(weight_key(x[j].x), weight_key(x[j].y), weight_key(x[j].z), weight_key(x[j].w));
                } else {
                    y = make_uint4(key_of(t, x[j].x), key_of(t + 1, x[j].y), key_of(t + 2, x[j].z), key_of(t + 3, x[j].w));
                }
                *reinterpret_cast<uint4*>(keys + 32 * i + 128 * j + 4 * lane) = y;
                count_bin(y.x);
                count_bin(y.y);
                count_bin(y.z);
                count_bin(y.w);
            }
        }
        __syncwarp();
    }
    // f(key) for each of this warp's tokens, in any order
    auto each = [&](auto f) {
        if (HELD) {
            for (int i = 0; i < per / 4; ++i) {
                const uint4 x = *reinterpret_cast<const uint4*>(keys + 128 * i + 4 * lane);
                f(x.x);
                f(x.y);
                f(x.z);
                f(x.w);
            }
        } else {
#pragma unroll 8
            for (int i = 0; i < per; ++i) f(key_of(base + 32 * i, weight_at(base + 32 * i)));
        }
    };
    // the cluster's three counts; the warps' own stay in s_warp[turn ^ 1], the CTAs' in s_count[turn ^ 1]
    int turn = 0;
    auto join = [&](unsigned (&n)[3]) {
        if (per <= 31) {  // at most 992 each in a warp: one reduction of ten bits each
            const unsigned all = __reduce_add_sync(0xffffffffu, n[0] | n[1] << 10 | n[2] << 20);
            n[0] = all & 1023u;
            n[1] = all >> 10 & 1023u;
            n[2] = all >> 20;
        } else {
#pragma unroll
            for (int j = 0; j < 3; ++j) n[j] = __reduce_add_sync(0xffffffffu, n[j]);
        }
        if (lane < 3) s_warp[turn][warp][lane] = lane == 0 ? n[0] : lane == 1 ? n[1] : n[2];
        __syncthreads();
        if (size == 1) {
#pragma unroll
            for (int j = 0; j < 3; ++j) n[j] = __reduce_add_sync(0xffffffffu, lane < kWarps ? s_warp[turn][lane][j] : 0u);
        } else {
            if (warp < 3) {
                const unsigned sum = __reduce_add_sync(0xffffffffu, lane < kWarps ? s_warp[turn][lane][warp] : 0u);
                if (lane < size) *cluster.map_shared_rank(&s_count[turn][rank][warp], lane) = sum;
            }
            cluster.sync();
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                n[j] = 0;
                for (int r = 0; r < size; ++r) n[j] += s_count[turn][r][j];
            }
        }
        turn ^= 1;
    };
    if (!HELD) each(count_bin);
    if (size > 1) cluster.sync();
    else __syncthreads();

    // the bin of the largest key that at least k tokens reach: thread i has the i-th four bins
    {
        uint4 y = reinterpret_cast<const uint4*>(s_bin)[tid];
#pragma unroll 4
        for (int r = 1; r < size; ++r) {
            const uint4 z = reinterpret_cast<const uint4*>(cluster.map_shared_rank(s_bin, (rank + r) & (size - 1)))[tid];
            y.x += z.x;
            y.y += z.y;
            y.z += z.z;
            y.w += z.w;
        }
        const unsigned mine = y.x + y.y + y.z + y.w;
        unsigned upto = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const unsigned z = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += z;
        }
        if (lane == 31) s_warp[1][warp][0] = upto;
        __syncthreads();
        upto += __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[1][lane][0] : 0u);
        unsigned above = upto - mine;
        if (above < k && upto >= k) {
            const unsigned n[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (above < k && above + n[j] >= k) {
                    s_cut[0] = kBins - 1 - (4 * tid + j);
                    s_cut[1] = above + n[j];
                    s_cut[2] = above;
                }
                above += n[j];
            }
        }
        __syncthreads();
    }

    // that key: `found` so far, which at_found tokens reach, and above ones reach what lies behind its range
    uint32_t found = s_cut[0] << kBinShift;
    unsigned at_found = s_cut[1], above = s_cut[2];
    int bit = kBinShift;
#pragma unroll 1
    while (at_found - above > kFew && bit > 0) {
        const bool last = bit == 1;  // a single bit is left: the three are one
        bit = last ? 0 : bit - 2;
        const uint32_t c1 = found | 1u << bit, c2 = last ? c1 : found | 2u << bit, c3 = last ? c1 : found | 3u << bit;
        unsigned n[3] = {0, 0, 0};
        each([&](uint32_t x) {
            n[0] += x >= c1;
            n[1] += x >= c2;
            n[2] += x >= c3;
        });
        join(n);
        if (n[2] >= k) {
            found = c3;
            at_found = n[2];
        } else if (n[1] >= k) {
            found = c2;
            at_found = n[1];
            above = n[2];
        } else if (n[0] >= k) {
            found = c1;
            at_found = n[0];
            above = n[1];
        } else {
            above = n[0];
        }
    }
    if (bit > 0) {
        // few keys are left in the range: one CTA goes on with one a thread, a bit and a barrier at a time
        unsigned mine = 0;
        each([&](uint32_t x) { mine += x >> bit == found >> bit && x != 0; });
        unsigned at = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const unsigned y = __shfl_up_sync(0xffffffffu, at, off);
            if (lane >= off) at += y;
        }
        unsigned all = __shfl_sync(0xffffffffu, at, 31);
        if (lane == 0 && all) all = atomicAdd(cluster.map_shared_rank(&s_nfew, 0), all);
        at += __shfl_sync(0xffffffffu, all, 0) - mine;
        uint32_t* few = cluster.map_shared_rank(s_few, 0);
        if (mine)
            each([&](uint32_t x) {
                if (x >> bit == found >> bit && x != 0 && at < kFew) few[at++] = x;
            });
        if (size > 1) cluster.sync();
        else __syncthreads();
        if (rank == 0) {
            const uint32_t x = tid < (int)min(s_nfew, (unsigned)kFew) ? s_few[tid] : 0u;
            const int need = (int)(k - above);  // (at least one: those above are too few)
#pragma unroll 1
            while (--bit >= 0)
                if (__syncthreads_count(x >= (found | 1u << bit)) >= need) found |= 1u << bit;
            if (size > 1 && tid < size) *cluster.map_shared_rank(&s_found, tid) = found;
        }
        if (size > 1) {
            cluster.sync();
            found = s_found;
        }
    }

    // how many stay without regard to ties, and how many tie, up to each warp
    unsigned n[3] = {0, 0, 0};
    each([&](uint32_t x) {
        n[0] += x > found;
        n[1] += x == found;
    });
    join(n);
    const unsigned need = k - n[0];  // ties that stay: the first ones
    unsigned stay_before = __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[turn ^ 1][lane][0] : 0u);
    unsigned tie_before = __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[turn ^ 1][lane][1] : 0u);
    if (size > 1)
        for (int r = 0; r < rank; ++r) {
            stay_before += s_count[turn ^ 1][r][0];
            tie_before += s_count[turn ^ 1][r][1];
        }
    const unsigned below = (1u << lane) - 1u;
    const bool all_ties = need == n[1];
    unsigned before = stay_before + tie_before;
    for (int i = 0; i < per; ++i) {
        const int t = base + 32 * i;
        const uint32_t x = HELD ? keys[32 * i + lane] : key_of(t, weight_at(t));
        if (all_ties) {
            const unsigned m = __ballot_sync(0xffffffffu, x >= found);
            if (x >= found) kept[before + __popc(m & below)] = t;
            before += __popc(m);
        } else {
            const unsigned ms = __ballot_sync(0xffffffffu, x > found), mt = __ballot_sync(0xffffffffu, x == found);
            const unsigned my_tie = tie_before + __popc(mt & below);
            // kept ones before this token: those that stay, and ties up to `need`
            if (x > found || (x == found && my_tie < need)) kept[stay_before + __popc(ms & below) + min(my_tie, need)] = t;
            stay_before += __popc(ms);
            tie_before += __popc(mt);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(128) move_kernel(const EvictArgs a, int pages, long long items) {
    constexpr int LPR = D * 2 / 16, RPI = 32 / LPR;  // lanes of a row, rows of an access
    constexpr int ACC = 16 / RPI;                    // accesses for 16 tokens
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    pdl_wait();
    pdl_trigger();
    if (item >= items) return;
    const int page = (int)(item % pages);
    const long long row = item / pages;  // (sequence, KV head)
    const int b = (int)(row / a.H_kv), h = (int)(row - (long long)b * a.H_kv);
    const int m = a.new_lens[b];
    const int j0 = page * a.ps;
    if (j0 >= m) return;
    const int phys = a.dst_table[(long long)b * a.max_pages + page];
    if (phys < 0 || phys >= a.num_phys) {
        if (lane == 0) raise_status(a.status, SPD_DEV_BAD_PAGE);
        return;
    }
    const int r0 = lane / LPR, ch = lane % LPR;
    const long long dst = ((long long)phys * a.H_kv + h) * a.ps;
    const float* w = a.w + row * a.max_pages * a.ps;
    float* w_out = a.w_out + row * a.max_pages * a.ps;
    __nv_bfloat162 mn[4], mx[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        mn[i] = __floats2bfloat162_rn(__int_as_float(0x7f800000), __int_as_float(0x7f800000));
        mx[i] = __floats2bfloat162_rn(__int_as_float(0xff800000), __int_as_float(0xff800000));
    }
    for (int s0 = 0; s0 < a.ps && j0 + s0 < m; s0 += 16) {
        const int n = min(16, m - j0 - s0);
        // lane i < n: the i-th token's old row
        long long from = -1;
        if (lane < n) {
            const int t = a.kept[row * a.budget + j0 + s0 + lane];
            const int p = a.page_table[(long long)b * a.max_pages + t / a.ps];
            if (p < 0 || p >= a.num_phys) raise_status(a.status, SPD_DEV_BAD_PAGE);
            else from = ((long long)p * a.H_kv + h) * a.ps + t % a.ps;
            w_out[j0 + s0 + lane] = w[t];
        }
        uint4 k[ACC], v[ACC];
#pragma unroll
        for (int i = 0; i < ACC; ++i) {
            const long long src = __shfl_sync(0xffffffffu, from, i * RPI + r0);
            k[i] = v[i] = make_uint4(0, 0, 0, 0);
            if (src >= 0) {
                k[i] = *(reinterpret_cast<const uint4*>(a.K) + src * LPR + ch);
                v[i] = *(reinterpret_cast<const uint4*>(a.V) + src * LPR + ch);
            }
        }
#pragma unroll
        for (int i = 0; i < ACC; ++i) {
            if (i * RPI + r0 >= n) continue;
            const long long to = (dst + s0 + i * RPI + r0) * LPR + ch;
            reinterpret_cast<uint4*>(a.K)[to] = k[i];
            reinterpret_cast<uint4*>(a.V)[to] = v[i];
            const __nv_bfloat162* e = reinterpret_cast<const __nv_bfloat162*>(&k[i]);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                mn[x] = __hmin2(mn[x], e[x]);
                mx[x] = __hmax2(mx[x], e[x]);
            }
        }
    }
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t*>(&mn[i]), off);
            const uint32_t y = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t*>(&mx[i]), off);
            mn[i] = __hmin2(mn[i], *reinterpret_cast<const __nv_bfloat162*>(&x));
            mx[i] = __hmax2(mx[i], *reinterpret_cast<const __nv_bfloat162*>(&y));
        }
    }
    if (r0 == 0) {
        uint4* out = reinterpret_cast<uint4*>(a.summ + (row * a.max_pages + page) * 2LL * D);
        out[ch] = *reinterpret_cast<uint4*>(mn);
        out[LPR + ch] = *reinterpret_cast<uint4*>(mx);
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, int num_sms, cudaStream_t st) {
    if (a.B <= 0) return cudaSuccess;
    const long long most = (long long)a.max_pages * a.ps, rows = (long long)a.B * a.H_kv;
    // CTAs of a row: with rows enough to fill the SMs, as few as hold it, three on an SM where that is enough; with fewer, up to two CTAs an
    // SM in all
    unsigned cluster = 1;
    auto holds = [&](int held) { return (long long)cluster * held >= most; };
    if (rows >= num_sms) {
        while (cluster < kMaxCluster && !holds(kHeldMany)) cluster *= 2;
    } else {
        while (cluster < kMaxCluster && (!holds(kHeld) || (long long)(2 * cluster) * rows <= 2 * num_sms)) cluster *= 2;
    }
    const bool held = holds(kHeld);
    // (a warp's tokens are a multiple of 128)
    const long long room = ((most + cluster * kWarps - 1) / (cluster * kWarps) + 127) / 128 * 128 * kWarps;
    const size_t smem = held ? (size_t)room * sizeof(uint32_t) : 0;
    static std::atomic<bool> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !known[dev].load(std::memory_order_acquire))) {
        e = cudaFuncSetAttribute(choose_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)((kHeld + 128 * kWarps) * sizeof(uint32_t)));
        if (e == cudaSuccess && dev < 64) known[dev].store(true, std::memory_order_release);
    }
    if (e != cudaSuccess) return e;
    // (an ordinary launch: CTAs that wait with their shared memory behind a call's move, or another kernel, take its L1; a run of such
    // calls over 8 rows of 65,521 tokens: 10 us less each, 27 us now)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, held ? choose_kernel<true> : choose_kernel<false>, a);
    if (e != cudaSuccess) return e;
    // no sequence has more than `budget` tokens left
    const int pages = (int)((most < a.budget ? most : a.budget) + a.ps - 1) / a.ps;
    const long long items = rows * pages;
    const dim3 grid((unsigned)((items + 3) / 4));
    auto move = a.D == 128 ? move_kernel<128> : move_kernel<64>;
    // Few items of few rows are launched early: 0.2 to 0.4 us less in a graph with up to 14 items an SM, the 4 us of a launch in a single
    // call.  From 27 to 215 items an SM early and ordinary launches are equally fast, with more the early one is up to 17 % slower (64 rows of
    // 32,768: 445 us against 379; 8 of 100,000: 169 against 161); 48 lies between.
    if (rows < num_sms && items <= 48 * num_sms) return launch_pdl(move, grid, dim3(128), 0, st, a, pages, items);
    // Where the choice or the move fills the SMs, an ordinary launch too: the rows in flight need the L1 that an SM gives back only once it has
    // no shared memory in use (64 sequences of 8K-16K tokens: 65 us less than with CTAs that are there early, 393 us now).
    cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, move, a, pages, items);
}

}  // namespace spd
