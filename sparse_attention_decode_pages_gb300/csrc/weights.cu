// weights.cu -- the attention weight that the newest queries give to every cached token,
// added to what the token had.
//
// With lse known from the attention itself there is no softmax to carry: token t of a KV head gets
// sum_r exp(scale q_r . k_t - lse_r), so tokens are independent, nothing is joined across
// CTAs, and the order of every sum is fixed.  The keys are read once, which is what
// bounds it (the values are not needed).
//
// Few query rows of a KV head: a CTA takes a run of tokens of one (sequence, KV head), a warp 16 of them at a time: 16 tokens' keys
// of a page come to a ring of the warp's own as one TMA box, two of them in flight, 24 warps an SM.
// They are the A operand of mma.m16n8k16: lane (g, c) = (lane / 4, lane % 4) reads 16-byte pieces 2 c and 2 c + 1 of
// 64 channels of tokens g and g + 8, which with the box's 128-byte swizzle lie on different banks; the contraction's order of
// channels that this gives is the one in which the queries, the B operand, are read.  Eight query rows at a time the scores of the 16 tokens are weighed and summed
// in the lanes, over the four lanes of a token at the end.  (64 sequences of 8K-16K tokens, 4 rows: 250 us, 98 % of the measured
// copy peak; one of 4,099: 6.4 us.)  More rows: tiles_kernel below (the same, 28 rows: 254 us, 97 %; by the first kernel 261).
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"

namespace spd {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kStages = 2;  // of a warp's ring
// More query rows of a KV head go through tensor memory: 16 sequences of 0 to 30,000 tokens, 28 rows 97 -> 83 us, 112 rows of half as
// many heads 75 -> 47; one sequence of 1,000, 28 rows 4.2 -> 4.8.  (16 rows: 87.4 / 82.6, but 64 sequences of 1 to 2,000 tokens 28.1 / 31.3,
// and one of 4,099 with 4 rows 6.4 / 8.3, which is the commonest call.)
constexpr int kFewRows = 16;
// So do any rows where the page table has room for this many tokens: few rows' runs follow the table's width (4 rows, 8 sequences of
// 4,000 tokens in a table for 131,072: 36 us, so 28; one of 131,001: 55, so 49).
constexpr int kWideTable = 32768;
constexpr size_t kMostSmem = 226 * 1024;
constexpr int kLeastRun = 16 * kWarps, kMostRun = 32 * kLeastRun;  // tokens of a CTA: up to 32 tiles a warp, one a lane

// The status bit of a sequence whose length or path is wrong, or 0; the same for the whole CTA.  SYNC: with a barrier of the CTA
// where length and count are right.
template <bool SYNC>
__device__ __forceinline__ unsigned wrong(const WeightsArgs& a, int b, int len, int N) {
    if (N < 0 || N > a.T) return SPD_DEV_BAD_TREE;
    if (len < N || seq_pages(len, a.ps, a.max_pages) < 0) return SPD_DEV_BAD_LEN;
    int bad_path = 0;
    if (a.path && threadIdx.x < N) {  // (N <= 64 threads)
        const int at = a.path[(long long)b * a.T + threadIdx.x];
        bad_path = at < 0 || at >= a.T;
    }
    return (a.path || SYNC) && __syncthreads_or(bad_path) ? SPD_DEV_BAD_TREE : 0;
}

template <int D, bool SEL>
__global__ void __launch_bounds__(kThreads, 3) weights_kernel(const WeightsArgs a, const __grid_constant__ CUtensorMap map, int rows_padded, int runs, int run_tokens) {
    constexpr int TILE = 16 * D * 2;
    constexpr int QROW = D * 2 + 16;  // bytes of a query row in shared memory: rows on different banks
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    uint8_t* s_q = smem + kWarps * kStages * TILE;                       // [rows_padded][QROW]
    float* s_lse = reinterpret_cast<float*>(s_q + rows_padded * QROW);   // lse * log2(e); +inf: adds nothing
    int* s_lim = reinterpret_cast<int*>(s_lse + rows_padded);            // the last position that a row sees
    __shared__ uint64_t s_full[kWarps][kStages];
    __shared__ unsigned s_pages[kMostRun / 16 / 32];                     // selected pages of the run
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int G = a.H_q / a.H_kv, T = a.T;
    const int row = blockIdx.x / runs, run = blockIdx.x - row * runs;  // (sequence, KV head) and its run
    const int b = row / a.H_kv, h = row - b * a.H_kv;
    const int t0 = run * run_tokens;
    const float INF = __int_as_float(0x7f800000);
    if (SEL && tid < kMostRun / 16 / 32) s_pages[tid] = 0;
    if (lane < kStages) mbar_init(&s_full[warp][lane], 1);
    mbar_fence_init();
    __syncwarp();
    pdl_wait();
    pdl_trigger();
    const int len = a.seq_lens[b];
    const int N = a.n_path ? a.n_path[b] : T;  // query rows' tokens
    if (const unsigned bit = wrong<SEL>(a, b, len, N)) {  // (behind it s_pages is 0)
        if (run == 0 && h == 0 && tid == 0) raise_status(a.status, bit);
        return;
    }
    if (t0 >= len) return;
    const int fresh = len - N;  // the first token without a weight of its own
    const int R = N * G, groups = (R + 7) >> 3;
    const int ntiles = (min(run_tokens, len - t0) + 15) >> 4;
    const int P = (int)(((unsigned)len + a.ps - 1) / a.ps);
    if (SEL) {
        int n = a.nsel[row];
        if (n < 0 || n > a.k_max) {
            if (run == 0 && tid == 0) raise_status(a.status, SPD_DEV_BAD_SEL);
            n = n < 0 ? 0 : a.k_max;
        }
        const int p0 = t0 / a.ps, np = (run_tokens + a.ps - 1) / a.ps;
        bool bad = false;
        for (int i = tid; i < n; i += kThreads) {
            const int p = a.sel[(long long)row * a.k_max + i];
            bad |= p < 0 || p >= P;
            if (p >= p0 && p < p0 + np) atomicOr(&s_pages[(p - p0) >> 5], 1u << ((p - p0) & 31));
        }
        if (bad && run == 0) raise_status(a.status, SPD_DEV_BAD_SEL);
        __syncthreads();
    }
    // lane i: the page of this warp's i-th tile, or -1: no keys to read
    int my_phys = -1;
    {
        const int tile = warp + kWarps * lane;
        if (tile < ntiles) {
            const int page = (t0 + tile * 16) / a.ps, in = page - t0 / a.ps;
            if (!SEL || (s_pages[in >> 5] >> (in & 31) & 1u)) {
                const int phys = a.page_table[(long long)b * a.max_pages + page];
                if (phys < 0 || phys >= a.num_phys) raise_status(a.status, SPD_DEV_BAD_PAGE);
                else my_phys = phys;
            }
        }
    }
    unsigned there = __ballot_sync(0xffffffffu, my_phys >= 0);  // tiles that are read
    const int mine = warp < ntiles ? (ntiles - warp + kWarps - 1) / kWarps : 0;
    uint8_t* ring = smem + warp * (kStages * TILE);
    auto ask = [&](int i, int slot) {  // the i-th tile's keys
        const int phys = __shfl_sync(0xffffffffu, my_phys, i);
        if (lane == 0) {
            const int at = (t0 + (warp + kWarps * i) * 16) % a.ps;
            mbar_arrive_expect_tx(&s_full[warp][slot], TILE);
            tma_load_3d(ring + slot * TILE, &map, 0, (phys * a.H_kv + h) * a.ps + at, 0, &s_full[warp][slot]);
        }
    };
    unsigned todo = there;  // tiles to ask for
    auto ask_next = [&](int slot) {
        if (!todo) return;
        ask(__ffs((int)todo) - 1, slot);
        todo &= todo - 1;
    };
    for (int i = 0; i < kStages; ++i) ask_next(i);

    bool dead = false;
    for (int i = tid; i < groups * 8 * (D / 8); i += kThreads) {
        const int r = i / (D / 8), ch = i % (D / 8), t = r / G;
        uint4 v = make_uint4(0, 0, 0, 0);
        float lse = INF;
        int lim = -1;
        if (r < R) {
            const int node = a.path ? a.path[(long long)b * T + t] : t;
            const long long at = ((long long)b * T + node) * a.H_q + h * G + (r - t * G);
            v = __ldg(reinterpret_cast<const uint4*>(a.q + at * D) + ch);
            if (ch == 0) {
                lse = a.lse[at] * kLog2e;
                dead |= lse == -INF;
                if (lse == -INF) lse = INF;
                else lim = fresh + t;
            }
        }
        *reinterpret_cast<uint4*>(s_q + r * QROW + ch * 16) = v;
        if (ch == 0) {
            s_lse[r] = lse;
            s_lim[r] = lim;
        }
    }
    // rows that add nothing see no token (an infinite key would make NaN of them): those that fill up the last group, and others
    const bool none_dead = !__syncthreads_or(dead);
    const int filled = R & 7 ? groups - 1 : -1;

    const long long wrow = (long long)row * a.max_pages * a.ps + t0;
    if (SEL) {
        // most tokens are of no selected page: their weights only decay, by all threads in a row
        __shared__ unsigned s_there[kWarps];
        if (lane == 0) s_there[warp] = there;
        __syncthreads();
        const int end = min(run_tokens, len - t0);
        constexpr int kAhead = 8;  // (w_in may be w_out: loads do not move before stores by themselves)
        for (int i0 = tid; i0 < end; i0 += kAhead * kThreads) {
            float w[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + k * kThreads;
                w[k] = a.w_in && i < end && t0 + i < fresh ? a.w_in[wrow + i] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + k * kThreads, tile = i >> 4;
                if (i < end && !(s_there[tile & (kWarps - 1)] >> (tile / kWarps) & 1u)) a.w_out[wrow + i] = a.decay * w[k];
            }
        }
    }
    // lane i < 16: the old weight of token i of a tile, asked for a tile ahead
    auto old_weight = [&](int i) {
        const int at = (warp + kWarps * i) * 16 + lane;
        return a.w_in && lane < 16 && i < mine && t0 + at < fresh ? a.w_in[wrow + at] : 0.f;
    };
    float w_next = SEL ? 0.f : old_weight(0);
    int slot = 0;
    uint32_t parity = 0;
    bool ok = true;
    for (int i = 0; i < mine; ++i) {
        if (SEL && !(there >> i & 1u)) continue;
        const int at = (warp + kWarps * i) * 16, pos = t0 + at + lane;
        float w = a.decay * (SEL ? old_weight(i) : w_next);
        if (!SEL) w_next = old_weight(i + 1);
        if (there >> i & 1u) {
            ok = __all_sync(0xffffffffu, mbar_wait_bounded(&s_full[warp][slot], parity, a.status, a.wait_ns));
            if (!ok) break;
            there &= ~(1u << i);
            uint4 k[D / 32][2];
            const uint8_t* src = ring + slot * TILE;
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                k[x][0] = *reinterpret_cast<const uint4*>(src + (x >> 1) * 2048 + swz128(g, 2 * c + (x & 1)));
                k[x][1] = *reinterpret_cast<const uint4*>(src + (x >> 1) * 2048 + 1024 + swz128(g, 2 * c + (x & 1)));
            }
            __syncwarp();  // the tile has been read
            ask_next(slot);
            if (++slot == kStages) {
                slot = 0;
                parity ^= 1u;
            }
            float sum0 = 0.f, sum1 = 0.f;  // of tokens g and g + 8
            const int p0 = t0 + at + g;
            const bool all = none_dead && t0 + at + 15 <= fresh;  // every row sees every token
            for (int j = 0; j < groups; ++j) {
                float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // (two chains of products)
                const uint8_t* q = s_q + (j * 8 + g) * QROW + c * 32;
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    const uint4 v = *reinterpret_cast<const uint4*>(q + (x >> 1) * 128 + (x & 1) * 16);
                    const uint32_t a0[4] = {k[x][0].x, k[x][1].x, k[x][0].y, k[x][1].y};
                    const uint32_t a1[4] = {k[x][0].z, k[x][1].z, k[x][0].w, k[x][1].w};
                    mma_bf16(s[0], a0, v.x, v.y);
                    mma_bf16(s[1], a1, v.z, v.w);
                }
                const float2 lse = *reinterpret_cast<const float2*>(s_lse + j * 8 + 2 * c);
                float e[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) e[x] = fast_exp2(fmaf(s[0][x] + s[1][x], a.scale_log2, x & 1 ? -lse.y : -lse.x));
                if (!all || j == filled) {
                    const int2 lim = *reinterpret_cast<const int2*>(s_lim + j * 8 + 2 * c);
                    if (p0 > lim.x) e[0] = 0.f;
                    if (p0 > lim.y) e[1] = 0.f;
                    if (p0 + 8 > lim.x) e[2] = 0.f;
                    if (p0 + 8 > lim.y) e[3] = 0.f;
                }
                sum0 += e[0] + e[1];
                sum1 += e[2] + e[3];
            }
#pragma unroll
            for (int off = 1; off < 4; off <<= 1) {
                sum0 += __shfl_xor_sync(0xffffffffu, sum0, off);
                sum1 += __shfl_xor_sync(0xffffffffu, sum1, off);
            }
            const float lo = __shfl_sync(0xffffffffu, sum0, (lane & 7) * 4), hi = __shfl_sync(0xffffffffu, sum1, (lane & 7) * 4);
            w += lane & 8 ? hi : lo;
        }
        if (lane < 16 && pos < len) a.w_out[wrow + at + lane] = w;
    }
    // copies in flight land before their memory is given back
    if (!ok)
        for (unsigned left = there & ~todo; left; left &= left - 1) {
            mbar_wait_bounded(&s_full[warp][slot], parity, a.status, a.wait_ns > kDefaultWaitNs ? a.wait_ns : kDefaultWaitNs);
            if (++slot == kStages) {
                slot = 0;
                parity ^= 1u;
            }
        }
}

// The same for many query rows: S = K Q^T on the 5th-generation tensor cores, M = 128 tokens by N = up to 128 rows, K = channels, so
// that a thread has one token (a lane of tensor memory) and adds up its rows' weights by itself.  Eight warps do that, four a
// tile of tokens, two tiles in turn; a warp copies the keys, a page a box, and one issues the products.  Two CTAs an SM.
// Bound by memory up to 128 rows (16 sequences of 16,384 tokens, 64 rows 93 us, 128 rows 105); behind that a tile's turns of products and
// weights follow one another (256 rows 246, 512 rows 472: 15 exponentials an SM and ns, a quarter of what an SM can).
constexpr int kTileThreads = 320, kTileTokens = 128, kTileRows = 128;
constexpr size_t kTileLeastSmem = 78 * 1024;  // no third CTA on an SM, whose tensor memory two share
template <int D>
struct Tiles {
    static constexpr int HALVES = D / 64, TILE = kTileTokens * D * 2, STAGES = 65536 / TILE;
    static constexpr int GROUP = HALVES * 1024;  // atoms of 8 tokens by 64 channels, a page's of all channels together
    static size_t smem(int rows) { return 1024 + STAGES * TILE + (size_t)rows * (D * 2 + 8); }
    static_assert(1024 + STAGES * TILE + 8 * kTreeMax * (D * 2 + 8) <= kMostSmem, "512 query rows fit");
};

template <int D>
__global__ void __launch_bounds__(kTileThreads, 2) tiles_kernel(const WeightsArgs a, const __grid_constant__ CUtensorMap map, int rows_padded, int runs, int parts) {
    using C = Tiles<D>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    uint8_t* s_q = smem + STAGES * C::TILE;                                       // [half][rows_padded][128 bytes], swizzled
    float* s_neg = reinterpret_cast<float*>(s_q + (size_t)rows_padded * D * 2);   // -lse * log2(e); -inf: adds nothing
    int* s_lim = reinterpret_cast<int*>(s_neg + rows_padded);                     // the last position that a row sees
    __shared__ uint64_t s_full[STAGES], s_empty[STAGES], s_done[2], s_read[2], s_drain;
    __shared__ uint32_t s_tmem;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int G = a.H_q / a.H_kv, T = a.T;
    const int row = blockIdx.x / runs, run = blockIdx.x - row * runs;  // (sequence, KV head) and its run
    const int b = row / a.H_kv, h = row - b * a.H_kv;
    const float INF = __int_as_float(0x7f800000);
    const unsigned long long drain_ns = a.wait_ns > kDefaultWaitNs ? a.wait_ns : kDefaultWaitNs;
    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(s_empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_done + i, 1);
            mbar_init(s_read + i, 4);
        }
        mbar_init(&s_drain, 1);
        mbar_fence_init();
    }
    pdl_wait();
    pdl_trigger();
    const int len = a.seq_lens[b];
    const int N = a.n_path ? a.n_path[b] : T;  // query rows' tokens
    if (const unsigned bit = wrong<false>(a, b, len, N)) {
        if (run == 0 && h == 0 && tid == 0) raise_status(a.status, bit);
        return;
    }
    // the sequence's tokens in equal runs whatever the table's width (4,000 tokens in a table for 131,072: 6.4 us; in runs of that
    // width's 19.8): as many as fill the GPU, or of 1,024 tokens, and no more than there are CTAs
    const int many = min(runs, max(parts, (len + 1023) >> 10));
    const int run_tokens = max(2 * kTileTokens, ((len + many - 1) / many + kTileTokens - 1) / kTileTokens * kTileTokens), t0 = run * run_tokens;
    if (t0 >= len) return;
    if (warp == 9) tmem_alloc(&s_tmem, 2 * kTileRows);
    const int fresh = len - N;  // the first token without a weight of its own
    const int R = N * G, rows = (R + 15) & ~15, chunks = (rows + kTileRows - 1) / kTileRows;
    const int ntiles = (min(run_tokens, len - t0) + kTileTokens - 1) / kTileTokens;
    bool dead = false;
    for (int i = tid; i < rows * (D / 8); i += kTileThreads) {
        const int r = i / (D / 8), ch = i % (D / 8), t = r / G;
        uint4 v = make_uint4(0, 0, 0, 0);
        float neg = -INF;
        int lim = -1;
        if (r < R) {
            const int node = a.path ? a.path[(long long)b * T + t] : t;
            const long long at = ((long long)b * T + node) * a.H_q + h * G + (r - t * G);
            v = __ldg(reinterpret_cast<const uint4*>(a.q + at * D) + ch);
            if (ch == 0) {
                neg = -kLog2e * a.lse[at];
                dead |= neg == INF;
                if (neg == INF) neg = -INF;
                else lim = fresh + t;
            }
        }
        *reinterpret_cast<uint4*>(s_q + (size_t)(ch >> 3) * rows_padded * 128 + swz128(r, ch & 7)) = v;
        if (ch == 0) {
            s_neg[r] = neg;
            s_lim[r] = lim;
        }
    }
    async_proxy_fence();
    tmem_fence_before();
    // rows that add nothing see no token (an infinite key would make NaN of them): those that fill up the last 16, and others
    const bool none_dead = !__syncthreads_or(dead);
    tmem_fence_after();
    const uint32_t tmem = s_tmem;
    const int32_t* table = a.page_table + (long long)b * a.max_pages;
    const int lg_ps = __ffs(a.ps) - 1;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, a.status, a.wait_ns));
        return ok;
    };
    if (warp < 8) {
        // ======================================================== weights
        const int g = warp >> 2;
        const uint32_t tm = tmem + g * kTileRows + ((uint32_t)((warp & 3) * 32) << 16);
        const long long wrow = (long long)row * a.max_pages * a.ps;
        const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
        uint32_t parity = 0;
        for (int i = g; i < ntiles; i += 2) {
            const int first = t0 + i * kTileTokens, pos = first + (warp & 3) * 32 + lane;
            float old = 0.f;
            int phys = 0;
            if (pos < len) {
                phys = table[pos >> lg_ps];
                if (a.w_in && pos < fresh) old = a.w_in[wrow + pos];
            }
            const bool all = none_dead && first + kTileTokens - 1 <= fresh;  // every row sees every token
            float2 sum0 = make_float2(0.f, 0.f), sum1 = sum0;
            for (int c = 0; c < chunks; ++c) {
                if (!wait(s_done + g, parity)) break;
                parity ^= 1u;
                tmem_fence_after();
                const int end = min(kTileRows, rows - c * kTileRows);
#pragma unroll 2
                for (int x = 0; x < end; x += 16) {
                    uint32_t v[16];
                    tmem_ld(tm + x, v);
                    const int r = c * kTileRows + x;
                    tmem_wait_ld();
                    tmem_loaded(v);
                    const bool mask = !all || r + 16 > R;
#pragma unroll
                    for (int k = 0; k < 16; k += 4) {
                        const float4 neg = *reinterpret_cast<const float4*>(s_neg + r + k);
                        const float2 y0 = fma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), scale2, make_float2(neg.x, neg.y));
                        const float2 y1 = fma2(make_float2(__uint_as_float(v[k + 2]), __uint_as_float(v[k + 3])), scale2, make_float2(neg.z, neg.w));
                        float2 e0 = make_float2(fast_exp2(y0.x), fast_exp2(y0.y)), e1 = make_float2(fast_exp2(y1.x), fast_exp2(y1.y));
                        if (mask) {
                            const int4 lim = *reinterpret_cast<const int4*>(s_lim + r + k);
                            if (pos > lim.x) e0.x = 0.f;
                            if (pos > lim.y) e0.y = 0.f;
                            if (pos > lim.z) e1.x = 0.f;
                            if (pos > lim.w) e1.y = 0.f;
                        }
                        sum0 = add2(sum0, e0);
                        sum1 = add2(sum1, e1);
                    }
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_read + g);
            }
            if (!ok) break;
            if (pos < len) {
                const bool there = phys >= 0 && phys < a.num_phys;
                if (!there) raise_status(a.status, SPD_DEV_BAD_PAGE);
                a.w_out[wrow + pos] = a.decay * old + (there ? (sum0.x + sum0.y) + (sum1.x + sum1.y) : 0.f);
            }
        }
    } else if (warp == 8 && R > 0) {
        // ======================================================== copies
        const int ppt = kTileTokens >> lg_ps, P = (int)(((unsigned)len + a.ps - 1) >> lg_ps);
        const int none = (int)max(1LL, a.num_phys * a.H_kv);  // a row of pages that is not there: zeros
        auto ask = [&](int i) {
            const int page = (t0 >> lg_ps) + i * ppt + (lane & (ppt - 1));
            return i < ntiles && page < P ? table[page] : -1;
        };
        int next = ask(0), asked = 0;
        for (int i = 0; i < ntiles; ++i) {
            const int slot = i % STAGES, phys = next;
            next = ask(i + 1);
            if (!wait(s_empty + slot, ((uint32_t)(i / STAGES) & 1u) ^ 1u)) break;
            asked = i + 1;
            if (lane == 0) mbar_arrive_expect_tx(s_full + slot, C::TILE);
            __syncwarp();
            if (lane < ppt)
                tma_load_5d(smem + slot * C::TILE + lane * a.ps * (D * 2), &map, 0, 0, 0, 0, phys >= 0 && phys < a.num_phys ? phys * a.H_kv + h : none, s_full + slot);
        }
        // copies land before their memory is given back, whoever has waited for them
        for (int k = max(0, asked - STAGES); k < asked; ++k) mbar_wait_bounded(s_full + k % STAGES, (uint32_t)(k / STAGES) & 1u, a.status, drain_ns);
    } else if (warp == 9 && R > 0) {
        // ======================================================== products
        const uint32_t k_smem = smem_u32(smem), q_smem = smem_u32(s_q);
        uint32_t read_parity = 3;  // (of both halves of tensor memory: bits)
        for (int i = 0; i < ntiles && ok; i += 2)
            for (int c = 0; c < chunks && ok; ++c)
                for (int g = 0; g < 2 && i + g < ntiles; ++g) {
                    const int slot = (i + g) % STAGES;
                    if (c == 0 && !wait(s_full + slot, (uint32_t)((i + g) / STAGES) & 1u)) break;
                    if (!wait(s_read + g, read_parity >> g & 1u)) break;
                    read_parity ^= 1u << g;
                    tmem_fence_after();
                    if (elect_one()) {
                        const uint32_t idesc = umma_idesc_bf16(kTileTokens, min(kTileRows, rows - c * kTileRows), false, false);
                        const uint64_t dk = umma_desc(k_smem + slot * C::TILE, 0, C::GROUP, kSwizzle128);
                        const uint64_t dq = umma_desc(q_smem + c * kTileRows * 128, 0, 1024, kSwizzle128);
#pragma unroll
                        for (int x = 0; x < D / 16; ++x)
                            umma_f16_ss(tmem + g * kTileRows, dk + (((x >> 2) * 1024 + (x & 3) * 32) >> 4), dq + (((x >> 2) * rows_padded * 128 + (x & 3) * 32) >> 4), idesc,
                                        x > 0);
                        umma_commit(s_done + g);
                        if (c + 1 == chunks) umma_commit(s_empty + slot);
                    }
                    __syncwarp();
                }
        if (!ok) {  // products in flight end before their memory is given back
            if (elect_one()) umma_commit(&s_drain);
            __syncwarp();
            mbar_wait_bounded(&s_drain, 0, a.status, drain_ns);
        }
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == 9) tmem_free(tmem, 2 * kTileRows);
}

template <int D>
cudaError_t launch(const WeightsArgs& a, const CUtensorMap& map, int num_sms, cudaStream_t st) {
    static std::atomic<bool> known[64][3];
    const bool tiles = weights_by_tiles(a.T, a.H_q / a.H_kv, a.sel != nullptr, (long long)a.max_pages * a.ps);
    const int kind = tiles ? 2 : a.sel ? 1 : 0, step = tiles ? 16 : 8;
    const int padded = (a.T * (a.H_q / a.H_kv) + step - 1) / step * step;
    size_t smem = 1024 + (size_t)kWarps * kStages * 16 * D * 2 + (size_t)padded * (D * 2 + 16 + 8);
    static_assert(1024 + kWarps * kStages * 16 * D * 2 + 8 * kTreeMax * (D * 2 + 16 + 8) <= kMostSmem, "512 query rows fit");
    if (tiles) smem = Tiles<D>::smem(padded) > kTileLeastSmem ? Tiles<D>::smem(padded) : kTileLeastSmem;
    auto* kern = tiles ? tiles_kernel<D> : a.sel ? weights_kernel<D, true> : weights_kernel<D, false>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !known[dev][kind].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) known[dev][kind].store(true, std::memory_order_release);
    }
    const long long most = (long long)a.max_pages * a.ps, rows = (long long)a.B * a.H_kv;
    auto runs_of = [&](int run) { return (most + run - 1) / run; };
    int run = kMostRun;
    // two rounds of two CTAs an SM, or more (8 sequences of 2K-4K tokens, 4 rows: 17 us; for four rounds 27.6; 64 of 8K-16K: the same);
    // of the tiles' CTAs, which start more slowly, one an SM (8 sequences of 2K-4K tokens, 28 rows: 15.7 us; two an SM 17.9, four 21.5)
    while (run > (tiles ? 2 * kTileTokens : kLeastRun) && rows * runs_of(run) < (tiles ? 1 : 4) * num_sms) run /= 2;
    long long runs = runs_of(run), parts = run;
    if (tiles) {  // (a CTA without tokens costs some 0.1 us on each SM: a wide table's rows have fewer CTAs, with longer runs)
        parts = (2 * num_sms + rows - 1) / rows;
        const long long enough = 16LL * num_sms / rows > parts ? 16LL * num_sms / rows : parts;
        if (runs > enough) runs = enough;
    }
    return launch_pdl(kern, dim3((unsigned)(rows * runs)), dim3(tiles ? kTileThreads : kThreads), smem, st, a, map, padded, (int)runs, (int)parts);
}

}  // namespace

bool weights_by_tiles(int T, int G, bool selected, long long most) { return !selected && (T * G > kFewRows || most >= kWideTable); }

cudaError_t launch_weights_update(const WeightsArgs& a, const CUtensorMap& map, int num_sms, cudaStream_t st) {
    if (a.B <= 0) return cudaSuccess;
    return a.D == 128 ? launch<128>(a, map, num_sms, st) : launch<64>(a, map, num_sms, st);
}

}  // namespace spd
