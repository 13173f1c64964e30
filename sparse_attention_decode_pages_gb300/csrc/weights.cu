// weights.cu -- the attention weight that the newest queries give to every cached token,
// added to what the token had.
//
// With lse known from the attention itself there is no softmax to carry: token t of a KV head gets
// sum_r exp(scale q_r . k_t - lse_r), so tokens are independent, nothing is joined across
// CTAs, and the order of every sum is fixed.  The keys are read once, which is what
// bounds it (the values are not needed).
//
// A CTA takes a run of tokens of one (sequence, KV head), a warp 16 of them at a time: 16 tokens' keys of a page
// come to a ring of the warp's own as one TMA box, two of them in flight, 24 warps an SM (64 sequences
// of 8K-16K tokens, paths of up to 7 nodes: 260 us, 94 % of the measured copy peak; as plain rows of 256 bytes, two on the same
// banks, 300; by loads to registers 399).
// They are the A operand of mma.m16n8k16: lane (g, c) = (lane / 4, lane % 4) reads 16-byte pieces 2 c and 2 c + 1 of
// 64 channels of tokens g and g + 8, which with the box's 128-byte swizzle lie on different banks; the contraction's order of
// channels that this gives is the one in which the queries, the B operand, are read.  Eight query rows at a time the scores of the 16 tokens are weighed and summed
// in the lanes, over the four lanes of a token at the end.  (At the memory's rate with mma.sync, so nothing would be won by the
// products in tensor memory, whose 128 rows a query tile seldom fills.)
#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace spd {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kStages = 2;  // of a warp's ring
constexpr size_t kMostSmem = 226 * 1024;
constexpr int kLeastRun = 16 * kWarps, kMostRun = 32 * kLeastRun;  // tokens of a CTA: up to 32 tiles a warp, one a lane

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
    const bool first = run == 0 && h == 0 && tid == 0;
    if (N < 0 || N > T) {
        if (first) raise_status(a.status, SPD_DEV_BAD_TREE);
        return;
    }
    if (len < N || seq_pages(len, a.ps, a.max_pages) < 0) {
        if (first) raise_status(a.status, SPD_DEV_BAD_LEN);
        return;
    }
    int bad_path = 0;
    if (a.path && tid < N) {  // (N <= 64 threads)
        const int at = a.path[(long long)b * T + tid];
        bad_path = at < 0 || at >= T;
    }
    if ((a.path || SEL) && __syncthreads_or(bad_path)) {  // (and s_pages is 0)
        if (first) raise_status(a.status, SPD_DEV_BAD_TREE);
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

template <int D>
cudaError_t launch(const WeightsArgs& a, const CUtensorMap& map, int num_sms, cudaStream_t st) {
    static std::atomic<bool> known[64][2];
    const int padded = (a.T * (a.H_q / a.H_kv) + 7) / 8 * 8;
    const size_t smem = 1024 + (size_t)kWarps * kStages * 16 * D * 2 + (size_t)padded * (D * 2 + 16 + 8);
    static_assert(1024 + kWarps * kStages * 16 * D * 2 + 8 * kTreeMax * (D * 2 + 16 + 8) <= kMostSmem, "512 query rows fit");
    auto* kern = a.sel ? weights_kernel<D, true> : weights_kernel<D, false>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !known[dev][a.sel != nullptr].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) known[dev][a.sel != nullptr].store(true, std::memory_order_release);
    }
    const long long most = (long long)a.max_pages * a.ps, rows = (long long)a.B * a.H_kv;
    auto runs_of = [&](int run) { return (most + run - 1) / run; };
    int run = kMostRun;
    // two rounds of two CTAs an SM, or more (8 sequences of 2K-4K tokens, 7 nodes: 17.2 us; as plain rows 21.2, for four
    // rounds 27.6; 64 of 8K-16K: the same)
    while (run > kLeastRun && rows * runs_of(run) < 4 * num_sms) run /= 2;
    const long long runs = runs_of(run);
    return launch_pdl(kern, dim3((unsigned)(rows * runs)), dim3(kThreads), smem, st, a, map, padded, (int)runs, run);
}

}  // namespace

cudaError_t launch_weights_update(const WeightsArgs& a, const CUtensorMap& map, int num_sms, cudaStream_t st) {
    if (a.B <= 0) return cudaSuccess;
    return a.D == 128 ? launch<128>(a, map, num_sms, st) : launch<64>(a, map, num_sms, st);
}

}  // namespace spd
