// weights.cu -- the attention weight that the newest queries give to every cached token,
// added to what the token had.
//
// With lse known from the attention itself there is no softmax to carry: token t of a KV head gets
// sum_r exp(scale q_r . k_t - lse_r), so tokens are independent, nothing is joined across
// CTAs, and the order of every sum is fixed.  The keys are read once, which is what
// bounds it (the values are not needed).
//
// A CTA takes a run of tokens of one (sequence, KV head); a warp 16 of them at a time: their keys go from
// global memory to registers as the A operand of mma.m16n8k16 (lane (g, c) = (lane / 4,
// lane % 4) loads 16 bytes, channels 32 i + 8 c ..., of tokens g and g + 8; the contraction's order of
// channels that this gives is the one in which the queries, the B operand, are read from
// shared memory), the next 16 tokens' keys are in flight meanwhile.  Eight query rows at a time the scores
// of the 16 tokens are weighed and summed in the lanes, over the four lanes of a token at the end.
#include "common.cuh"
#include "kernels.h"

namespace spd {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kRun = 512;  // tokens of a CTA: a multiple of 16 * kWarps and of the page sizes

template <int D>
struct Tile {
    uint4 k[D / 32][2];  // channels 32 i + 8 c ... of tokens g and g + 8
};

template <int D, bool SEL>
__global__ void __launch_bounds__(kThreads) weights_kernel(const WeightsArgs a, int rows_padded, int runs) {
    constexpr int QROW = D * 2 + 16;  // bytes of a query row in shared memory: rows on different banks
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t* s_q = smem;                                                    // [rows_padded][QROW]
    float* s_lse = reinterpret_cast<float*>(smem + rows_padded * QROW);     // lse * log2(e); +inf: adds nothing
    int* s_lim = reinterpret_cast<int*>(s_lse + rows_padded);               // the last position that a row sees
    __shared__ unsigned s_pages;                                            // selected pages of the run
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int G = a.H_q / a.H_kv, T = a.T;
    const int row = blockIdx.x / runs, run = blockIdx.x - row * runs;  // (sequence, KV head) and its run
    const int b = row / a.H_kv, h = row - b * a.H_kv;
    const int t0 = run * kRun;
    const float INF = __int_as_float(0x7f800000);
    if (SEL && tid == 0) s_pages = 0;
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
    if (a.path) {
        int bad = 0;
        for (int i = tid; i < N; i += kThreads) {
            const int at = a.path[(long long)b * T + i];
            bad |= at < 0 || at >= T;
        }
        if (__syncthreads_or(bad)) {
            if (first) raise_status(a.status, SPD_DEV_BAD_TREE);
            return;
        }
    }
    if (t0 >= len) return;
    const int fresh = len - N;  // the first token without a weight of its own
    const int R = N * G, groups = (R + 7) >> 3;
    const long long table = (long long)b * a.max_pages;

    // this warp's first keys are asked for before the queries are brought in
    const int ntiles = (min(kRun, len - t0) + 15) >> 4;
    const int P = (int)(((unsigned)len + a.ps - 1) / a.ps);
    if (SEL) {
        __syncthreads();  // s_pages is 0
        int n = a.nsel[row];
        if (n < 0 || n > a.k_max) {
            if (run == 0 && tid == 0) raise_status(a.status, SPD_DEV_BAD_SEL);
            n = n < 0 ? 0 : a.k_max;
        }
        const int p0 = t0 / a.ps;
        bool bad = false;
        for (int i = tid; i < n; i += kThreads) {
            const int p = a.sel[(long long)row * a.k_max + i];
            bad |= p < 0 || p >= P;
            if (p >= p0 && p < p0 + kRun / a.ps) atomicOr(&s_pages, 1u << (p - p0));
        }
        if (bad && run == 0) raise_status(a.status, SPD_DEV_BAD_SEL);
        __syncthreads();
    }
    auto page_of = [&](int tile) {  // its page-table entry, or -1: no keys to read
        if (tile >= ntiles) return -1;
        const int page = (t0 + tile * 16) / a.ps;
        if (SEL && !(s_pages >> (page - t0 / a.ps) & 1u)) return -1;
        const int phys = a.page_table[table + page];
        if (phys < 0 || phys >= a.num_phys) {
            raise_status(a.status, SPD_DEV_BAD_PAGE);
            return -1;
        }
        return phys;
    };
    auto load = [&](int tile, int phys, Tile<D>& x) {
        if (phys < 0) return;
        const int slot = (t0 + tile * 16) % a.ps;
        const uint8_t* src = reinterpret_cast<const uint8_t*>(a.K) + ((((long long)phys * a.H_kv + h) * a.ps + slot + g) * D + 8 * c) * 2;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            x.k[i][0] = __ldg(reinterpret_cast<const uint4*>(src + i * 64));
            x.k[i][1] = __ldg(reinterpret_cast<const uint4*>(src + i * 64 + 8 * D * 2));
        }
    };
    Tile<D> cur, nxt;
    int phys = page_of(warp);
    load(warp, phys, cur);
    int phys_next = page_of(warp + kWarps);

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
                if (lse == -INF) lse = INF;
                lim = fresh + t;
            }
        }
        *reinterpret_cast<uint4*>(s_q + r * QROW + ch * 16) = v;
        if (ch == 0) {
            s_lse[r] = lse;
            s_lim[r] = lim;
        }
    }
    __syncthreads();

    const long long wrow = (long long)row * a.max_pages * a.ps + t0;
    for (int tile = warp; tile < ntiles; tile += kWarps) {
        // the old weight: lane i < 16 keeps that of token i
        const int pos = t0 + tile * 16 + lane;
        float w = 0.f;
        if (a.w_in && lane < 16 && pos < fresh) w = a.decay * a.w_in[wrow + tile * 16 + lane];
        load(tile + kWarps, phys_next, nxt);
        const int phys_after = page_of(tile + 2 * kWarps);
        if (phys >= 0) {
            float sum0 = 0.f, sum1 = 0.f;  // of tokens g and g + 8
            const int p0 = t0 + tile * 16 + g;
            const bool all = t0 + tile * 16 + 15 <= fresh;  // every row sees every token
            for (int j = 0; j < groups; ++j) {
                float s[4] = {0.f, 0.f, 0.f, 0.f};
                const uint8_t* q = s_q + (j * 8 + g) * QROW + c * 16;
#pragma unroll
                for (int i = 0; i < D / 32; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4*>(q + i * 64);
                    const uint32_t a0[4] = {cur.k[i][0].x, cur.k[i][1].x, cur.k[i][0].y, cur.k[i][1].y};
                    const uint32_t a1[4] = {cur.k[i][0].z, cur.k[i][1].z, cur.k[i][0].w, cur.k[i][1].w};
                    mma_bf16(s, a0, v.x, v.y);
                    mma_bf16(s, a1, v.z, v.w);
                }
                const float2 lse = *reinterpret_cast<const float2*>(s_lse + j * 8 + 2 * c);
                float e[4] = {fast_exp2(fmaf(s[0], a.scale_log2, -lse.x)), fast_exp2(fmaf(s[1], a.scale_log2, -lse.y)),
                              fast_exp2(fmaf(s[2], a.scale_log2, -lse.x)), fast_exp2(fmaf(s[3], a.scale_log2, -lse.y))};
                if (!all) {
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
        if (lane < 16 && pos < len) a.w_out[wrow + tile * 16 + lane] = w;
        cur = nxt;
        phys = phys_next;
        phys_next = phys_after;
    }
}

template <int D>
cudaError_t launch(const WeightsArgs& a, cudaStream_t st) {
    const int padded = (a.T * (a.H_q / a.H_kv) + 7) / 8 * 8;
    const size_t smem = (size_t)padded * (D * 2 + 16 + 8);
    auto* kern = a.sel ? weights_kernel<D, true> : weights_kernel<D, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const long long runs = ((long long)a.max_pages * a.ps + kRun - 1) / kRun;
    return launch_pdl(kern, dim3((unsigned)(runs * a.B * a.H_kv)), dim3(kThreads), smem, st, a, padded, (int)runs);
}

}  // namespace

cudaError_t launch_weights_update(const WeightsArgs& a, cudaStream_t st) {
    if (a.B <= 0) return cudaSuccess;
    return a.D == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace spd
