// attn4.cu -- attention over the 4-bit paged cache: sparse decode over the selected
// pages and dense causal verification over the whole cache.
//
// A unit is a run of at most pages_per_split pages of one (sequence, KV head) row;
// it holds all R = T * G query rows of the KV head in n-tiles of eight.  A CTA of four
// warps takes one unit, 64 tokens (a step) at a time from a ring that bulk copies fill.
// On the tensor cores (mma.sync m16n8k16, fp16 in, fp32 out):
//
//   S^T = K Q^T        warp w: the step's 16-token chunk w, every query row
//   O^T += V^T P^T     warp w: channels (w & 1) * D / 2 ... of chunks 2 (w >> 1), + 1
//
// so tokens and channels fill the MMA rows and the few query rows its columns, every
// key and value is converted to fp16 once in the CTA, and a warp holds half of O (64
// registers at 32 query rows; the two halves of the tokens are joined at the end); P
// goes between the warps through shared memory as ready B fragments.  Two barriers a
// step: one carries the vote on the references, one publishes P.
// Warp k % 4 issues step k's copies, a lane for each piece, from what its lanes have
// resolved (selection entry, page-table entry) for its next eight steps.
//
// code * scale is exact in fp16, so the products are those of the values the cache
// stands for.  The contraction's channel order is free: lane (g, c) = (lane / 4,
// lane % 4) holds the D / 4 channels from c * D / 4 on of tokens g and g + 8,
// contiguous in memory; of V it holds D / 16 neighbouring channels of tokens 2c, 2c+1,
// 2c+8, 2c+9 -- in a chunk's tokens taken in the order 0 1 3 2 4 5 7 6, 8 ..., with which
// neither the 64-byte key rows nor the 32-byte slices of the value rows that are read
// together share banks more than twice.  Queries are scaled by a power of two into fp16's range (the factor goes
// into the logits' scale).  Online softmax in fp32 in base 2; a column's reference
// moves only when a logit exceeds it by kHead4, and weights carry a factor 2^kBias4 so
// that what fp16 drops of a weight lies 2^-32 below the reference.
#include <atomic>

#include "kv4.cuh"
#include "kernels.h"

namespace spd {

constexpr float kHead4 = 8.f;  // log2 headroom before the running maximum moves
constexpr float kBias4 = 7.f;  // 2^(kHead4 + kBias4) = 32768 stays within fp16

// Without `volatile`: the compiler may order these among the conversions.
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// The token of MMA row r (0-7; r + 8 likewise) of a chunk.
__device__ __forceinline__ int chunk_token(int r) { return r ^ ((r >> 1) & 1); }

constexpr float kLow4 = -3.0e38f;  // a column's reference before its first visible token

template <int D, int NT>
struct Attn4Cfg {
    static constexpr int WARPS = 4, THREADS = 128;
    static constexpr int COLS = NT * 8;
    static constexpr int STAGES = 4;                      // steps in the ring
    static constexpr int CHUNK = kv4_tile_bytes(16, D);   // bytes of 16 tokens' keys and values
    static constexpr int STEP = WARPS * CHUNK;
    static constexpr bool QREG = NT == 1;                 // Q's fragments stay in registers (else in shared memory)
    // half [NT][D / 32][32 lanes][8]: B fragments of Q^T, 16 bytes for each lane and code word
    static constexpr int OFF_Q = STAGES * STEP;
    static constexpr int OFF_P = OFF_Q + COLS * D * 2;    // uint2 [WARPS][NT][32 lanes]: B fragments of P^T
    static constexpr int OFF_FAC = OFF_P + WARPS * NT * 256;  // float [COLS]: logit scale of each query row
    static constexpr int OFF_RED = OFF_FAC + COLS * 4;        // float [WARPS][COLS]: maxima, then sums
    static constexpr int OFF_BAR = OFF_RED + WARPS * COLS * 4;  // uint64 [STAGES]
    static constexpr int OFF_META = OFF_BAR + STAGES * 8;       // int4 [STAGES]: the chunks' first positions or -1
    static constexpr int SMEM = OFF_META + STAGES * 16;
    static constexpr int OCC = NT <= 2 ? 4 : (NT == 4 ? 3 : 2);  // CTAs on an SM
    static_assert(COLS * D * 4 <= STAGES * STEP, "half of O is handed over in the ring");
    static_assert(STAGES - 1 <= WARPS, "a warp issues one of the first steps");
    static_assert(STAGES % 2 == 0, "meta is 16-byte aligned");
};

template <int D, int NT, bool SPARSE>
__global__ void __launch_bounds__(128, Attn4Cfg<D, NT>::OCC) attn4_kernel(const Attn4Args a) {
    using C = Attn4Cfg<D, NT>;
    constexpr int COLS = C::COLS, STAGES = C::STAGES, WARPS = C::WARPS;
    constexpr int KW = D / 32;   // 32-bit code words of a lane's share of a key row
    constexpr int MT = D / 32;   // 16-channel m-tiles of a warp's half of O^T
    constexpr int CODES = kv4_codes_bytes(16, D), HALF = kv4_half_bytes(16, D);  // of a chunk
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_last, s_late;
    float* s_fac = reinterpret_cast<float*>(smem + C::OFF_FAC);
    float* s_red = reinterpret_cast<float*>(smem + C::OFF_RED);
    __half* s_q = reinterpret_cast<__half*>(smem + C::OFF_Q);
    uint2* s_p = reinterpret_cast<uint2*>(smem + C::OFF_P);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    int4* meta = reinterpret_cast<int4*>(smem + C::OFF_META);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int chalf = warp & 1, tpair = warp >> 1;  // this warp's half of the channels and pair of chunks of O
    const int gt = chunk_token(g);  // the token of the lane's first key row; the second is 8 behind
    const int G = a.H_q / a.H_kv, R = a.T * G;
    const float NEG_INF = __int_as_float(0xff800000);

    const int row = blockIdx.x / a.num_splits, split = blockIdx.x % a.num_splits;
    const int b = row / a.H_kv, h = row - b * a.H_kv;
    auto out_index = [&](int r) -> long long {
        const int t = r / G;
        return ((long long)b * a.T + t) * a.H_q + h * G + (r - t * G);
    };
    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) mbar_init(full + i, 1);
        mbar_fence_init();
        s_late = 0;
    }
    pdl_wait();
    pdl_trigger();

    const int start = split * a.pages_per_split;
    const int cpp = a.ps >> 4;  // chunks per page
    // this warp issues steps 4 m + warp; lane i resolves chunk i % 4 of its step m = base + i / 4.
    // The first selection entries are read together with the lengths.
    auto chunk_of = [&](int m) { return 16 * (m + (lane >> 2)) + 4 * warp + (lane & 3); };
    int lp_next = -1, ph_next = -1;  // the next eight steps' logical pages and page-table entries, unchecked
    if (SPARSE && chunk_of(0) / cpp < a.k_max - start) lp_next = a.sel[(long long)row * a.k_max + start + chunk_of(0) / cpp];
    const int len = a.seq_lens[b];
    int P = seq_pages(len, a.ps, a.max_pages);
    if (P < 0) {
        if (tid == 0) raise_status(a.status, SPD_DEV_BAD_LEN);
        P = 0;
    }
    int n_items = P;
    if (SPARSE) {
        n_items = a.nsel[row];
        if (n_items < 0 || n_items > a.k_max) {
            if (tid == 0) raise_status(a.status, SPD_DEV_BAD_SEL);
            n_items = n_items < 0 ? 0 : a.k_max;
        }
    }
    const int count = min(a.pages_per_split, n_items - start);
    if (count <= 0) {
        if (split == 0)
            for (int i = tid; i < R * (D / 8); i += C::THREADS) {
                const long long oi = out_index(i / (D / 8));
                *reinterpret_cast<uint4*>(a.o + oi * D + (i % (D / 8)) * 8) = make_uint4(0, 0, 0, 0);
                if (i % (D / 8) == 0 && a.lse) a.lse[oi] = NEG_INF;
            }
        return;
    }
    const int nsplit = (n_items + a.pages_per_split - 1) / a.pages_per_split;
    const int chunks = count * cpp;
    const int steps = (chunks + WARPS - 1) / WARPS;

    auto next_pages = [&](int m) {
        const int ci = chunk_of(m);
        lp_next = -1;
        if (ci < chunks) lp_next = SPARSE ? a.sel[(long long)row * a.k_max + start + ci / cpp] : start + ci / cpp;
    };
    auto next_entries = [&]() {
        ph_next = lp_next >= 0 && lp_next < P ? a.page_table[(long long)b * a.max_pages + lp_next] : -1;
    };
    int ph_cur = -1, pos_cur = -1;  // physical page and first position (-1: nothing to read)
    auto take_next = [&](int m) {
        const int ci = chunk_of(m);
        ph_cur = pos_cur = -1;
        if (ci < chunks) {
            if (lp_next < 0 || lp_next >= P) {
                raise_status(a.status, SPD_DEV_BAD_SEL);
            } else if (ph_next < 0 || ph_next >= a.num_phys) {
                raise_status(a.status, SPD_DEV_BAD_PAGE);
            } else {
                const int at = lp_next * a.ps + (ci - ci / cpp * cpp) * 16;
                if (at < len) {
                    ph_cur = ph_next;
                    pos_cur = at;
                }
            }
        }
    };
    // issues step k (k % 4 == warp): lane 4 q + i copies piece i of chunk q (keys' codes and
    // scales, values' codes and scales), or lane 4 q the whole chunk where a page is one
    const int codes = kv4_codes_bytes(a.ps, D), half = kv4_half_bytes(a.ps, D);
    auto issue = [&](int k) {
        const int slot = k % STAGES, from = (k >> 2 & 7) * 4;
        const int phys = __shfl_sync(0xffffffffu, ph_cur, from + (lane >> 2 & 3));
        const int pos = __shfl_sync(0xffffffffu, pos_cur, from + (lane >> 2 & 3));
        const unsigned there = __ballot_sync(0xffffffffu, pos >= 0 && (lane & 3) == 0 && lane < 16);
        if (lane < 16 && (lane & 3) == 0) reinterpret_cast<int*>(meta + slot)[lane >> 2] = pos;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full + slot, __popc(there) * C::CHUNK);
        __syncwarp();
        if (lane < 16 && pos >= 0) {
            const int i = lane & 3;
            const uint8_t* tile = a.kv4 + ((long long)phys * a.H_kv + h) * (2LL * half);
            uint8_t* dst = smem + slot * C::STEP + (lane >> 2) * C::CHUNK;
            if (a.ps == 16) {
                if (i == 0) bulk_load(dst, tile, C::CHUNK, full + slot);
            } else {
                const int t0 = pos & (a.ps - 1);
                const uint8_t* src = tile + (i >> 1) * half + (i & 1 ? codes + t0 * (D / 16) : t0 * (D / 2));
                bulk_load(dst + (i >> 1) * HALF + (i & 1) * CODES, src, i & 1 ? HALF - CODES : CODES, full + slot);
            }
        }
    };
    if (!SPARSE) next_pages(0);
    next_entries();
    take_next(0);
    __syncthreads();  // the barriers are initialised
    if (warp < STAGES - 1 && warp < steps) issue(warp);
    if (steps > 32) next_pages(8);

    // the query rows in fp16, each scaled by 2^-e so that its largest channel lies in [1, 2),
    // stored as the lanes read them: two channels of a row for each lane and turn here
    for (int r = warp; r < COLS; r += WARPS) {
        float2 x[D / 64];
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            x[i] = make_float2(0.f, 0.f);
            if (r < R)
                x[i] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(a.q + out_index(r) * D + 2 * lane + 64 * i));
            amax = fmaxf(amax, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        int e = (int)(__float_as_uint(amax) >> 23) - 127;
        if (e > 126 || e < -126) e = e > 126 ? 126 : -126;
        if (amax == 0.f) e = 0;
        const float down = pow2f(-e);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const int ch = 2 * lane + 64 * i, qc = ch / (D / 4), w = ch % (D / 4) / 8;
            *reinterpret_cast<uint32_t*>(s_q + (((r >> 3) * KW + w) * 32 + (r & 7) * 4 + qc) * 8 + ch % 8) =
                pack_f16(x[i].x * down, x[i].y * down);
        }
        if (lane == 0) s_fac[r] = a.scale_log2 * pow2f(e);
    }
    __syncthreads();

    auto q_frag = [&](int n, int w) { return *reinterpret_cast<const uint4*>(s_q + ((n * KW + w) * 32 + lane) * 8); };
    uint4 qf[C::QREG ? KW : 1];
    if constexpr (C::QREG) {
#pragma unroll
        for (int w = 0; w < KW; ++w) qf[w] = q_frag(0, w);
    }
    float fac[NT][2], ref[NT][2], l[NT][2];  // ref: the reference less kBias4
    float oacc[NT][MT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            fac[n][j] = s_fac[n * 8 + 2 * c + j];
            ref[n][j] = kLow4;
            l[n][j] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) oacc[n][i][0] = oacc[n][i][1] = oacc[n][i][2] = oacc[n][i][3] = 0.f;
    }

    for (int k = 0; k < steps; ++k) {
        const int slot = k % STAGES;
        const uint8_t* stage = smem + slot * C::STEP;
        const bool landed = mbar_wait_bounded(full + slot, (uint32_t)(k / STAGES) & 1u, a.status, a.wait_ns);
        const int4 firsts = meta[slot];
        const int pos0 = warp == 0 ? firsts.x : warp == 1 ? firsts.y : warp == 2 ? firsts.z : firsts.w;
        float sc[NT][4], y[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
        float top = NEG_INF;
        if (pos0 >= 0) {
            const uint8_t* kt = stage + warp * C::CHUNK;
            uint32_t kw[2][KW], ks[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = gt + 8 * j;
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4*>(kt + t * 64 + c * 16);
                    kw[j][0] = x.x;
                    kw[j][1] = x.y;
                    kw[j][KW - 2] = x.z;
                    kw[j][KW - 1] = x.w;
                    ks[j] = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(kt + CODES + t * 8 + 2 * c));
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(kt + t * 32 + c * 8);
                    kw[j][0] = x.x;
                    kw[j][1] = x.y;
                    ks[j] = e4m3x2_to_f16(kt[CODES + t * 4 + c]);
                }
            }
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                uint32_t h0[4], h1[4];
                e2m1x8_to_f16(kw[0][w], h0);
                e2m1x8_to_f16(kw[1][w], h1);
                const uint32_t s0 = __byte_perm(ks[0], 0, w < 2 ? 0x1010 : 0x3232), s1 = __byte_perm(ks[1], 0, w < 2 ? 0x1010 : 0x3232);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h0[i] = hmul2(h0[i], s0);
                    h1[i] = hmul2(h1[i], s1);
                }
                const uint32_t a0[4] = {h0[0], h1[0], h0[1], h1[1]}, a1[4] = {h0[2], h1[2], h0[3], h1[3]};
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 q = C::QREG ? qf[C::QREG ? w : 0] : q_frag(n, w);
                    mma_f16(sc[n], a0, q.x, q.y);
                    mma_f16(sc[n], a1, q.z, q.w);
                }
            }
            // y: logits in base 2 less ref, hidden tokens at -inf
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) y[n][j] = fmaf(sc[n][j], fac[n][j & 1], -ref[n][j & 1]);
            if (pos0 + 15 > len - a.T) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = n * 8 + 2 * c + (j & 1);
                        const int lim = r < R ? len - a.T + r / G : len - 1;  // the last token that the row sees
                        if (pos0 + gt + 8 * (j >> 1) > lim) y[n][j] = NEG_INF;
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) top = fmaxf(fmaxf(fmaxf(y[n][0], y[n][1]), fmaxf(y[n][2], y[n][3])), top);
        } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) y[n][0] = y[n][1] = y[n][2] = y[n][3] = NEG_INF;
        }
        if (!landed) s_late = 1;
        // every warp is done with step k - 1 behind this; the vote: some reference has to move
        const bool move = __syncthreads_or(top > kHead4 + kBias4);
        if (s_late) {  // the copies in flight land before the CTA ends; the row is given up
            for (int j = k; j < min(k + STAGES - 1, steps); ++j)
                mbar_wait_bounded(full + j % STAGES, (uint32_t)(j / STAGES) & 1u, a.status, a.wait_ns);
            break;
        }
        const int kn = k + STAGES - 1;  // into the slot of step k - 1
        if (kn < steps && (kn & 3) == warp) {
            if (kn >= 32 && (kn & 28) == 0) {  // this warp's next eight steps
                take_next(kn >> 2);
                next_pages((kn >> 2) + 8);
            } else if ((kn & 28) == 8) {
                next_entries();
            }
            issue(kn);
        }
        if (move) {
            // from the logits themselves: an unset reference leaves nothing of them in y
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = fmaxf(y[n][j] == NEG_INF ? NEG_INF : sc[n][j] * fac[n][j],
                                    y[n][j + 2] == NEG_INF ? NEG_INF : sc[n][j + 2] * fac[n][j]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
                    if (g == 0) s_red[warp * COLS + n * 8 + 2 * c + j] = x;
                }
            }
            __syncthreads();
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = NEG_INF;
#pragma unroll
                    for (int i = 0; i < WARPS; ++i) x = fmaxf(x, s_red[i * COLS + n * 8 + 2 * c + j]);
                    x = fmaxf(ref[n][j], x - kBias4);
                    const float corr = fast_exp2(ref[n][j] - x);
                    ref[n][j] = x;
                    if (y[n][j] != NEG_INF) y[n][j] = fmaf(sc[n][j], fac[n][j], -x);
                    if (y[n][j + 2] != NEG_INF) y[n][j + 2] = fmaf(sc[n][j + 2], fac[n][j], -x);
                    l[n][j] *= corr;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        oacc[n][i][j] *= corr;
                        oacc[n][i][j + 2] *= corr;
                    }
                }
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                p[j] = fast_exp2(y[n][j]);
                l[n][j & 1] += p[j];
            }
            s_p[(warp * NT + n) * 32 + lane] = make_uint2(transpose8(pack_f16(p[0], p[1])), transpose8(pack_f16(p[2], p[3])));
        }
        __syncthreads();  // P is there (and, after a move, s_red has been read)
        // this warp's half of the channels of two chunks
        auto pv = [&](int q, int pos, bool whole) {
            const uint8_t* vt = stage + q * C::CHUNK + HALF;
            uint32_t v[4], vs[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = chunk_token(2 * c + (j & 1)) + 8 * (j >> 1);
                if constexpr (D == 128) {
                    v[j] = *reinterpret_cast<const uint32_t*>(vt + t * 64 + chalf * 32 + 4 * g);
                    vs[j] = vt[CODES + t * 8 + chalf * 4 + (g >> 1)];
                } else {
                    v[j] = *reinterpret_cast<const uint16_t*>(vt + t * 32 + chalf * 16 + 2 * g);
                    vs[j] = vt[CODES + t * 4 + chalf * 2 + (g >> 2)];
                }
                // slots past the sequence's end may hold anything: their scale counts as 0
                if (!whole && pos + t >= len) vs[j] = 0u;
            }
            const uint32_t s01 = e4m3x2_to_f16(vs[0] + vs[1] * 256u), s23 = e4m3x2_to_f16(vs[2] + vs[3] * 256u);
            // byte i of a word: the lane's channel 2i (lo) or 2i + 1 (hi) of a token pair, the
            // earlier token in the low bits
            uint32_t lo01[4], hi01[4], lo23[4], hi23[4];
            if constexpr (D == 128) {
                e2m1x8_to_f16((v[0] & 0x0f0f0f0fu) | ((v[1] << 4) & 0xf0f0f0f0u), lo01);
                e2m1x8_to_f16(((v[0] >> 4) & 0x0f0f0f0fu) | (v[1] & 0xf0f0f0f0u), hi01);
                e2m1x8_to_f16((v[2] & 0x0f0f0f0fu) | ((v[3] << 4) & 0xf0f0f0f0u), lo23);
                e2m1x8_to_f16(((v[2] >> 4) & 0x0f0f0f0fu) | (v[3] & 0xf0f0f0f0u), hi23);
            } else {
                const uint32_t v02 = v[0] | v[2] << 16, v13 = v[1] | v[3] << 16;
                uint32_t lo[4], hi[4];
                e2m1x8_to_f16((v02 & 0x0f0f0f0fu) | ((v13 << 4) & 0xf0f0f0f0u), lo);
                e2m1x8_to_f16(((v02 >> 4) & 0x0f0f0f0fu) | (v13 & 0xf0f0f0f0u), hi);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    lo01[i] = lo[i];
                    hi01[i] = hi[i];
                    lo23[i] = lo[2 + i];
                    hi23[i] = hi[2 + i];
                }
            }
            uint2 pf[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) pf[n] = s_p[(q * NT + n) * 32 + lane];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const uint32_t av[4] = {hmul2(lo01[i], s01), hmul2(hi01[i], s01), hmul2(lo23[i], s23), hmul2(hi23[i], s23)};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(oacc[n][i], av, pf[n].x, pf[n].y);
            }
        };
        const int qa = tpair ? firsts.z : firsts.x, qb = tpair ? firsts.w : firsts.y;
        if (qa >= 0 && qb >= 0 && max(qa, qb) + 16 <= len) {
            pv(2 * tpair, qa, true);
            pv(2 * tpair + 1, qb, true);
        } else {
            if (qa >= 0) pv(2 * tpair, qa, false);
            if (qb >= 0) pv(2 * tpair + 1, qb, false);
        }
    }

    // the sums of the warps' chunks joined, and O of the second chunk pair handed to the first
    __syncthreads();
    float4* s_o = reinterpret_cast<float4*>(smem) + chalf * NT * MT * 32;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], off);
            if (g == 0) s_red[warp * COLS + n * 8 + 2 * c + j] = l[n][j];
        }
        if (tpair) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
                s_o[(n * MT + i) * 32 + lane] = make_float4(oacc[n][i][0], oacc[n][i][1], oacc[n][i][2], oacc[n][i][3]);
        }
    }
    __syncthreads();
    if (!tpair) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const float4 x = s_o[(n * MT + i) * 32 + lane];
                oacc[n][i][0] += x.x;
                oacc[n][i][1] += x.y;
                oacc[n][i][2] += x.z;
                oacc[n][i][3] += x.w;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = n * 8 + 2 * c + j;
                if (r >= R) continue;
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < WARPS; ++i) sum += s_red[i * COLS + r];
                const float inv = sum == 0.f ? 0.f : a.v_scale / sum;
                const float lse = sum == 0.f ? NEG_INF : (ref[n][j] + log2f(sum)) * kLn2;
                const int d = chalf * (D / 2) + g * (D / 16);  // the lane's 2 MT channels
                const bool first = warp == 0 && g == 0;
                if (nsplit == 1) {
                    const long long oi = out_index(r);
#pragma unroll
                    for (int i = 0; i < MT; i += 2)
                        *reinterpret_cast<uint2*>(a.o + oi * D + d + 2 * i) =
                            make_uint2(pack_bf16(oacc[n][i][j] * inv, oacc[n][i][j + 2] * inv),
                                       pack_bf16(oacc[n][i + 1][j] * inv, oacc[n][i + 1][j + 2] * inv));
                    if (first && a.lse) a.lse[oi] = lse;
                } else {
                    const long long at = ((long long)row * a.num_splits + split) * R + r;
#pragma unroll
                    for (int i = 0; i < MT; i += 2)
                        *reinterpret_cast<float4*>(a.part_o + at * D + d + 2 * i) =
                            make_float4(oacc[n][i][j] * inv, oacc[n][i][j + 2] * inv, oacc[n][i + 1][j] * inv,
                                        oacc[n][i + 1][j + 2] * inv);
                    if (first) a.part_lse[at] = lse;
                }
            }
        }
    }
    if (nsplit == 1) return;
    __syncthreads();
    if (tid == 0) {
        fence_acq_rel_gpu();
        const int done = atomic_add_acq_rel(a.counters + row, 1);
        s_last = done == nsplit - 1;
        if (s_last) a.counters[row] = 0;
        fence_acq_rel_gpu();
    }
    __syncthreads();
    if (!s_last) return;
    for (int i = tid; i < R * (D / 4); i += C::THREADS) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        const long long at = (long long)row * a.num_splits * R + r;
        float top = NEG_INF;
        for (int k = 0; k < nsplit; ++k) top = fmaxf(top, __ldcg(a.part_lse + at + (long long)k * R));
        float sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < nsplit; ++k) {
            const float pl = __ldcg(a.part_lse + at + (long long)k * R);
            const float w = pl == NEG_INF ? 0.f : fast_exp2((pl - top) * kLog2e);
            const float4 x = __ldcg(reinterpret_cast<const float4*>(a.part_o + (at + (long long)k * R) * D + d));
            sum += w;
            o.x += w * x.x;
            o.y += w * x.y;
            o.z += w * x.z;
            o.w += w * x.w;
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const long long oi = out_index(r);
        *reinterpret_cast<uint2*>(a.o + oi * D + d) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
        if (d == 0 && a.lse) a.lse[oi] = sum == 0.f ? NEG_INF : top + log2f(sum) * kLn2;
    }
}

namespace {

typedef void (*Attn4Fn)(const Attn4Args);

template <int D, int NT, bool SPARSE>
void pick(Attn4Fn* fn, int* smem, int* threads) {
    *fn = attn4_kernel<D, NT, SPARSE>;
    *smem = Attn4Cfg<D, NT>::SMEM;
    *threads = Attn4Cfg<D, NT>::THREADS;
}

template <int D>
void pick_R(int R, bool sparse, Attn4Fn* fn, int* smem, int* threads) {
    if (sparse) pick<D, 1, true>(fn, smem, threads);  // one position: R = G <= 8
    else if (R <= 8) pick<D, 1, false>(fn, smem, threads);
    else if (R <= 16) pick<D, 2, false>(fn, smem, threads);
    else if (R <= 32) pick<D, 4, false>(fn, smem, threads);
    else pick<D, 8, false>(fn, smem, threads);
}

// The kernel for R query rows of a KV head, its dynamic shared memory and block.
void attn4_variant(int D, int R, bool sparse, Attn4Fn* fn, int* smem, int* threads) {
    if (D == 128) pick_R<128>(R, sparse, fn, smem, threads);
    else pick_R<64>(R, sparse, fn, smem, threads);
}

}  // namespace

// The kernel's attribute for its shared memory and its CTAs on an SM, asked of the driver
// once for a device and a variant.
static cudaError_t attn4_ready(int D, int R, bool sparse, int* occ) {
    constexpr int kDevices = 64, kVariants = 10;
    static std::atomic<int> known[kDevices][kVariants];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int v = (D == 128 ? 5 : 0) + (sparse ? 4 : R <= 8 ? 0 : R <= 16 ? 1 : R <= 32 ? 2 : 3);
    int n = dev < kDevices ? known[dev][v].load(std::memory_order_acquire) : 0;
    if (n == 0) {
        Attn4Fn fn;
        int smem, threads;
        attn4_variant(D, R, sparse, &fn, &smem, &threads);
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem);
        if (e != cudaSuccess) return e;
        if (n < 1) n = 1;
        if (dev < kDevices) known[dev][v].store(n, std::memory_order_release);
    }
    *occ = n;
    return cudaSuccess;
}

int occ_attn4(int D, int R, bool sparse) {
    int n = 1;
    return attn4_ready(D, R, sparse, &n) == cudaSuccess ? n : 1;
}

cudaError_t launch_attn4(const Attn4Args& a, bool sparse, cudaStream_t st) {
    Attn4Fn fn;
    int smem, threads, occ;
    const int R = a.T * (a.H_q / a.H_kv);
    attn4_variant(a.D, R, sparse, &fn, &smem, &threads);
    cudaError_t e = attn4_ready(a.D, R, sparse, &occ);
    if (e != cudaSuccess) return e;
    return launch_pdl(fn, dim3((unsigned)((long long)a.B * a.H_kv * a.num_splits)), dim3(threads), smem, st, a);
}

}  // namespace spd
