// attn4.cu -- attention over the 4-bit paged cache: sparse decode over the selected
// pages and dense causal verification over the whole cache.
//
// A unit is a run of at most pages_per_split pages of one (sequence, KV head) row;
// it holds all R = T * G query rows of the KV head in n-tiles of eight.  A CTA
// takes one unit; its warps take the unit's 16-token chunks in turn, each on its own:
// lane i resolves the warp's i-th next chunk (selection entry, page-table entry), and
// the warp keeps a ring of chunks filled by bulk copies, refilling a slot as soon as it
// has read it, so no warp waits for another before the unit's end.
//
// Per chunk, on the tensor cores (mma.sync m16n8k16, fp16 in, fp32 out):
//
//   S^T = K Q^T   (rows: 16 tokens, columns: 8 query rows)
//   O^T += V^T P^T
//
// so the tokens fill the MMA rows and the few query rows its columns.  code * scale
// is exact in fp16, so the products are those of the values the cache stands for.
// The contraction's channel order is free: lane (g, c) = (lane / 4, lane % 4) holds
// the D / 4 channels from c * D / 4 on of tokens g and g + 8, contiguous in memory,
// and V's channels g * D / 8 ... of tokens 2c, 2c+1, 2c+8, 2c+9.  Queries are
// scaled by a power of two into fp16's range (the factor goes into the logits'
// scale).  Online softmax in fp32 in base 2; a column's reference moves only when a
// logit exceeds it by kHead4, and weights carry a factor 2^kBias4 so that what
// fp16 drops of a weight lies 2^-32 below the reference.
#include "kv4.cuh"
#include "kernels.h"

namespace spd {

constexpr float kHead4 = 8.f;  // log2 headroom before the running maximum moves
constexpr float kBias4 = 7.f;  // 2^(kHead4 + kBias4) = 32768 stays within fp16

__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

constexpr float kLow4 = -3.0e38f;  // a column's reference before its first visible token

template <int D, int NT>
struct Attn4Cfg {
    static constexpr int NTW = NT < 4 ? NT : 4;     // n-tiles of a warp
    static constexpr int NG = NT / NTW;             // warps that share a chunk's tokens
    static constexpr int TW = 4 / NG;               // chunks in work at once
    static constexpr int WARPS = NG * TW;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int COLS = NT * 8;
    static constexpr int STAGES = 4;                // ring slots of a warp
    static constexpr int CHUNK = kv4_tile_bytes(16, D);  // bytes of 16 tokens' keys and values
    static constexpr int RING = WARPS * STAGES * CHUNK;
    static constexpr int MERGE = TW * COLS * D * 4;  // float [TW][COLS][D], over the ring when it is done
    static constexpr int OFF_Q = RING > MERGE ? RING : MERGE;      // half [COLS][D]
    static constexpr int OFF_FAC = OFF_Q + COLS * D * 2;           // float [COLS]: logit scale of each query row
    static constexpr int OFF_M = OFF_FAC + COLS * 4;               // float [TW][COLS]
    static constexpr int OFF_L = OFF_M + TW * COLS * 4;            // float [TW][COLS]
    static constexpr int OFF_BAR = OFF_L + TW * COLS * 4;          // uint64 [WARPS][STAGES]
    static constexpr int OFF_META = OFF_BAR + WARPS * STAGES * 8;  // int [WARPS][STAGES]: first position or -1
    static constexpr int SMEM = OFF_META + WARPS * STAGES * 4;
    // CTAs that the registers leave room for on an SM
    static constexpr int OCC = NT <= 1 ? 5 : (NT == 2 ? 3 : 2);
};

template <int D, int NT, bool SPARSE>
__global__ void __launch_bounds__(Attn4Cfg<D, NT>::THREADS, Attn4Cfg<D, NT>::OCC) attn4_kernel(const Attn4Args a) {
    using C = Attn4Cfg<D, NT>;
    constexpr int NTW = C::NTW, TW = C::TW, COLS = C::COLS, STAGES = C::STAGES;
    constexpr int KW = D / 32;  // 32-bit code words of a lane's share of a key row
    constexpr int VW = D / 64;  // and of a value row
    constexpr int MT = D / 16;  // 16-channel m-tiles of O^T
    constexpr int CODES = kv4_codes_bytes(16, D), HALF = kv4_half_bytes(16, D);  // of a chunk
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_last;
    float* s_fac = reinterpret_cast<float*>(smem + C::OFF_FAC);
    float* s_m = reinterpret_cast<float*>(smem + C::OFF_M);
    float* s_l = reinterpret_cast<float*>(smem + C::OFF_L);
    __half* s_q = reinterpret_cast<__half*>(smem + C::OFF_Q);
    float* s_o = reinterpret_cast<float*>(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int tw = warp % TW, ng = warp / TW;
    uint8_t* ring = smem + warp * STAGES * C::CHUNK;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * STAGES;
    int* meta = reinterpret_cast<int*>(smem + C::OFF_META) + warp * STAGES;
    const int G = a.H_q / a.H_kv, R = a.T * G;
    const float NEG_INF = __int_as_float(0xff800000);

    const int row = blockIdx.x / a.num_splits, split = blockIdx.x % a.num_splits;
    const int b = row / a.H_kv, h = row - b * a.H_kv;
    auto out_index = [&](int r) -> long long {
        const int t = r / G;
        return ((long long)b * a.T + t) * a.H_q + h * G + (r - t * G);
    };
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) mbar_init(full + i, 1);
        mbar_fence_init();
    }
    __syncwarp();
    pdl_wait();
    pdl_trigger();

    const int start = split * a.pages_per_split;
    const int cpp = a.ps >> 4;  // chunks per page
    // chunk k of this warp is chunk tw + k * TW of the unit; the first selection entries
    // are read together with the length and the count
    int sel0 = 0;
    if (SPARSE && start + (tw + lane * TW) / cpp < a.k_max) sel0 = a.sel[(long long)row * a.k_max + start + (tw + lane * TW) / cpp];
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
    const int mine = chunks > tw ? (chunks - tw + TW - 1) / TW : 0;  // of this warp

    // this lane's chunk base + lane: its physical page and first position (-1: nothing to read)
    auto resolve = [&](int base, int& phys, int& pos) {
        phys = pos = -1;
        const int k = base + lane;
        if (k < mine) {
            const int ci = tw + k * TW, item = ci / cpp;
            const int lp = !SPARSE ? start + item : base == 0 ? sel0 : a.sel[(long long)row * a.k_max + start + item];
            if (lp < 0 || lp >= P) {
                raise_status(a.status, SPD_DEV_BAD_SEL);
            } else {
                const int at = lp * a.ps + (ci - item * cpp) * 16;
                const int ph = a.page_table[(long long)b * a.max_pages + lp];
                if (ph < 0 || ph >= a.num_phys) raise_status(a.status, SPD_DEV_BAD_PAGE);
                else if (at < len) {
                    phys = ph;
                    pos = at;
                }
            }
        }
    };
    int ph_cur, pos_cur, ph_next = -1, pos_next = -1;
    resolve(0, ph_cur, pos_cur);
    // issues chunk k into its slot (by the whole warp; the copies by lanes 0-3)
    const int codes = kv4_codes_bytes(a.ps, D), half = kv4_half_bytes(a.ps, D);
    auto issue = [&](int k) {
        const int slot = k % STAGES;
        const int phys = __shfl_sync(0xffffffffu, ph_cur, k & 31), pos = __shfl_sync(0xffffffffu, pos_cur, k & 31);
        if (lane == 0) {
            meta[slot] = pos;
            mbar_arrive_expect_tx(full + slot, pos >= 0 ? C::CHUNK : 0);
        }
        __syncwarp();
        if (pos >= 0) {
            const uint8_t* tile = a.kv4 + ((long long)phys * a.H_kv + h) * (2LL * half);
            uint8_t* dst = ring + slot * C::CHUNK;
            if (a.ps == 16) {
                if (lane == 0) bulk_load(dst, tile, C::CHUNK, full + slot);
            } else if (lane < 4) {  // keys' codes and scales, values' codes and scales
                const int t0 = pos & (a.ps - 1);
                const uint8_t* src = tile + (lane >> 1) * half + (lane & 1 ? codes + t0 * (D / 16) : t0 * (D / 2));
                bulk_load(dst + (lane >> 1) * HALF + (lane & 1) * CODES, src, lane & 1 ? HALF - CODES : CODES, full + slot);
            }
        }
    };
#pragma unroll
    for (int k = 0; k < STAGES; ++k)
        if (k < mine) issue(k);
    if (mine > 32) resolve(32, ph_next, pos_next);

    // the query rows in fp16, each scaled by 2^-e so that its largest channel lies in [1, 2)
    for (int r = warp; r < COLS; r += C::WARPS) {
        float x[D / 32];
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            x[i] = r < R ? __bfloat162float(reinterpret_cast<const bf16*>(a.q)[out_index(r) * D + lane + 32 * i]) : 0.f;
            amax = fmaxf(amax, fabsf(x[i]));
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        int e = (int)(__float_as_uint(amax) >> 23) - 127;
        if (e > 126 || e < -126) e = e > 126 ? 126 : -126;
        if (amax == 0.f) e = 0;
        const float down = pow2f(-e);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) s_q[r * D + lane + 32 * i] = __float2half_rn(x[i] * down);
        if (lane == 0) s_fac[r] = a.scale_log2 * pow2f(e);
    }
    __syncthreads();

    uint32_t qf[NTW][2 * KW][2];
    float fac[NTW][2], m[NTW][2], l[NTW][2];
    float oacc[NTW][MT][4];
#pragma unroll
    for (int n = 0; n < NTW; ++n) {
        const int col0 = (ng * NTW + n) * 8;
#pragma unroll
        for (int k = 0; k < 2 * KW; ++k) {
            const uint2 q = *reinterpret_cast<const uint2*>(s_q + (col0 + g) * D + c * (D / 4) + 4 * k);
            qf[n][k][0] = q.x;
            qf[n][k][1] = q.y;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            fac[n][j] = s_fac[col0 + 2 * c + j];
            m[n][j] = kLow4;
            l[n][j] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) oacc[n][i][0] = oacc[n][i][1] = oacc[n][i][2] = oacc[n][i][3] = 0.f;
    }

    for (int k = 0; k < mine; ++k) {
        const int slot = k % STAGES;
        if (!mbar_wait_bounded(full + slot, (uint32_t)(k / STAGES) & 1u, a.status, a.wait_ns)) {
            // the chunks in flight land before the shared memory is used for anything else
            for (int j = k + 1; j < min(k + STAGES, mine); ++j)
                mbar_wait_bounded(full + j % STAGES, (uint32_t)(j / STAGES) & 1u, a.status, a.wait_ns);
            break;
        }
        const int pos0 = meta[slot];
        const uint8_t* kt = ring + slot * C::CHUNK;
        const uint8_t* vt = kt + HALF;
        uint32_t kw[2][KW], vw[4][VW];
        uint32_t ks[2], vs[4];
        if (pos0 >= 0) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = g + 8 * j;
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4*>(kt + t * 64 + c * 16);
                    kw[j][0] = x.x;
                    kw[j][1] = x.y;
                    kw[j][KW - 2] = x.z;
                    kw[j][KW - 1] = x.w;
                    ks[j] = *reinterpret_cast<const uint16_t*>(kt + CODES + t * 8 + 2 * c);
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(kt + t * 32 + c * 8);
                    kw[j][0] = x.x;
                    kw[j][1] = x.y;
                    ks[j] = kt[CODES + t * 4 + c];
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 2 * c + (j & 1) + 8 * (j >> 1);
                if constexpr (D == 128) {
                    const uint2 x = *reinterpret_cast<const uint2*>(vt + t * 64 + g * 8);
                    vw[j][0] = x.x;
                    vw[j][VW - 1] = x.y;
                } else {
                    vw[j][0] = *reinterpret_cast<const uint32_t*>(vt + t * 32 + g * 4);
                }
                vs[j] = vt[CODES + t * (D / 16) + (D == 128 ? g : g >> 1)];
            }
        }
        __syncwarp();  // the slot has been read: refill it
        const int kn = k + STAGES;
        if (kn < mine) {
            if ((kn & 31) == 0) {
                ph_cur = ph_next;
                pos_cur = pos_next;
                resolve(kn + 32, ph_next, pos_next);
            }
            issue(kn);
        }
        if (pos0 < 0) continue;

        float sc[NTW][4];
#pragma unroll
        for (int n = 0; n < NTW; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
        const uint32_t ks0 = e4m3x2_to_f16(ks[0]), ks1 = e4m3x2_to_f16(ks[1]);
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            uint32_t h0[4], h1[4];
            e2m1x8_to_f16(kw[0][w], h0);
            e2m1x8_to_f16(kw[1][w], h1);
            const uint32_t s0 = __byte_perm(ks0, 0, w < 2 ? 0x1010 : 0x3232), s1 = __byte_perm(ks1, 0, w < 2 ? 0x1010 : 0x3232);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h0[i] = hmul2(h0[i], s0);
                h1[i] = hmul2(h1[i], s1);
            }
            const uint32_t a0[4] = {h0[0], h1[0], h0[1], h1[1]}, a1[4] = {h0[2], h1[2], h0[3], h1[3]};
#pragma unroll
            for (int n = 0; n < NTW; ++n) {
                mma_f16(sc[n], a0, qf[n][2 * w][0], qf[n][2 * w][1]);
                mma_f16(sc[n], a1, qf[n][2 * w + 1][0], qf[n][2 * w + 1][1]);
            }
        }
        // logits in base 2, relative to the reference and raised by kBias4; hidden tokens at -inf
        if (pos0 + 15 > len - a.T) {
            // slots past the sequence's end may hold anything: their scale counts as 0
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (pos0 + 2 * c + (j & 1) + 8 * (j >> 1) >= len) vs[j] = 0u;
#pragma unroll
            for (int n = 0; n < NTW; ++n) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int r = (ng * NTW + n) * 8 + 2 * c + (j & 1);
                    const int lim = r < R ? len - a.T + r / G : len - 1;  // the last token that the row sees
                    const float z = sc[n][j] * fac[n][j & 1];
                    sc[n][j] = pos0 + g + 8 * (j >> 1) <= lim ? z : NEG_INF;
                }
            }
        } else {
#pragma unroll
            for (int n = 0; n < NTW; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) sc[n][j] *= fac[n][j & 1];
        }
        bool move = false;
#pragma unroll
        for (int n = 0; n < NTW; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) move |= fmaxf(sc[n][j], sc[n][j + 2]) > m[n][j] + kHead4;
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int n = 0; n < NTW; ++n) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = fmaxf(sc[n][j], sc[n][j + 2]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
                    x = fmaxf(x, m[n][j]);
                    const float corr = fast_exp2(m[n][j] - x);
                    m[n][j] = x;
                    l[n][j] *= corr;
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        oacc[n][i][j] *= corr;
                        oacc[n][i][j + 2] *= corr;
                    }
                }
            }
        }
        uint32_t pf[NTW][2];
#pragma unroll
        for (int n = 0; n < NTW; ++n) {
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                p[j] = fast_exp2(sc[n][j] - (m[n][j & 1] - kBias4));
                l[n][j & 1] += p[j];
            }
            pf[n][0] = movmatrix_t(pack_f16(p[0], p[1]));
            pf[n][1] = movmatrix_t(pack_f16(p[2], p[3]));
        }
        const uint32_t s01 = e4m3x2_to_f16(vs[0] | vs[1] << 8), s23 = e4m3x2_to_f16(vs[2] | vs[3] << 8);
#pragma unroll
        for (int w = 0; w < VW; ++w) {
            // byte i of the words below: channel 2i (first and third word) or 2i + 1 of a token
            // pair, the earlier token in the low bits
            uint32_t x[4][4];
            e2m1x8_to_f16((vw[0][w] & 0x0f0f0f0fu) | ((vw[1][w] << 4) & 0xf0f0f0f0u), x[0]);
            e2m1x8_to_f16(((vw[0][w] >> 4) & 0x0f0f0f0fu) | (vw[1][w] & 0xf0f0f0f0u), x[1]);
            e2m1x8_to_f16((vw[2][w] & 0x0f0f0f0fu) | ((vw[3][w] << 4) & 0xf0f0f0f0u), x[2]);
            e2m1x8_to_f16(((vw[2][w] >> 4) & 0x0f0f0f0fu) | (vw[3][w] & 0xf0f0f0f0u), x[3]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t av[4] = {hmul2(x[0][i], s01), hmul2(x[1][i], s01), hmul2(x[2][i], s23),
                                        hmul2(x[3][i], s23)};
#pragma unroll
                for (int n = 0; n < NTW; ++n) mma_f16(oacc[n][4 * w + i], av, pf[n][0], pf[n][1]);
            }
        }
    }

    // the warps' states joined: reference maxima, then sums and outputs relative to the largest
#pragma unroll
    for (int n = 0; n < NTW; ++n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[n][j] += __shfl_xor_sync(0xffffffffu, l[n][j], off);
            const int col = (ng * NTW + n) * 8 + 2 * c + j;
            if (g == 0) s_m[tw * COLS + col] = m[n][j];
        }
    }
    __syncthreads();  // and every warp is done with its ring
#pragma unroll
    for (int n = 0; n < NTW; ++n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col = (ng * NTW + n) * 8 + 2 * c + j;
            float top = kLow4;
#pragma unroll
            for (int i = 0; i < TW; ++i) top = fmaxf(top, s_m[i * COLS + col]);
            const float f = fast_exp2(m[n][j] - top);
            if (g == 0) s_l[tw * COLS + col] = l[n][j] * f;
            float* out = s_o + (tw * COLS + col) * D + g * (D / 8);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                *reinterpret_cast<float2*>(out + 2 * i) = make_float2(oacc[n][i][j] * f, oacc[n][i][j + 2] * f);
        }
    }
    __syncthreads();
    for (int i = tid; i < R * (D / 4); i += C::THREADS) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        float top = NEG_INF, sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < TW; ++k) {
            top = fmaxf(top, s_m[k * COLS + r]);
            sum += s_l[k * COLS + r];
            const float4 x = *reinterpret_cast<const float4*>(s_o + (k * COLS + r) * D + d);
            o.x += x.x;
            o.y += x.y;
            o.z += x.z;
            o.w += x.w;
        }
        const float inv = sum == 0.f ? 0.f : a.v_scale / sum;
        o.x *= inv;
        o.y *= inv;
        o.z *= inv;
        o.w *= inv;
        const float lse = sum == 0.f ? NEG_INF : (top - kBias4 + log2f(sum)) * kLn2;
        if (nsplit == 1) {
            const long long oi = out_index(r);
            *reinterpret_cast<uint2*>(a.o + oi * D + d) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
            if (d == 0 && a.lse) a.lse[oi] = lse;
        } else {
            const long long at = ((long long)row * a.num_splits + split) * R + r;
            *reinterpret_cast<float4*>(a.part_o + at * D + d) = o;
            if (d == 0) a.part_lse[at] = lse;
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

int occ_attn4(int D, int ps, int R, bool sparse) {
    Attn4Fn fn;
    int smem, threads, n = 0;
    attn4_variant(D, R, sparse, &fn, &smem, &threads);
    cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem);
    return n < 1 ? 1 : n;
}

cudaError_t launch_attn4(const Attn4Args& a, bool sparse, cudaStream_t st) {
    Attn4Fn fn;
    int smem, threads;
    attn4_variant(a.D, a.T * (a.H_q / a.H_kv), sparse, &fn, &smem, &threads);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(fn, dim3((unsigned)((long long)a.B * a.H_kv * a.num_splits)), dim3(threads), smem, st, a);
}

}  // namespace spd
