// attn4_decode.cu -- attention over the 4-bit paged cache for up to eight query rows of a
// KV head: sparse decode over the selected pages, and dense decode (or the verification
// of a few positions) over the whole cache.
//
// A unit is a run of at most pages_per_split pages of one (sequence, KV head) row.  A CTA of
// four warps takes one unit; its warps take the unit's pairs of 16-token chunks in turn, each
// on its own: lane i resolves the warp's i-th next chunk (selection entry, page-table
// entry), and the warp keeps a ring of pairs filled by bulk copies, refilling a slot as soon
// as it has read it, so no warp waits for another before the unit's end.  (With barriers
// between the warps -- keys and values split over them -- the same products took 28 us
// where this takes 22.6; one pair at a time instead of one chunk saves a wait, a vote and
// a refill.)
//
// Per chunk, on the tensor cores (mma.sync m16n8k16, fp16 in, fp32 out):
//
//   S^T = K Q^T   (rows: 16 tokens, columns: 8 query rows)
//   O^T += V^T P^T
//
// so the tokens fill the MMA rows and the few query rows its columns.  tcgen05 would
// spend 16 columns and a hand-over between conversions and products on them (41 us for the
// batch below, tried; two CTAs on an SM take 1.1 us for 128 tokens each here, 1.5 with
// attn4_verify.cu's 32 columns); for more rows it wins.  code * scale is exact in fp16,
// so the products are those of the values the cache stands for.  The contraction's
// channel order is free: lane (g, c) = (lane / 4, lane % 4) holds the D / 4 channels from
// c * D / 4 on of tokens g and g + 8, contiguous in memory, and V's channels g * D / 8 ...
// of tokens 2c, 2c+1, 2c+8, 2c+9.
//
// Measured on the pipes: a chunk costs an SM quarter 64 conversions (2 cycles each), 64
// fp16 products and 16 mma (8 cycles each, during which nothing else issues), 320 to 390
// cycles in all.  64 sequences x 64 pages of 16 tokens, 32 / 8 heads of 128: 22.6 us, 3.4 TB/s of
// keys and values, 50 % of the measured copy peak.  Half of that is those cycles (54 chunks an SM
// quarter: 9 to 11 us); the other half is a unit's start (length, selection, page table, first copy,
// one behind the other, and the queries' scaling) and the join of its warps, about 9 us, which
// overlap no other work of the unit, and 512 units on 152 SMs, of which those with four end
// last.  One sequence of 131,072 tokens in 76 splits: 39.5 us, 3.8 TB/s, 56 %.
#include "attn4.cuh"

namespace spd {

namespace {

__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

template <int D>
struct DecodeCfg {
    static constexpr int WARPS = 4, THREADS = 128;
    static constexpr int COLS = 8;
    static constexpr int CHUNK = kv4_tile_bytes(16, D);  // bytes of 16 tokens' keys and values
    static constexpr int STAGES = 2;                     // pairs of chunks in a warp's ring
    static constexpr int RING = WARPS * STAGES * 2 * CHUNK;
    static constexpr int MERGE = WARPS * COLS * D * 4;   // float [WARPS][COLS][D], over the ring when it is done
    static constexpr int OFF_Q = RING > MERGE ? RING : MERGE;   // half [D / 32][32 lanes][8]: B fragments of Q^T
    static constexpr int OFF_FAC = OFF_Q + COLS * D * 2;        // float [COLS]: logit scale of each query row
    static constexpr int OFF_M = OFF_FAC + COLS * 4;            // float [WARPS][COLS]
    static constexpr int OFF_L = OFF_M + WARPS * COLS * 4;      // float [WARPS][COLS]
    static constexpr int OFF_BAR = OFF_L + WARPS * COLS * 4;    // uint64 [WARPS][STAGES]
    static constexpr int OFF_META = OFF_BAR + WARPS * STAGES * 8;  // int2 [WARPS][STAGES]: first positions or -1
    static constexpr int SMEM = OFF_META + WARPS * STAGES * 8;
    static constexpr int OCC = 4;  // CTAs on an SM
};

template <int D, bool SPARSE>
__global__ void __launch_bounds__(128, DecodeCfg<D>::OCC) decode4_kernel(const Attn4Args a) {
    using C = DecodeCfg<D>;
    constexpr int COLS = C::COLS, STAGES = C::STAGES, WARPS = C::WARPS;
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
    uint8_t* ring = smem + warp * STAGES * 2 * C::CHUNK;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR) + warp * STAGES;
    int2* meta = reinterpret_cast<int2*>(smem + C::OFF_META) + warp * STAGES;
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
    const int cpp_log2 = __ffs(a.ps) - 5;  // chunks per page: 1, 2 or 4
    // pair m of this warp is chunks 8 m + 2 warp and the next one of the unit; lane i resolves
    // chunk i % 2 of pair base + i / 2.  The query rows and the first selection entries are
    // read together with the lengths.
    auto chunk_of = [&](int m) { return 8 * (m + (lane >> 1)) + 2 * warp + (lane & 1); };
    int lp_next = -1, ph_next = -1;  // the next 16 pairs' logical pages and page-table entries, unchecked
    if (SPARSE && (chunk_of(0) >> cpp_log2) < a.k_max - start)
        lp_next = a.sel[(long long)row * a.k_max + start + (chunk_of(0) >> cpp_log2)];
    constexpr int RW = COLS / WARPS;
    float2 qx[RW][D / 64];
#pragma unroll
    for (int j = 0; j < RW; ++j)
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            qx[j][i] = make_float2(0.f, 0.f);
            if (warp + WARPS * j < R)
                qx[j][i] = __bfloat1622float2(
                    *reinterpret_cast<const __nv_bfloat162*>(a.q + out_index(warp + WARPS * j) * D + 2 * lane + 64 * i));
        }
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
    const int chunks = count << cpp_log2;
    const int pairs = chunks > 2 * warp ? (chunks - 2 * warp + 7) / 8 : 0;  // of this warp

    auto next_pages = [&](int m) {
        const int ci = chunk_of(m);
        lp_next = -1;
        if (ci < chunks) lp_next = SPARSE ? a.sel[(long long)row * a.k_max + start + (ci >> cpp_log2)] : start + (ci >> cpp_log2);
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
                const int at = lp_next * a.ps + (ci & ((1 << cpp_log2) - 1)) * 16;
                if (at < len) {
                    ph_cur = ph_next;
                    pos_cur = at;
                }
            }
        }
    };
    // issues pair m into slot: lane 4 q + i copies piece i of chunk q (keys' codes and scales,
    // values' codes and scales), or lane 4 q the whole chunk where a page is one
    const int codes = kv4_codes_bytes(a.ps, D), half = kv4_half_bytes(a.ps, D);
    auto issue = [&](int m, int slot) {
        const int from = (m & 15) * 2 + (lane >> 2 & 1);
        const int phys = __shfl_sync(0xffffffffu, ph_cur, from), pos = __shfl_sync(0xffffffffu, pos_cur, from);
        const unsigned there = __ballot_sync(0xffffffffu, pos >= 0 && (lane & 27) == 0);
        if ((lane & 27) == 0) reinterpret_cast<int*>(meta + slot)[lane >> 2] = pos;
        if (lane == 0) mbar_arrive_expect_tx(full + slot, __popc(there) * C::CHUNK);
        __syncwarp();
        if (lane < 8 && pos >= 0) {
            const int i = lane & 3;
            const uint8_t* tile = a.kv4 + ((long long)phys * a.H_kv + h) * (2LL * half);
            uint8_t* dst = ring + (2 * slot + (lane >> 2)) * C::CHUNK;
            if (cpp_log2 == 0) {
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
#pragma unroll
    for (int m = 0; m < STAGES; ++m)
        if (m < pairs) issue(m, m);
    if (pairs > 16) next_pages(16);

    // the query rows in fp16, each scaled by 2^-e so that its largest channel lies in [1, 2)
    // (the factor goes into the logits' scale), stored as the lanes read them
#pragma unroll
    for (int j = 0; j < RW; ++j) {
        const int r = warp + WARPS * j;
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) amax = fmaxf(amax, fmaxf(fabsf(qx[j][i].x), fabsf(qx[j][i].y)));
        const int e = query_exponent(amax);
        const float down = pow2f(-e);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const int ch = 2 * lane + 64 * i, qc = ch / (D / 4), w = ch % (D / 4) / 8;
            *reinterpret_cast<uint32_t*>(s_q + (w * 32 + r * 4 + qc) * 8 + ch % 8) = pack_f16(qx[j][i].x * down, qx[j][i].y * down);
        }
        if (lane == 0) s_fac[r] = a.scale_log2 * pow2f(e);
    }
    __syncthreads();

    uint4 qf[KW];
#pragma unroll
    for (int w = 0; w < KW; ++w) qf[w] = *reinterpret_cast<const uint4*>(s_q + (w * 32 + lane) * 8);
    float fac[2], ref[2], l[2];  // ref: the reference less kBias4
    float oacc[MT][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        fac[j] = s_fac[2 * c + j];
        ref[j] = kLow4;
        l[j] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) oacc[i][0] = oacc[i][1] = oacc[i][2] = oacc[i][3] = 0.f;

    int slot = 0;
    uint32_t parity = 0;
    for (int m = 0; m < pairs; ++m) {
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(full + slot, parity, a.status, a.wait_ns))) {
            // the pairs in flight land before the shared memory is used for anything else
            for (int j = m; j < min(m + STAGES, pairs); ++j)
                mbar_wait_bounded(full + j % STAGES, (uint32_t)(j / STAGES) & 1u, a.status, drain_limit(a));
            __syncwarp();
            break;
        }
        const int2 first = meta[slot];
        const uint8_t* pair = ring + 2 * slot * C::CHUNK;
        // logits of both chunks (one that is not there: of whatever the ring holds)
        float sc[2][4];
        uint32_t vw[2][4][VW], vs[2][4];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint8_t* kt = pair + q * C::CHUNK;
            const uint8_t* vt = kt + HALF;
            uint32_t kw[2][KW], ks[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = g + 8 * j;
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
            for (int j = 0; j < 4; ++j) {
                const int t = 2 * c + (j & 1) + 8 * (j >> 1);
                if constexpr (D == 128) {
                    const uint2 x = *reinterpret_cast<const uint2*>(vt + t * 64 + g * 8);
                    vw[q][j][0] = x.x;
                    vw[q][j][VW - 1] = x.y;
                } else {
                    vw[q][j][0] = *reinterpret_cast<const uint32_t*>(vt + t * 32 + g * 4);
                }
                vs[q][j] = vt[CODES + t * (D / 16) + (D == 128 ? g : g >> 1)];
            }
            sc[q][0] = sc[q][1] = sc[q][2] = sc[q][3] = 0.f;
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
                mma_f16(sc[q], a0, qf[w].x, qf[w].y);
                mma_f16(sc[q], a1, qf[w].z, qf[w].w);
            }
        }
        __syncwarp();  // the slot has been read: refill it
        const int mn = m + STAGES;
        if (mn < pairs) {
            if ((mn & 15) == 0) {
                take_next(mn);
                next_pages(mn + 16);
            } else if ((mn & 15) == 4) {
                next_entries();
            }
            issue(mn, slot);
        }
        if (++slot == STAGES) {
            slot = 0;
            parity ^= 1u;
        }
        // y: logits in base 2 less ref, hidden tokens at -inf
        float y[2][4];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[q][j] = fmaf(sc[q][j], fac[j & 1], -ref[j & 1]);
        if (min(first.x, first.y) < 0 || max(first.x, first.y) + 15 > len - a.T) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int pos0 = q ? first.y : first.x;
                const int left = pos0 < 0 ? 0 : len - pos0;  // tokens of the chunk
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // slots past the sequence's end may hold anything: their scale counts as 0
                    if (2 * c + (j & 1) + 8 * (j >> 1) >= left) vs[q][j] = 0u;
                    const int r = 2 * c + (j & 1);
                    const int seen = r < R ? left - a.T + r / G : left - 1;  // the last token of the chunk that the row sees
                    if (pos0 < 0 || g + 8 * (j >> 1) > seen) y[q][j] = NEG_INF;
                }
            }
        }
        float top = y[0][0];
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int j = q == 0 ? 1 : 0; j < 4; ++j) top = fmaxf(top, y[q][j]);
        if (__any_sync(0xffffffffu, top > kHead4 + kBias4)) {  // some reference has to move
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // from the logits themselves: an unset reference leaves nothing of them in y
                float z[4] = {sc[0][j] * fac[j], sc[0][j + 2] * fac[j], sc[1][j] * fac[j], sc[1][j + 2] * fac[j]};
                float x = NEG_INF;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (y[i >> 1][j + 2 * (i & 1)] == NEG_INF) z[i] = NEG_INF;
                    x = fmaxf(x, z[i]);
                }
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
                x = fmaxf(ref[j], x - kBias4);
                const float corr = fast_exp2(ref[j] - x);
                ref[j] = x;
                l[j] *= corr;
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i >> 1][j + 2 * (i & 1)] = z[i] - x;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    oacc[i][j] *= corr;
                    oacc[i][j + 2] *= corr;
                }
            }
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                p[j] = fast_exp2(y[q][j]);
                l[j & 1] += p[j];
            }
            const uint32_t p0 = transpose8(pack_f16(p[0], p[1])), p1 = transpose8(pack_f16(p[2], p[3]));
            const uint32_t s01 = e4m3x2_to_f16(vs[q][0] + vs[q][1] * 256u), s23 = e4m3x2_to_f16(vs[q][2] + vs[q][3] * 256u);
#pragma unroll
            for (int w = 0; w < VW; ++w) {
                // byte i of the words below: channel 2i (first and third word) or 2i + 1 of a token
                // pair, the earlier token in the low bits
                uint32_t x[4][4];
                e2m1x8_to_f16((vw[q][0][w] & 0x0f0f0f0fu) | ((vw[q][1][w] << 4) & 0xf0f0f0f0u), x[0]);
                e2m1x8_to_f16(((vw[q][0][w] >> 4) & 0x0f0f0f0fu) | (vw[q][1][w] & 0xf0f0f0f0u), x[1]);
                e2m1x8_to_f16((vw[q][2][w] & 0x0f0f0f0fu) | ((vw[q][3][w] << 4) & 0xf0f0f0f0u), x[2]);
                e2m1x8_to_f16(((vw[q][2][w] >> 4) & 0x0f0f0f0fu) | (vw[q][3][w] & 0xf0f0f0f0u), x[3]);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t av[4] = {hmul2(x[0][i], s01), hmul2(x[1][i], s01), hmul2(x[2][i], s23), hmul2(x[3][i], s23)};
                    mma_f16(oacc[4 * w + i], av, p0, p1);
                }
            }
        }
    }

    // the warps' states joined: references, then sums and outputs relative to the largest
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], off);
        if (g == 0) s_m[warp * COLS + 2 * c + j] = ref[j];
    }
    __syncthreads();  // and every warp is done with its ring
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int col = 2 * c + j;
        float top = kLow4;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) top = fmaxf(top, s_m[i * COLS + col]);
        const float f = fast_exp2(ref[j] - top);
        if (g == 0) s_l[warp * COLS + col] = l[j] * f;
        float* out = s_o + (warp * COLS + col) * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < MT; ++i) *reinterpret_cast<float2*>(out + 2 * i) = make_float2(oacc[i][j] * f, oacc[i][j + 2] * f);
    }
    __syncthreads();
    for (int i = tid; i < R * (D / 4); i += C::THREADS) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        float top = kLow4, sum = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < WARPS; ++k) {
            top = fmaxf(top, s_m[k * COLS + r]);
            sum += s_l[k * COLS + r];
            const float4 x = *reinterpret_cast<const float4*>(s_o + (k * COLS + r) * D + d);
            o.x += x.x;
            o.y += x.y;
            o.z += x.z;
            o.w += x.w;
        }
        const float inv = sum == 0.f ? 0.f : a.v_scale / sum;
        const float lse = sum == 0.f ? NEG_INF : (top + log2f(sum)) * kLn2;
        if (nsplit == 1) {
            const long long oi = out_index(r);
            *reinterpret_cast<uint2*>(a.o + oi * D + d) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
            if (d == 0 && a.lse) a.lse[oi] = lse;
        } else {
            const long long at = ((long long)row * a.parts + split) * R + r;
            *reinterpret_cast<float4*>(a.part_o + at * D + d) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
            if (d == 0) a.part_lse[at] = lse;
        }
    }
    join_splits<D, C::THREADS, false>(a, row, split, nsplit, R, &s_last, out_index);
}

template <int D>
cudaError_t launch_d(const Attn4Args& a, bool sparse, cudaStream_t st) {
    using C = DecodeCfg<D>;
    static_assert(C::SMEM <= 48 * 1024, "within what a kernel may use unasked");
    const dim3 grid((unsigned)((long long)a.B * a.H_kv * a.num_splits)), block(C::THREADS);
    return sparse ? launch_pdl(decode4_kernel<D, true>, grid, block, C::SMEM, st, a)
                  : launch_pdl(decode4_kernel<D, false>, grid, block, C::SMEM, st, a);
}

}  // namespace

int occ_attn4_decode() { return DecodeCfg<128>::OCC; }

cudaError_t launch_attn4_decode(const Attn4Args& a, bool sparse, cudaStream_t st) {
    return a.D == 128 ? launch_d<128>(a, sparse, st) : launch_d<64>(a, sparse, st);
}

}  // namespace spd
