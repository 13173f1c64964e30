// rope.cu -- queries and keys of new tokens on their way from the projection to
// the attention: norm of each head's row and position rotation in one pass
// (qk_norm_rope), and the same with the keys and values written into the paged
// cache and the touched pages' key summaries rebuilt (kv_append_rope).
//
// Both read every element once and write it once; what bounds them is memory
// for long prompts and the launch for single tokens.  Measured, heads of 128:
// qk_norm_rope of 32 / 8 heads, 16,381 tokens: 67.2 us, 5.1 TB/s, 75 % of the measured copy
// peak; one token 2.2 us.  kv_append_rope of 16 / 8 heads, 4 x 4,095 tokens: 54.7 us,
// 5.0 TB/s, 74 %; 64 sequences' single tokens 3.1 us.
#include "rope.cuh"

namespace spd {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
// A warp takes kRopeTurns rows of heads a lane group at a time from one token: four
// (D = 128) or eight (D = 64) heads whose loads are in flight together and share the
// token's angles and the weights.  (32 + 8 heads of 128, one row / 16,381 rows: 2 turns
// 2.2 / 67.2 us, 4 turns 3.8 / 113 us.)
constexpr int kRopeTurns = 2;

__host__ __device__ constexpr int rope_heads_per_warp(int D) { return kRopeTurns * 32 / (D / 8); }

// Tokens of a warp: the second shares the first one's weights, addresses and rotation, and its
// loads are in flight with the first one's.  (One row / 16,381 rows: 1 token
// 1.6 / 70.3 us, 2 tokens 2.2 / 67.2; 4 tokens 106.)
constexpr int kRopeTokens = 2;

// One side (queries or keys) of kRopeTokens tokens by one warp: heads h0 ... of `heads` of rows
// row ... that lie below a.rows.  pos < 0: the token's position is not one of the table's (or
// its sequence is skipped): zero rows.
template <int D>
__device__ __forceinline__ void rope_warp(const RopeArgs& a, const uint16_t* src, long long stride, uint16_t* dst,
                                          const uint16_t* weight, int h0, int heads, long long row,
                                          const int (&pos)[kRopeTokens]) {
    constexpr int L = D / 8, HT = 32 / L;
    const int lane = threadIdx.x & 31, l = lane % L, h = h0 + lane / L;
    const RopeLane r = rope_lane<D>(l, a.rot, a.interleaved);
    const int there = (heads - h + HT - 1) / HT;  // turns of this lane
    uint2 x0[kRopeTokens][kRopeTurns], x1[kRopeTokens][kRopeTurns];
    float4 cs[kRopeTokens], sn[kRopeTokens];
    const uint16_t* p = src + row * stride + h * D;
#pragma unroll
    for (int t = 0; t < kRopeTokens; ++t) {
        const bool live = pos[t] >= 0 && row + t < a.rows;
#pragma unroll
        for (int i = 0; i < kRopeTurns; ++i) {
            x0[t][i] = x1[t][i] = make_uint2(0u, 0u);
            if (live && i < there) {
                x0[t][i] = *reinterpret_cast<const uint2*>(p + i * HT * D + r.o0);
                x1[t][i] = *reinterpret_cast<const uint2*>(p + i * HT * D + r.o1);
            }
        }
        cs[t] = sn[t] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live && r.turned) {
            const float* table = a.table + (long long)pos[t] * a.rot + 4 * l;
            cs[t] = __ldg(reinterpret_cast<const float4*>(table));
            sn[t] = __ldg(reinterpret_cast<const float4*>(table + (a.rot >> 1)));
        }
        p += stride;
    }
    float w[8];
    rope_weights(weight, r, w);
    uint16_t* q = dst + (row * heads + h) * D;
#pragma unroll
    for (int t = 0; t < kRopeTokens; ++t) {
        const int turns = row + t < a.rows ? there : 0;
#pragma unroll
        for (int i = 0; i < kRopeTurns; ++i) {
            float x[8];
            unpack4(x0[t][i], x);
            unpack4(x1[t][i], x + 4);
            rope_row<D>(x, weight != nullptr, w, a.eps, r, a.interleaved, cs[t], sn[t]);
            if (i < turns) {
                *reinterpret_cast<uint2*>(q + i * HT * D + r.o0) = pos[t] >= 0 ? pack4(x) : make_uint2(0u, 0u);
                *reinterpret_cast<uint2*>(q + i * HT * D + r.o1) = pos[t] >= 0 ? pack4(x + 4) : make_uint2(0u, 0u);
            }
        }
        q += heads * D;
    }
}

// A warp's tokens are kRopeTokens from kRopeTokens * (blockIdx.x * kRopeWarps + warp) on, its
// heads group blockIdx.y: the query heads' groups, then the key heads'.
template <int D>
__global__ void __launch_bounds__(kRopeThreads, 4) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int HW = rope_heads_per_warp(D);
    pdl_wait();
    pdl_trigger();
    const long long row = ((long long)blockIdx.x * kRopeWarps + (threadIdx.x >> 5)) * kRopeTokens;
    if (row >= a.rows) return;
    int pos[kRopeTokens];
#pragma unroll
    for (int t = 0; t < kRopeTokens; ++t) {
        pos[t] = a.rot > 0 && row + t < a.rows ? a.positions[row + t] : 0;
        if (a.rot > 0 && (pos[t] < 0 || pos[t] >= a.n_pos)) {
            if ((threadIdx.x & 31) == 0) raise_status(a.status, SPD_DEV_BAD_POS);
            pos[t] = -1;
        }
    }
    const int q_groups = (a.H_q + HW - 1) / HW;
    if ((int)blockIdx.y < q_groups)
        rope_warp<D>(a, a.q, a.q_stride, a.q_out, a.q_weight, blockIdx.y * HW, a.H_q, row, pos);
    else
        rope_warp<D>(a, a.k, a.k_stride, a.k_out, a.k_weight, (blockIdx.y - q_groups) * HW, a.H_kv, row, pos);
}

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t st) {
    const int hw = rope_heads_per_warp(a.D);
    const dim3 block(kRopeThreads);
    const dim3 grid((unsigned)((a.rows + kRopeWarps * kRopeTokens - 1) / (kRopeWarps * kRopeTokens)),
                    (unsigned)((a.H_q + hw - 1) / hw + (a.H_kv + hw - 1) / hw));
    if (a.D == 128) return launch_pdl(qk_norm_rope_kernel<128>, grid, block, 0, st, a);
    return launch_pdl(qk_norm_rope_kernel<64>, grid, block, 0, st, a);
}

// kv_append_rope: one grid of two kinds of CTA.  The first are the append's, one per
// (sequence, touched page, two KV heads), four warps a head: each takes every fourth
// group of the page's rows, older keys read from the cache and new ones normalised,
// rotated and stored, and the channel-wise min / max of all valid rows, as rounded,
// joined through shared memory, becomes the page's summary.  The CTAs behind them take
// the query heads as qk_norm_rope does.
// Groups of new rows whose loads a lane keeps in flight (1 / 2: 54.7 / 56.2 us for the 4 x 4,095
// tokens, 3.1 / 3.5 for 64 single ones), and KV heads of an append's CTA (1 / 2 / 4: 57.7 /
// 54.7 / 52.9 and 3.5 / 3.1 / 3.3 us; four leave half of the warps idle where there are two).
constexpr int kNewBatch = 1;
constexpr int kPageHeads = 2;
constexpr int kPageParts = kRopeWarps / kPageHeads;

template <int D>
__global__ void __launch_bounds__(kRopeThreads, 4) append_rope_kernel(const AppendRopeArgs p) {
    constexpr int L = D / 8;        // lanes per row
    constexpr int RPI = 32 / L;     // rows per warp instruction
    constexpr int STEP = kPageParts * RPI, kOldBatch = 2;
    __shared__ uint4 s_mm[kRopeWarps][L][2];
    const AppendArgs& a = p.append;
    const RopeArgs& ro = p.rope;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int head_ctas = (a.H_kv + kPageHeads - 1) / kPageHeads;
    const int page_ctas = a.B * p.touched * head_ctas;
    if ((int)blockIdx.x >= page_ctas) {
        // a warp: one group of the query heads of tokens row ... of all B * T, row = b * T + t at
        // position len - T + t
        constexpr int HW = rope_heads_per_warp(D);
        const unsigned groups = (ro.H_q + HW - 1) / HW;
        const unsigned unit = (blockIdx.x - page_ctas) * kRopeWarps + warp;  // below 2^31 + kRopeWarps (checked by the host)
        const unsigned row = unit / groups * kRopeTokens;
        if (row >= ro.rows) return;
        int pos[kRopeTokens];
#pragma unroll
        for (int i = 0; i < kRopeTokens; ++i) {
            pos[i] = -1;
            if (row + i < ro.rows) {
                const int b = (int)((row + i) / (unsigned)a.T), t = (int)(row + i - (unsigned)b * a.T);
                const int len = a.seq_lens[b];
                // a sequence that is skipped gets zero rows (the page CTAs report it)
                const bool skipped = len < a.T || len > a.max_pages * (long long)a.ps || (ro.rot > 0 && len > ro.n_pos);
                pos[i] = skipped ? -1 : len - a.T + t;
            }
        }
        rope_warp<D>(ro, ro.q, ro.q_stride, ro.q_out, ro.q_weight, (unit - unit / groups * groups) * HW, ro.H_q, row, pos);
        return;
    }
    const int page_cta = blockIdx.x / head_ctas, h = (blockIdx.x - page_cta * head_ctas) * kPageHeads + warp / kPageParts;
    const int part = warp % kPageParts;
    const int b = page_cta / p.touched;
    const int len = a.seq_lens[b];
    const bool first_cta = page_cta == b * p.touched;
    if (len < a.T || len > a.max_pages * (long long)a.ps) {
        if (threadIdx.x == 0 && first_cta) raise_status(a.status, SPD_DEV_BAD_LEN);
        return;
    }
    if (ro.rot > 0 && len > ro.n_pos) {
        if (threadIdx.x == 0 && first_cta) raise_status(a.status, SPD_DEV_BAD_POS);
        return;
    }
    const int first = len - a.T;  // position of the first new token
    const int pg = first / a.ps + (page_cta - b * p.touched);
    if ((long long)pg * a.ps >= len) return;  // (the page behind a sequence of 2^31 - 1 tokens starts past 32 bits)
    const int valid = min(a.ps, len - pg * a.ps);
    const long long phys = a.page_table[(long long)b * a.max_pages + pg];
    if (phys < 0 || phys >= a.num_phys) {
        if (threadIdx.x == 0) raise_status(a.status, SPD_DEV_BAD_PAGE);
        return;
    }
    const int r0 = lane / L, l = lane % L;
    const RopeLane rl = rope_lane<D>(l, ro.rot, ro.interleaved);
    float wk[8];
    rope_weights(ro.k_weight, rl, wk);
    const __nv_bfloat162 pinf = __floats2bfloat162_rn(__int_as_float(0x7f800000), __int_as_float(0x7f800000));
    const __nv_bfloat162 ninf = __floats2bfloat162_rn(__int_as_float(0xff800000), __int_as_float(0xff800000));
    const int nold = min(valid, max(0, first - pg * a.ps));
    __nv_bfloat162 mn[4], mx[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        mn[i] = pinf;
        mx[i] = ninf;
    }
    if (h < a.H_kv) {
        const long long row0 = (phys * a.H_kv + h) * a.ps;
        uint16_t* kt = a.K + row0 * D;
        uint16_t* vt = a.V + row0 * D;
        auto fold = [&](const uint2& u0, const uint2& u1) {
            const uint32_t e[4] = {u0.x, u0.y, u1.x, u1.y};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&e[i]);
                mn[i] = __hmin2(mn[i], v);
                mx[i] = __hmax2(mx[i], v);
            }
        };
        for (int t0 = part * RPI + r0; t0 < nold; t0 += kOldBatch * STEP) {
            uint2 k0[kOldBatch], k1[kOldBatch];
#pragma unroll
            for (int u = 0; u < kOldBatch; ++u)
                if (t0 + u * STEP < nold) {
                    k0[u] = *reinterpret_cast<const uint2*>(kt + (t0 + u * STEP) * D + rl.o0);
                    k1[u] = *reinterpret_cast<const uint2*>(kt + (t0 + u * STEP) * D + rl.o1);
                }
#pragma unroll
            for (int u = 0; u < kOldBatch; ++u)
                if (t0 + u * STEP < nold) fold(k0[u], k1[u]);
        }
        // new rows: kNewBatch loads of keys, values and angles in flight a lane, then the rows
        // by the whole warp (the norm's shuffles)
        const uint16_t* ks = ro.k + ((long long)b * a.T - first + pg * a.ps) * ro.k_stride + h * D;
        const uint16_t* vs = p.v + ((long long)b * a.T - first + pg * a.ps) * p.v_stride + h * D + 8 * l;
        const float* angles = ro.table + (long long)pg * a.ps * ro.rot + 4 * l;
        for (int tb = nold + part * RPI; tb < valid; tb += kNewBatch * STEP) {
            uint2 k0[kNewBatch], k1[kNewBatch];
            uint4 v[kNewBatch];
            float4 cs[kNewBatch], sn[kNewBatch];
#pragma unroll
            for (int u = 0; u < kNewBatch; ++u) {
                const int t = tb + u * STEP + r0;
                k0[u] = k1[u] = make_uint2(0u, 0u);
                cs[u] = sn[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (t < valid) {
                    k0[u] = *reinterpret_cast<const uint2*>(ks + t * ro.k_stride + rl.o0);
                    k1[u] = *reinterpret_cast<const uint2*>(ks + t * ro.k_stride + rl.o1);
                    v[u] = *reinterpret_cast<const uint4*>(vs + t * p.v_stride);
                    if (rl.turned) {
                        cs[u] = __ldg(reinterpret_cast<const float4*>(angles + t * ro.rot));
                        sn[u] = __ldg(reinterpret_cast<const float4*>(angles + t * ro.rot + (ro.rot >> 1)));
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < kNewBatch; ++u) {
                const int t = tb + u * STEP + r0;
                if (tb + u * STEP >= valid) break;
                float x[8];
                unpack4(k0[u], x);
                unpack4(k1[u], x + 4);
                rope_row<D>(x, ro.k_weight != nullptr, wk, ro.eps, rl, ro.interleaved, cs[u], sn[u]);
                if (t < valid) {
                    const uint2 u0 = pack4(x), u1 = pack4(x + 4);
                    *reinterpret_cast<uint2*>(kt + t * D + rl.o0) = u0;
                    *reinterpret_cast<uint2*>(kt + t * D + rl.o1) = u1;
                    *reinterpret_cast<uint4*>(vt + t * D + 8 * l) = v[u];
                    fold(u0, u1);
                }
            }
        }
#pragma unroll
        for (int off = L; off < 32; off <<= 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t a_ = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t*>(&mn[i]), off);
                uint32_t b_ = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t*>(&mx[i]), off);
                mn[i] = __hmin2(mn[i], *reinterpret_cast<__nv_bfloat162*>(&a_));
                mx[i] = __hmax2(mx[i], *reinterpret_cast<__nv_bfloat162*>(&b_));
            }
        }
        if (r0 == 0) {
            s_mm[warp][l][0] = *reinterpret_cast<uint4*>(mn);
            s_mm[warp][l][1] = *reinterpret_cast<uint4*>(mx);
        }
    }
    __syncthreads();
    if (part == 0 && r0 == 0 && h < a.H_kv) {
#pragma unroll
        for (int q = 1; q < kPageParts; ++q) {
            const uint4 n = s_mm[warp + q][l][0], x = s_mm[warp + q][l][1];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mn[i] = __hmin2(mn[i], reinterpret_cast<const __nv_bfloat162*>(&n)[i]);
                mx[i] = __hmax2(mx[i], reinterpret_cast<const __nv_bfloat162*>(&x)[i]);
            }
        }
        uint16_t* out = a.summ + (((long long)b * a.H_kv + h) * a.max_pages + pg) * 2LL * D;
        const uint32_t* n = reinterpret_cast<const uint32_t*>(mn);
        const uint32_t* x = reinterpret_cast<const uint32_t*>(mx);
        *reinterpret_cast<uint2*>(out + rl.o0) = make_uint2(n[0], n[1]);
        *reinterpret_cast<uint2*>(out + rl.o1) = make_uint2(n[2], n[3]);
        *reinterpret_cast<uint2*>(out + D + rl.o0) = make_uint2(x[0], x[1]);
        *reinterpret_cast<uint2*>(out + D + rl.o1) = make_uint2(x[2], x[3]);
    }
}

long long append_rope_ctas(const AppendRopeArgs& p) {
    const int hw = rope_heads_per_warp(p.append.D);
    const long long units = p.rope.q ? (p.rope.rows + kRopeTokens - 1) / kRopeTokens * ((p.rope.H_q + hw - 1) / hw) : 0;
    return (long long)p.append.B * append_touched(p.append.T, p.append.ps, p.append.max_pages) *
               ((p.append.H_kv + kPageHeads - 1) / kPageHeads) +
           (units + kRopeWarps - 1) / kRopeWarps;
}

cudaError_t launch_append_rope(const AppendRopeArgs& in, cudaStream_t st) {
    AppendRopeArgs p = in;
    p.touched = append_touched(p.append.T, p.append.ps, p.append.max_pages);
    dim3 grid((unsigned)append_rope_ctas(p)), block(kRopeThreads);
    if (p.append.D == 128) return launch_pdl(append_rope_kernel<128>, grid, block, 0, st, p);
    return launch_pdl(append_rope_kernel<64>, grid, block, 0, st, p);
}

}  // namespace spd
