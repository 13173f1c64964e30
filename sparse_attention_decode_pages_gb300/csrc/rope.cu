// rope.cu -- queries and keys of new tokens on their way from the projection to
// the attention: norm of each head's row and position rotation in one pass
// (qk_norm_rope), and the same with the keys and values written into the paged
// cache and the touched pages' key summaries rebuilt (kv_append_rope).
//
// Both read every element once and write it once; what bounds them is memory
// for long prompts and the launch for single tokens.
#include "rope.cuh"

namespace spd {

// One unit = kHeadsPerUnit heads of one token, held by D / 8 lanes: the token's
// angles and the heads' loads are all in flight together.
constexpr int kHeadsPerUnit = 4;
constexpr int kRopeThreads = 256;

template <int D>
__device__ __forceinline__ void rope_unit(const RopeArgs& a, long long unit, int lane_in_unit, long long row, int pos,
                                          bool live) {
    const int heads = a.H_q + a.H_kv;
    const int per_row = (heads + kHeadsPerUnit - 1) / kHeadsPerUnit;
    const int h0 = (int)(unit - row * per_row) * kHeadsPerUnit;
    const RopeLane r = rope_lane<D>(lane_in_unit, a.rot, a.interleaved);
    const bool bad = live && a.rot > 0 && (pos < 0 || pos >= a.n_pos);
    if (bad && lane_in_unit == 0) raise_status(a.status, SPD_DEV_BAD_POS);
    float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live && !bad && r.turned) {
        const float* t = a.table + (long long)pos * a.rot + 4 * lane_in_unit;
        cs = __ldg(reinterpret_cast<const float4*>(t));
        sn = __ldg(reinterpret_cast<const float4*>(t + (a.rot >> 1)));
    }
    uint2 x0[kHeadsPerUnit], x1[kHeadsPerUnit];
#pragma unroll
    for (int i = 0; i < kHeadsPerUnit; ++i) {
        const int h = h0 + i;
        x0[i] = x1[i] = make_uint2(0u, 0u);
        if (live && h < heads) {
            const uint16_t* src = h < a.H_q ? a.q + row * a.q_stride + h * D : a.k + row * a.k_stride + (h - a.H_q) * D;
            x0[i] = *reinterpret_cast<const uint2*>(src + r.o0);
            x1[i] = *reinterpret_cast<const uint2*>(src + r.o1);
        }
    }
    float wq[8], wk[8];
    rope_weights(a.q_weight, r, wq);
    rope_weights(a.k_weight, r, wk);
#pragma unroll
    for (int i = 0; i < kHeadsPerUnit; ++i) {
        const int h = h0 + i;
        const bool is_q = h < a.H_q;
        const bool norm = is_q ? a.q_weight != nullptr : a.k_weight != nullptr;
        float x[8], w[8];
        unpack4(x0[i], x);
        unpack4(x1[i], x + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = is_q ? wq[j] : wk[j];
        rope_row<D>(x, a.q_weight != nullptr || a.k_weight != nullptr, norm, w, a.eps, r, a.interleaved, cs, sn);
        if (live && h < heads) {
            uint16_t* dst = is_q ? a.q_out + (row * a.H_q + h) * D : a.k_out + (row * a.H_kv + (h - a.H_q)) * D;
            *reinterpret_cast<uint2*>(dst + r.o0) = bad ? make_uint2(0u, 0u) : pack4(x);
            *reinterpret_cast<uint2*>(dst + r.o1) = bad ? make_uint2(0u, 0u) : pack4(x + 4);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int L = D / 8;
    pdl_wait();
    pdl_trigger();
    const int per_row = (a.H_q + a.H_kv + kHeadsPerUnit - 1) / kHeadsPerUnit;
    const long long unit = (long long)blockIdx.x * (kRopeThreads / L) + threadIdx.x / L;
    const long long row = unit / per_row;
    const bool live = row < a.rows;
    const int pos = live && a.rot > 0 ? a.positions[row] : 0;
    rope_unit<D>(a, unit, threadIdx.x % L, live ? row : 0, pos, live);
}

cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t st) {
    const long long per_row = (a.H_q + a.H_kv + kHeadsPerUnit - 1) / kHeadsPerUnit;
    const long long units = a.rows * per_row;
    const int upb = kRopeThreads / (a.D / 8);
    dim3 grid((unsigned)((units + upb - 1) / upb)), block(kRopeThreads);
    if (a.D == 128) return launch_pdl(qk_norm_rope_kernel<128>, grid, block, 0, st, a);
    return launch_pdl(qk_norm_rope_kernel<64>, grid, block, 0, st, a);
}

// kv_append_rope: one grid of two kinds of CTA.  The first B * touched CTAs are the
// append's, one per (sequence, touched page), a warp per KV head: the page's rows
// are visited once, older keys read from the cache and new ones normalised,
// rotated and stored, and the channel-wise min / max of all valid rows, as rounded,
// becomes the page's summary.  The CTAs behind them take the query heads in the
// units of qk_norm_rope.
template <int D>
__global__ void __launch_bounds__(kRopeThreads) append_rope_kernel(const AppendRopeArgs p) {
    constexpr int L = D / 8;        // lanes per row
    constexpr int RPI = 32 / L;     // rows per warp instruction
    const AppendArgs& a = p.append;
    const RopeArgs& ro = p.rope;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    pdl_wait();
    pdl_trigger();
    const int page_ctas = a.B * p.touched;
    if ((int)blockIdx.x >= page_ctas) {
        // query heads of token row = b * T + t at position len - T + t
        const int per_row = (ro.H_q + kHeadsPerUnit - 1) / kHeadsPerUnit;
        const long long unit = (long long)(blockIdx.x - page_ctas) * (blockDim.x / L) + threadIdx.x / L;
        const long long row = unit / per_row;
        const bool live = row < ro.rows;
        int pos = 0;
        if (live) {
            const int b = (int)(row / a.T), t = (int)(row - (long long)b * a.T);
            const int len = a.seq_lens[b];
            // a sequence that is skipped gets zero rows: an angle that the table does not hold
            pos = (len < a.T || len > a.max_pages * (long long)a.ps) ? -1 : len - a.T + t;
            if (pos >= 0 && ro.rot > 0 && len > ro.n_pos) pos = -1;
        }
        RopeArgs q = ro;
        q.H_kv = 0;
        q.status = nullptr;  // the page CTAs report
        rope_unit<D>(q, unit, threadIdx.x % L, live ? row : 0, pos, live);
        if (live && pos < 0 && ro.rot == 0) {  // no rotation: nothing above looked at the position
            const int h0 = (int)(unit - row * per_row) * kHeadsPerUnit;
            for (int h = h0; h < min(h0 + kHeadsPerUnit, ro.H_q); ++h)
                *reinterpret_cast<uint4*>(ro.q_out + (row * ro.H_q + h) * D + 8 * (threadIdx.x % L)) =
                    make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    const int b = blockIdx.x / p.touched;
    const int len = a.seq_lens[b];
    const bool first_cta = blockIdx.x % p.touched == 0;
    if (len < a.T || len > a.max_pages * (long long)a.ps) {
        if (threadIdx.x == 0 && first_cta) raise_status(a.status, SPD_DEV_BAD_LEN);
        return;
    }
    if (ro.rot > 0 && len > ro.n_pos) {
        if (threadIdx.x == 0 && first_cta) raise_status(a.status, SPD_DEV_BAD_POS);
        return;
    }
    const int first = len - a.T;  // position of the first new token
    const int pg = first / a.ps + (int)(blockIdx.x % p.touched);
    if (pg * a.ps >= len) return;
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
    for (int h = warp; h < a.H_kv; h += nwarps) {
        const long long row0 = (phys * a.H_kv + h) * a.ps;
        uint16_t* kt = a.K + row0 * D;
        uint16_t* vt = a.V + row0 * D;
        __nv_bfloat162 mn[4], mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mn[i] = pinf;
            mx[i] = ninf;
        }
        auto fold = [&](const uint2& u0, const uint2& u1) {
            const uint32_t e[4] = {u0.x, u0.y, u1.x, u1.y};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&e[i]);
                mn[i] = __hmin2(mn[i], v);
                mx[i] = __hmax2(mx[i], v);
            }
        };
        for (int t0 = r0; t0 < nold; t0 += kAppendBatch * RPI) {
            uint2 k0[kAppendBatch], k1[kAppendBatch];
#pragma unroll
            for (int u = 0; u < kAppendBatch; ++u)
                if (t0 + u * RPI < nold) {
                    k0[u] = *reinterpret_cast<const uint2*>(kt + (t0 + u * RPI) * D + rl.o0);
                    k1[u] = *reinterpret_cast<const uint2*>(kt + (t0 + u * RPI) * D + rl.o1);
                }
#pragma unroll
            for (int u = 0; u < kAppendBatch; ++u)
                if (t0 + u * RPI < nold) fold(k0[u], k1[u]);
        }
        // new rows, RPI at a time by the whole warp (the norm's shuffles)
        for (int tb = nold; tb < valid; tb += RPI) {
            const int t = tb + r0;
            const bool live = t < valid;
            const long long row = (long long)b * a.T + (pg * a.ps + t - first);
            uint2 u0 = make_uint2(0u, 0u), u1 = u0;
            float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (live) {
                const uint16_t* src = ro.k + row * ro.k_stride + h * D;
                u0 = *reinterpret_cast<const uint2*>(src + rl.o0);
                u1 = *reinterpret_cast<const uint2*>(src + rl.o1);
                v = *reinterpret_cast<const uint4*>(p.v + row * p.v_stride + h * D + 8 * l);
                if (rl.turned) {
                    const float* tb_ = ro.table + (long long)(pg * a.ps + t) * ro.rot + 4 * l;
                    cs = __ldg(reinterpret_cast<const float4*>(tb_));
                    sn = __ldg(reinterpret_cast<const float4*>(tb_ + (ro.rot >> 1)));
                }
            }
            float x[8];
            unpack4(u0, x);
            unpack4(u1, x + 4);
            rope_row<D>(x, ro.k_weight != nullptr, true, wk, ro.eps, rl, ro.interleaved, cs, sn);
            if (live) {
                u0 = pack4(x);
                u1 = pack4(x + 4);
                *reinterpret_cast<uint2*>(kt + t * D + rl.o0) = u0;
                *reinterpret_cast<uint2*>(kt + t * D + rl.o1) = u1;
                *reinterpret_cast<uint4*>(vt + t * D + 8 * l) = v;
                fold(u0, u1);
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
            uint16_t* out = a.summ + (((long long)b * a.H_kv + h) * a.max_pages + pg) * 2LL * D;
            const uint32_t* n = reinterpret_cast<const uint32_t*>(mn);
            const uint32_t* x = reinterpret_cast<const uint32_t*>(mx);
            *reinterpret_cast<uint2*>(out + rl.o0) = make_uint2(n[0], n[1]);
            *reinterpret_cast<uint2*>(out + rl.o1) = make_uint2(n[2], n[3]);
            *reinterpret_cast<uint2*>(out + D + rl.o0) = make_uint2(x[0], x[1]);
            *reinterpret_cast<uint2*>(out + D + rl.o1) = make_uint2(x[2], x[3]);
        }
    }
}

long long append_rope_ctas(const AppendRopeArgs& p) {
    const long long per_row = (p.rope.H_q + kHeadsPerUnit - 1) / kHeadsPerUnit;
    const int upb = kRopeThreads / (p.append.D / 8);
    const long long q_ctas = p.rope.q ? (p.rope.rows * per_row + upb - 1) / upb : 0;
    return (long long)p.append.B * append_touched(p.append.T, p.append.ps, p.append.max_pages) + q_ctas;
}

cudaError_t launch_append_rope(const AppendRopeArgs& in, cudaStream_t st) {
    AppendRopeArgs p = in;
    p.touched = append_touched(p.append.T, p.append.ps, p.append.max_pages);
    dim3 grid((unsigned)append_rope_ctas(p)), block(kRopeThreads);
    if (p.append.D == 128) return launch_pdl(append_rope_kernel<128>, grid, block, 0, st, p);
    return launch_pdl(append_rope_kernel<64>, grid, block, 0, st, p);
}

}  // namespace spd
