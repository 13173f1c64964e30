// kv4.cu -- the 4-bit paged cache's writer and reader: kv4_append quantises the T
// newest tokens' keys and values into the cache and rebuilds the key summaries of
// the pages they land in (over the values as held, so the scores bound the logits
// that the attention computes); kv4_read gives the T newest tokens back as bf16.
#include "kv4.cuh"
#include "kernels.h"

namespace spd {

constexpr int kKv4Threads = 256;
// Groups of new rows whose loads an appending lane keeps in flight, and of older ones.
constexpr int kNewBatch = 2;
constexpr int kOldBatch = 2;
constexpr int kPageHeads = 2;  // KV heads of an append's CTA
constexpr int kPageParts = kKv4Threads / 32 / kPageHeads;  // warps of a head

// The lane's eight channels of a row as four bf16 pairs, from its four bytes of codes
// and its group's scale byte.
__device__ __forceinline__ uint4 kv4_values(uint32_t codes, uint32_t scale_byte, float exp2) {
    uint32_t h[4];
    e2m1x8_to_f16(codes, h);
    const float s = e4m3_value(scale_byte) * exp2;
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        out[i] = pack_bf16(v.x * s, v.y * s);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

// a / s rounded correctly, r = 1 / s rounded correctly (Markstein: the quotient corrected by
// its exact remainder); for the finite magnitudes met here.
__device__ __forceinline__ float quotient(float a, float s, float r) {
    const float q = a * r;
    return fmaf(-fmaf(q, s, -a), r, q);
}

// Quantises the lane's eight channels (its group's other eight are the neighbour
// lane's): codes and the group's scale byte, exp2 = 2^exp.  The scale is the correctly
// rounded one.  Of the quotients x / s only the side of a border m between two codes
// matters.  x is an integer of at most 8 bits times a power of two, and so is m s (3 and
// 4 bits), so x / s is m itself or lies further from it than the rounding to 8 bits, half a
// step of bf16, can move it: x / s rounded to bf16 has the code of x / s.  It is formed in
// bf16 pairs as x rh + x rl with 1 / s = rh + rl to 2^-16, whose error is below the margin (the
// least, 1/240 - 1/256, is at m = 1/4, s = 15) and leaves a border exact.  rh is cut,
// not rounded, so that rl >= 0 and the sum of two zeros keeps x's sign.
__device__ __forceinline__ uint32_t kv4_quantise(const uint4& u, float exp2, float inv_exp2, uint32_t& scale_byte) {
    uint32_t e[4] = {u.x, u.y, u.z, u.w};
    // the largest magnitude, in bf16 pairs (exact); NaN where there is one
    __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&e[0]));
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162*>(&e[i])));
    m = __hmax2_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const float2 mf = __bfloat1622float2(m);
    constexpr float kTop = 6.f * 448.f;  // the largest value a group can hold, over exp2
    float amax = fmaxf(mf.x, mf.y) + 0.f * mf.x + 0.f * mf.y;  // NaN where either is NaN or infinite
    if (!(amax * inv_exp2 <= kTop)) {
        // rare: what lies past the largest value that can be held becomes it, NaN zero
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&e[i]));
            v.x = v.x == v.x ? fminf(fmaxf(v.x, -kTop * exp2), kTop * exp2) : 0.f;
            v.y = v.y == v.y ? fminf(fmaxf(v.y, -kTop * exp2), kTop * exp2) : 0.f;
            amax = fmaxf(amax, fmaxf(fabsf(v.x), fabsf(v.y)));
            e[i] = pack_bf16(v.x, v.y);
        }
        // the neighbour came here too: the two have looked at the same m
        amax = fmaxf(amax, __shfl_xor_sync(3u << (threadIdx.x & 30), amax, 1));
    }
    scale_byte = to_e4m3(quotient(amax * inv_exp2, 6.f, 1.f / 6.f));
    const float s1 = e4m3_value(scale_byte);
    const float r = s1 > 0.f ? __frcp_rn(s1) * inv_exp2 : 0.f;  // scale 0: the codes are zeros of x's sign
    const uint32_t rb = __float_as_uint(r), high = __byte_perm(rb, rb, 0x3232);
    const float rest = r - __uint_as_float(rb & 0xffff0000u);
    const __nv_bfloat162 rh = *reinterpret_cast<const __nv_bfloat162*>(&high), rl = __float2bfloat162_rn(rest);
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&e[i]);
        const __nv_bfloat162 q = __hfma2(x, rh, __hmul2_rn(x, rl));
        const uint32_t w = *reinterpret_cast<const uint32_t*>(&q);
        y[2 * i] = __uint_as_float(w << 16);
        y[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
    }
    return to_e2m1x8(y);
}

// One CTA per (sequence, touched page, two KV heads), four warps a head: each takes
// every fourth group of the page's rows, older ones read back from the cache, new ones
// quantised and stored, and the min / max of the values of all valid rows, joined
// through shared memory, becomes the page's summary.  Bound by the instructions of the
// quantisation (issue 70 %).  8 heads of 128, 8 x 2,039 tokens, pages of 32: 23.3 us, 3.7 TB/s, 55 %
// of the measured copy peak (one batch of loads ahead 25.6; 1 / 2 / 4 heads a CTA 42.1 /
// 40.4 / 39.5 us with the reading behind it, but four leave half of the warps idle where
// there are two heads).
template <int D>
__global__ void __launch_bounds__(kKv4Threads, 4) kv4_append_kernel(const Kv4Args a) {
    constexpr int L = D / 8;     // lanes per row
    constexpr int RPI = 32 / L;  // rows per warp instruction
    constexpr int STEP = kPageParts * RPI;
    __shared__ uint4 s_mm[kKv4Threads / 32][L][2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head_ctas = (a.H_kv + kPageHeads - 1) / kPageHeads;
    const int b = blockIdx.x / head_ctas, h = (blockIdx.x - b * head_ctas) * kPageHeads + warp / kPageParts;
    const int part = warp % kPageParts;
    pdl_wait();
    pdl_trigger();
    const int len = a.seq_lens[b];
    if (len < a.T || len > (long long)a.max_pages * a.ps) {
        if (threadIdx.x == 0 && blockIdx.y == 0) raise_status(a.status, SPD_DEV_BAD_LEN);
        return;
    }
    const int first = len - a.T;
    const int p = first / a.ps + (int)blockIdx.y;
    if (p >= a.max_pages || (long long)p * a.ps >= len) return;
    const int valid = min(a.ps, len - p * a.ps);
    const long long phys = a.page_table[(long long)b * a.max_pages + p];
    if (phys < 0 || phys >= a.num_phys) {
        if (threadIdx.x == 0) raise_status(a.status, SPD_DEV_BAD_PAGE);
        return;
    }
    const int r0 = lane / L, l = lane % L;
    const int half = kv4_half_bytes(a.ps, D), codes_bytes = kv4_codes_bytes(a.ps, D);
    const float k2 = pow2f(a.k_exp), ik2 = pow2f(-a.k_exp), v2 = pow2f(a.v_exp), iv2 = pow2f(-a.v_exp);
    const __half2 pinf = __floats2half2_rn(__int_as_float(0x7f800000), __int_as_float(0x7f800000));
    const __half2 ninf = __floats2half2_rn(__int_as_float(0xff800000), __int_as_float(0xff800000));
    const int nold = min(valid, max(0, first - p * a.ps));
    __half2 mn[4], mx[4];  // of code * scale, exact in fp16
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        mn[i] = pinf;
        mx[i] = ninf;
    }
    if (h < a.H_kv) {
        uint8_t* kt = a.kv4 + (phys * a.H_kv + h) * (2LL * half);
        uint8_t* vt = kt + half;
        auto fold = [&](uint32_t codes, uint32_t scale) {
            uint32_t c4[4];
            e2m1x8_to_f16(codes, c4);
            const uint32_t s2 = e4m3x2_to_f16(scale * 0x101u);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t v = hmul2(c4[i], s2);
                mn[i] = __hmin2(mn[i], *reinterpret_cast<const __half2*>(&v));
                mx[i] = __hmax2(mx[i], *reinterpret_cast<const __half2*>(&v));
            }
        };
        for (int t0 = part * RPI + r0; t0 < nold; t0 += kOldBatch * STEP) {
            uint32_t c[kOldBatch], s[kOldBatch];
#pragma unroll
            for (int u = 0; u < kOldBatch; ++u)
                if (t0 + u * STEP < nold) {
                    c[u] = *reinterpret_cast<const uint32_t*>(kt + (t0 + u * STEP) * (D / 2) + 4 * l);
                    s[u] = kt[codes_bytes + (t0 + u * STEP) * (D / 16) + l / 2];
                }
#pragma unroll
            for (int u = 0; u < kOldBatch; ++u)
                if (t0 + u * STEP < nold) fold(c[u], s[u]);
        }
        // new rows: kNewBatch loads in flight a lane, then by the whole warp (the groups' maxima
        // are exchanged)
        const long long src = (((long long)b * a.T + (p * a.ps - first)) * a.H_kv + h) * (D / 8) + l;
        for (int tb = nold + part * RPI; tb < valid; tb += kNewBatch * STEP) {
            uint4 k[kNewBatch], v[kNewBatch];
#pragma unroll
            for (int u = 0; u < kNewBatch; ++u) {
                const int t = tb + u * STEP + r0;
                k[u] = v[u] = make_uint4(0u, 0u, 0u, 0u);
                if (t < valid) {
                    k[u] = __ldg(reinterpret_cast<const uint4*>(a.k_new) + src + (long long)t * a.H_kv * (D / 8));
                    v[u] = __ldg(reinterpret_cast<const uint4*>(a.v_new) + src + (long long)t * a.H_kv * (D / 8));
                }
            }
#pragma unroll
            for (int u = 0; u < kNewBatch; ++u) {
                const int t = tb + u * STEP + r0;
                if (tb + u * STEP >= valid) break;
                uint32_t ks, vs;
                const uint32_t kc = kv4_quantise(k[u], k2, ik2, ks);
                const uint32_t vc = kv4_quantise(v[u], v2, iv2, vs);
                if (t < valid) {
                    *reinterpret_cast<uint32_t*>(kt + t * (D / 2) + 4 * l) = kc;
                    *reinterpret_cast<uint32_t*>(vt + t * (D / 2) + 4 * l) = vc;
                    if (!(l & 1)) {
                        kt[codes_bytes + t * (D / 16) + l / 2] = (uint8_t)ks;
                        vt[codes_bytes + t * (D / 16) + l / 2] = (uint8_t)vs;
                    }
                    fold(kc, ks);
                }
            }
        }
#pragma unroll
        for (int off = L; off < 32; off <<= 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mn[i] = __hmin2(mn[i], __shfl_xor_sync(0xffffffffu, mn[i], off));
                mx[i] = __hmax2(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], off));
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
                mn[i] = __hmin2(mn[i], reinterpret_cast<const __half2*>(&n)[i]);
                mx[i] = __hmax2(mx[i], reinterpret_cast<const __half2*>(&x)[i]);
            }
        }
        uint4* out = reinterpret_cast<uint4*>(a.summ + (((long long)b * a.H_kv + h) * a.max_pages + p) * 2LL * D);
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = __half22float2(mn[i]), y = __half22float2(mx[i]);
            lo[i] = pack_bf16(x.x * k2, x.y * k2);
            hi[i] = pack_bf16(y.x * k2, y.y * k2);
        }
        out[l] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        out[L + l] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
}

cudaError_t launch_kv4_append(const Kv4Args& a, cudaStream_t st) {
    dim3 grid((unsigned)((long long)a.B * ((a.H_kv + kPageHeads - 1) / kPageHeads)),
              (unsigned)append_touched(a.T, a.ps, a.max_pages));
    dim3 block(kKv4Threads);
    if (a.D == 128) return launch_pdl(kv4_append_kernel<128>, grid, block, 0, st, a);
    return launch_pdl(kv4_append_kernel<64>, grid, block, 0, st, a);
}

// A warp takes one token's KV heads, D / 8 lanes a head and kReadTurns heads a lane group
// whose loads are in flight together; its group of heads is blockIdx.y.  Bound by memory:
// 8 heads of 128, 8 x 2,039 tokens: 16.2 us, 5.4 TB/s, 79 % of the measured copy peak
// (2 / 4 / 8 turns: 16.5 / 16.2 / 16.9 us).
constexpr int kReadTurns = 4;

template <int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(const Kv4Args a) {
    constexpr int L = D / 8, HT = 32 / L;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, l = lane % L, h0 = blockIdx.y * (HT * kReadTurns) + lane / L;
    const unsigned row = blockIdx.x * (kKv4Threads / 32) + (threadIdx.x >> 5);  // b * T + t
    const unsigned b = row / (unsigned)a.T;
    if (b >= (unsigned)a.B) return;
    const int t = (int)(row - b * a.T), len = a.seq_lens[b];
    long long phys = -1;
    int slot = 0;
    if (len < a.T || len > (long long)a.max_pages * a.ps) {
        if (lane == 0) raise_status(a.status, SPD_DEV_BAD_LEN);
    } else {
        const unsigned pos = len - a.T + t, p = pos / (unsigned)a.ps;
        slot = (int)(pos - p * a.ps);
        phys = a.page_table[(long long)b * a.max_pages + p];
        if (phys < 0 || phys >= a.num_phys) {
            if (lane == 0) raise_status(a.status, SPD_DEV_BAD_PAGE);
            phys = -1;
        }
    }
    const int half = kv4_half_bytes(a.ps, D), codes_bytes = kv4_codes_bytes(a.ps, D);
    const uint8_t* tile = a.kv4 + (phys < 0 ? 0 : phys * a.H_kv + h0) * (2LL * half);
    const int co = slot * (D / 2) + 4 * l, so = codes_bytes + slot * (D / 16) + l / 2;
    uint32_t kc[kReadTurns], ks[kReadTurns], vc[kReadTurns], vs[kReadTurns];
#pragma unroll
    for (int i = 0; i < kReadTurns; ++i) {
        kc[i] = ks[i] = vc[i] = vs[i] = 0u;
        if (phys >= 0 && h0 + i * HT < a.H_kv) {
            const uint8_t* kt = tile + i * HT * (2LL * half);
            kc[i] = *reinterpret_cast<const uint32_t*>(kt + co);
            ks[i] = kt[so];
            vc[i] = *reinterpret_cast<const uint32_t*>(kt + half + co);
            vs[i] = kt[half + so];
        }
    }
    const float k2 = pow2f(a.k_exp), v2 = pow2f(a.v_exp);
    const long long at = ((long long)row * a.H_kv + h0) * L + l;
#pragma unroll
    for (int i = 0; i < kReadTurns; ++i)
        if (h0 + i * HT < a.H_kv) {
            reinterpret_cast<uint4*>(a.k_out)[at + i * HT * L] = kv4_values(kc[i], ks[i], k2);
            reinterpret_cast<uint4*>(a.v_out)[at + i * HT * L] = kv4_values(vc[i], vs[i], v2);
        }
}

cudaError_t launch_kv4_read(const Kv4Args& a, cudaStream_t st) {
    const long long rows = (long long)a.B * a.T;
    const int warps = kKv4Threads / 32, heads = 32 / (a.D / 8) * kReadTurns;
    dim3 grid((unsigned)((rows + warps - 1) / warps), (unsigned)((a.H_kv + heads - 1) / heads)), block(kKv4Threads);
    if (a.D == 128) return launch_pdl(kv4_read_kernel<128>, grid, block, 0, st, a);
    return launch_pdl(kv4_read_kernel<64>, grid, block, 0, st, a);
}

}  // namespace spd
