// kv4.cu -- the 4-bit paged cache's writer and reader: kv4_append quantises the T
// newest tokens' keys and values into the cache and rebuilds the key summaries of
// the pages they land in (over the values as held, so the scores bound the logits
// that the attention computes); kv4_read gives the T newest tokens back as bf16.
#include "kv4.cuh"
#include "kernels.h"

namespace spd {

constexpr int kKv4Threads = 256;

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

// Quantises the lane's eight channels (its group's other eight are the neighbour
// lane's): codes and the group's scale byte.  Divisions are rounded correctly, so the
// codes are those of the exact quotients: a border between codes times a scale has
// few enough bits that no rounded quotient crosses it.
__device__ __forceinline__ uint32_t kv4_quantise(const uint4& u, float inv_exp2, uint32_t& scale_byte) {
    const __nv_bfloat162* e = reinterpret_cast<const __nv_bfloat162*>(&u);
    float x[8];
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __bfloat1622float2(e[i]);
        x[2 * i] = v.x * inv_exp2;
        x[2 * i + 1] = v.y * inv_exp2;
        amax = fmaxf(amax, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));  // NaN counts as 0
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    scale_byte = to_e4m3(__fdiv_rn(amax, 6.f));
    const float s = e4m3_value(scale_byte);
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float v = x[2 * i + j];
            y[j] = s > 0.f ? __fdiv_rn(v, s) : copysignf(0.f, v);
            if (!(v == v)) y[j] = 0.f;
        }
        codes |= to_e2m1x2(y[0], y[1]) << (8 * i);
    }
    return codes;
}

// One CTA per (sequence, touched page), a warp per KV head, as in kv_append_refresh:
// older rows are read back from the cache, new ones quantised and stored, and the
// min / max of the values of all valid rows becomes the page's summary.
template <int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_append_kernel(const Kv4Args a) {
    constexpr int L = D / 8;     // lanes per row
    constexpr int RPI = 32 / L;  // rows per warp instruction
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const int b = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    const int len = a.seq_lens[b];
    if (len < a.T || len > (long long)a.max_pages * a.ps) {
        if (threadIdx.x == 0 && blockIdx.y == 0) raise_status(a.status, SPD_DEV_BAD_LEN);
        return;
    }
    const int first = len - a.T;
    const int p = first / a.ps + (int)blockIdx.y;
    if (p >= a.max_pages || p * a.ps >= len) return;
    const int valid = min(a.ps, len - p * a.ps);
    const long long phys = a.page_table[(long long)b * a.max_pages + p];
    if (phys < 0 || phys >= a.num_phys) {
        if (threadIdx.x == 0) raise_status(a.status, SPD_DEV_BAD_PAGE);
        return;
    }
    const int r0 = lane / L, l = lane % L;
    const int half = kv4_half_bytes(a.ps, D), codes_bytes = kv4_codes_bytes(a.ps, D);
    const float k2 = pow2f(a.k_exp), ik2 = pow2f(-a.k_exp), iv2 = pow2f(-a.v_exp);
    const __nv_bfloat162 pinf = __floats2bfloat162_rn(__int_as_float(0x7f800000), __int_as_float(0x7f800000));
    const __nv_bfloat162 ninf = __floats2bfloat162_rn(__int_as_float(0xff800000), __int_as_float(0xff800000));
    const int nold = min(valid, max(0, first - p * a.ps));
    for (int h = warp; h < a.H_kv; h += nwarps) {
        uint8_t* kt = a.kv4 + (phys * a.H_kv + h) * (2LL * half);
        uint8_t* vt = kt + half;
        __nv_bfloat162 mn[4], mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mn[i] = pinf;
            mx[i] = ninf;
        }
        auto fold = [&](uint32_t codes, uint32_t scale) {
            const uint4 v = kv4_values(codes, scale, k2);
            const __nv_bfloat162* e = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mn[i] = __hmin2(mn[i], e[i]);
                mx[i] = __hmax2(mx[i], e[i]);
            }
        };
        for (int t0 = r0; t0 < nold; t0 += kAppendBatch * RPI) {
            uint32_t c[kAppendBatch], s[kAppendBatch];
#pragma unroll
            for (int u = 0; u < kAppendBatch; ++u)
                if (t0 + u * RPI < nold) {
                    c[u] = *reinterpret_cast<const uint32_t*>(kt + (t0 + u * RPI) * (D / 2) + 4 * l);
                    s[u] = kt[codes_bytes + (t0 + u * RPI) * (D / 16) + l / 2];
                }
#pragma unroll
            for (int u = 0; u < kAppendBatch; ++u)
                if (t0 + u * RPI < nold) fold(c[u], s[u]);
        }
        for (int tb = nold; tb < valid; tb += RPI) {  // by the whole warp: the groups' maxima are exchanged
            const int t = tb + r0;
            const bool live = t < valid;
            uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
            if (live) {
                const long long src = (((long long)b * a.T + (p * a.ps + t - first)) * a.H_kv + h) * (D / 8) + l;
                k = __ldg(reinterpret_cast<const uint4*>(a.k_new) + src);
                v = __ldg(reinterpret_cast<const uint4*>(a.v_new) + src);
            }
            uint32_t ks, vs;
            const uint32_t kc = kv4_quantise(k, ik2, ks);
            const uint32_t vc = kv4_quantise(v, iv2, vs);
            if (live) {
                *reinterpret_cast<uint32_t*>(kt + t * (D / 2) + 4 * l) = kc;
                *reinterpret_cast<uint32_t*>(vt + t * (D / 2) + 4 * l) = vc;
                if (!(l & 1)) {
                    kt[codes_bytes + t * (D / 16) + l / 2] = (uint8_t)ks;
                    vt[codes_bytes + t * (D / 16) + l / 2] = (uint8_t)vs;
                }
                fold(kc, ks);
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
            uint4* out = reinterpret_cast<uint4*>(
                a.summ + (((long long)b * a.H_kv + h) * a.max_pages + p) * 2LL * D);
            out[l] = *reinterpret_cast<uint4*>(mn);
            out[L + l] = *reinterpret_cast<uint4*>(mx);
        }
    }
}

cudaError_t launch_kv4_append(const Kv4Args& a, cudaStream_t st) {
    dim3 grid((unsigned)a.B, (unsigned)append_touched(a.T, a.ps, a.max_pages));
    dim3 block(32 * (a.H_kv < 8 ? a.H_kv : 8));
    if (a.D == 128) return launch_pdl(kv4_append_kernel<128>, grid, block, 0, st, a);
    return launch_pdl(kv4_append_kernel<64>, grid, block, 0, st, a);
}

// D / 8 lanes per (token, KV head) row, the keys' and the values' eight channels each.
template <int D>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(const Kv4Args a) {
    constexpr int L = D / 8;
    pdl_wait();
    pdl_trigger();
    const long long unit = (long long)blockIdx.x * (kKv4Threads / L) + threadIdx.x / L;
    const int l = threadIdx.x % L;
    const long long row = unit / a.H_kv;  // b * T + t
    const int h = (int)(unit - row * a.H_kv);
    const int b = (int)(row / a.T), t = (int)(row - (long long)b * a.T);
    if (b >= a.B) return;
    const int len = a.seq_lens[b];
    uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
    if (len < a.T || len > (long long)a.max_pages * a.ps) {
        if (l == 0) raise_status(a.status, SPD_DEV_BAD_LEN);
    } else {
        const int pos = len - a.T + t, p = pos / a.ps, slot = pos % a.ps;
        const long long phys = a.page_table[(long long)b * a.max_pages + p];
        if (phys < 0 || phys >= a.num_phys) {
            if (l == 0) raise_status(a.status, SPD_DEV_BAD_PAGE);
        } else {
            const int half = kv4_half_bytes(a.ps, D), codes_bytes = kv4_codes_bytes(a.ps, D);
            const uint8_t* kt = a.kv4 + (phys * a.H_kv + h) * (2LL * half);
            const uint8_t* vt = kt + half;
            const int co = slot * (D / 2) + 4 * l, so = codes_bytes + slot * (D / 16) + l / 2;
            k = kv4_values(*reinterpret_cast<const uint32_t*>(kt + co), kt[so], pow2f(a.k_exp));
            v = kv4_values(*reinterpret_cast<const uint32_t*>(vt + co), vt[so], pow2f(a.v_exp));
        }
    }
    const long long at = (row * a.H_kv + h) * L + l;
    reinterpret_cast<uint4*>(a.k_out)[at] = k;
    reinterpret_cast<uint4*>(a.v_out)[at] = v;
}

cudaError_t launch_kv4_read(const Kv4Args& a, cudaStream_t st) {
    const long long units = (long long)a.B * a.T * a.H_kv;
    const int upb = kKv4Threads / (a.D / 8);
    dim3 grid((unsigned)((units + upb - 1) / upb)), block(kKv4Threads);
    if (a.D == 128) return launch_pdl(kv4_read_kernel<128>, grid, block, 0, st, a);
    return launch_pdl(kv4_read_kernel<64>, grid, block, 0, st, a);
}

}  // namespace spd
