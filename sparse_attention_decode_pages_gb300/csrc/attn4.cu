// attn4.cu -- attention over the 4-bit paged cache: sparse decode over the selected
// pages and dense causal verification over the whole cache.
//
// A unit is a run of at most pages_per_split pages of one (sequence, KV head) row;
// it holds all R = T * G query rows of the KV head in n-tiles of eight.  A CTA
// takes one unit, its warps the unit's 16-token chunks in turn.  Per chunk, on the
// tensor cores (mma.sync m16n8k16, fp16 in, fp32 out):
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
// scale).  Online softmax in fp32 in base 2; a column's reference maximum moves only
// when a logit exceeds it by kHead4, and weights carry a factor 2^kBias4 so that what
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

template <int D, int NT>
struct Attn4Cfg {
    static constexpr int NTW = NT < 2 ? NT : 2;     // n-tiles of a warp
    static constexpr int NG = NT / NTW;             // warps that share a chunk's tokens
    static constexpr int TW = NG <= 2 ? 4 : 2;      // chunks in work at once
    static constexpr int WARPS = NG * TW;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int COLS = NT * 8;
    static constexpr int OFF_FAC = 0;                              // float [COLS]: logit scale of each query row
    static constexpr int OFF_M = OFF_FAC + COLS * 4;               // float [TW][COLS]
    static constexpr int OFF_L = OFF_M + TW * COLS * 4;            // float [TW][COLS]
    static constexpr int OFF_Q = OFF_L + TW * COLS * 4;            // half [COLS][D]
    static constexpr int OFF_O = OFF_Q + COLS * D * 2;             // float [TW][COLS][D]
    static constexpr int SMEM = OFF_O + TW * COLS * D * 4;
};

template <int D, int NT, bool SPARSE>
__global__ void __launch_bounds__(Attn4Cfg<D, NT>::THREADS) attn4_kernel(const Attn4Args a) {
    using C = Attn4Cfg<D, NT>;
    constexpr int NTW = C::NTW, TW = C::TW, COLS = C::COLS;
    constexpr int KW = D / 32;  // 32-bit code words of a lane's share of a key row
    constexpr int VW = D / 64;  // and of a value row
    constexpr int MT = D / 16;  // 16-channel m-tiles of O^T
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int s_last;
    float* s_fac = reinterpret_cast<float*>(smem + C::OFF_FAC);
    float* s_m = reinterpret_cast<float*>(smem + C::OFF_M);
    float* s_l = reinterpret_cast<float*>(smem + C::OFF_L);
    __half* s_q = reinterpret_cast<__half*>(smem + C::OFF_Q);
    float* s_o = reinterpret_cast<float*>(smem + C::OFF_O);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int tw = warp % TW, ng = warp / TW;
    const int G = a.H_q / a.H_kv, R = a.T * G;
    const float NEG_INF = __int_as_float(0xff800000);

    const int row = blockIdx.x / a.num_splits, split = blockIdx.x % a.num_splits;
    const int b = row / a.H_kv, h = row - b * a.H_kv;
    auto out_index = [&](int r) -> long long {
        const int t = r / G;
        return ((long long)b * a.T + t) * a.H_q + h * G + (r - t * G);
    };
    pdl_wait();
    pdl_trigger();

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
    const int start = split * a.pages_per_split;
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
    int lim[NTW][2];
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
            const int r = col0 + 2 * c + j;
            fac[n][j] = s_fac[r];
            m[n][j] = NEG_INF;
            l[n][j] = 0.f;
            lim[n][j] = r < R ? len - a.T + r / G : len - 1;
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) oacc[n][i][0] = oacc[n][i][1] = oacc[n][i][2] = oacc[n][i][3] = 0.f;
    }

    const int cpp = a.ps >> 4;  // chunks per page
    const int codes = kv4_codes_bytes(a.ps, D), half = kv4_half_bytes(a.ps, D);
    for (int ci = tw; ci < count * cpp; ci += TW) {
        const int item = ci / cpp, t0 = (ci - item * cpp) * 16;
        const int lp = SPARSE ? a.sel[(long long)row * a.k_max + start + item] : start + item;
        if (lp < 0 || lp >= P) {
            if (lane == 0) raise_status(a.status, SPD_DEV_BAD_SEL);
            continue;
        }
        const long long phys = a.page_table[(long long)b * a.max_pages + lp];
        if (phys < 0 || phys >= a.num_phys) {
            if (lane == 0) raise_status(a.status, SPD_DEV_BAD_PAGE);
            continue;
        }
        const int pos0 = lp * a.ps + t0;
        if (pos0 >= len) continue;
        const uint8_t* kt = a.kv4 + (phys * a.H_kv + h) * (2LL * half);
        const uint8_t* vt = kt + half;
        uint32_t kw[2][KW], vw[4][VW];
        uint32_t ks[2], vs[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int t = t0 + g + 8 * j;
            const uint32_t* p = reinterpret_cast<const uint32_t*>(kt + t * (D / 2) + c * (D / 8));
#pragma unroll
            for (int w = 0; w < KW; ++w) kw[j][w] = p[w];
            if (D == 128)
                ks[j] = *reinterpret_cast<const uint16_t*>(kt + codes + t * 8 + 2 * c);
            else
                ks[j] = kt[codes + t * 4 + c];
        }
        const int valid = len - pos0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int tc = 2 * c + (j & 1) + 8 * (j >> 1), t = t0 + tc;
            const uint32_t* p = reinterpret_cast<const uint32_t*>(vt + t * (D / 2) + g * (D / 16));
#pragma unroll
            for (int w = 0; w < VW; ++w) vw[j][w] = p[w];
            // slots past the sequence's end may hold anything: their scale counts as 0
            vs[j] = tc < valid ? vt[codes + t * (D / 16) + (D == 128 ? g : g >> 1)] : 0u;
        }

        float sc[NTW][4];
#pragma unroll
        for (int n = 0; n < NTW; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            uint32_t h0[4], h1[4];
            e2m1x8_to_f16(kw[0][w], h0);
            e2m1x8_to_f16(kw[1][w], h1);
            const uint32_t b0 = (ks[0] >> (8 * (w / 2))) & 0xffu, b1 = (ks[1] >> (8 * (w / 2))) & 0xffu;
            const uint32_t s0 = e4m3x2_to_f16(b0 * 0x101u), s1 = e4m3x2_to_f16(b1 * 0x101u);
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
        // logits in base 2, masked; the reference maximum; weights
        bool move = false;
#pragma unroll
        for (int n = 0; n < NTW; ++n) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float z = sc[n][j] * fac[n][j & 1];
                sc[n][j] = pos0 + g + 8 * (j >> 1) <= lim[n][j & 1] ? z : NEG_INF;
                move |= sc[n][j] > m[n][j & 1] + kHead4;
            }
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int n = 0; n < NTW; ++n) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float x = fmaxf(sc[n][j], sc[n][j + 2]);
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
                    x = fmaxf(x, m[n][j]);
                    const float corr = x == NEG_INF ? 1.f : fast_exp2(m[n][j] - x);
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
                const float ref = m[n][j & 1] == NEG_INF ? 0.f : m[n][j & 1] - kBias4;
                p[j] = fast_exp2(sc[n][j] - ref);
                l[n][j & 1] += p[j];
            }
            pf[n][0] = movmatrix_t(pack_f16(p[0], p[1]));
            pf[n][1] = movmatrix_t(pack_f16(p[2], p[3]));
        }
        const uint32_t s01 = e4m3x2_to_f16(vs[0] | vs[1] << 8), s23 = e4m3x2_to_f16(vs[2] | vs[3] << 8);
#pragma unroll
        for (int w = 0; w < VW; ++w) {
            // byte i of the words below: channel 2i (first two words) or 2i + 1 of a token
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
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NTW; ++n) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col = (ng * NTW + n) * 8 + 2 * c + j;
            float top = NEG_INF;
#pragma unroll
            for (int i = 0; i < TW; ++i) top = fmaxf(top, s_m[i * COLS + col]);
            const float f = m[n][j] == NEG_INF ? 0.f : fast_exp2(m[n][j] - top);
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

template <int D, int NT>
void pick(bool sparse, Attn4Fn* fn, int* smem, int* threads) {
    *fn = sparse ? attn4_kernel<D, NT, true> : attn4_kernel<D, NT, false>;
    *smem = Attn4Cfg<D, NT>::SMEM;
    *threads = Attn4Cfg<D, NT>::THREADS;
}

// The kernel for R query rows of a KV head, its dynamic shared memory and block.
void attn4_variant(int D, int R, bool sparse, Attn4Fn* fn, int* smem, int* threads) {
    if (D == 128) {
        if (R <= 8) pick<128, 1>(sparse, fn, smem, threads);
        else if (R <= 16) pick<128, 2>(sparse, fn, smem, threads);
        else if (R <= 32) pick<128, 4>(sparse, fn, smem, threads);
        else pick<128, 8>(sparse, fn, smem, threads);
    } else {
        if (R <= 8) pick<64, 1>(sparse, fn, smem, threads);
        else if (R <= 16) pick<64, 2>(sparse, fn, smem, threads);
        else if (R <= 32) pick<64, 4>(sparse, fn, smem, threads);
        else pick<64, 8>(sparse, fn, smem, threads);
    }
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
