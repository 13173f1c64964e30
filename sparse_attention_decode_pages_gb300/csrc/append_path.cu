// append_path.cu -- the keys and values of an accepted path, from the rows of a tree's nodes
// to the newest positions of the paged cache, with the summaries of the pages they
// land in.
//
// As the append of consecutive tokens: one CTA for a (sequence, touched page), one warp a KV head, every
// row of the page visited once.  Rows of the path are read from the nodes' rows and stored
// into the cache, older ones are read from it, and the channel-wise minima and maxima are formed on the
// way.  What is read from the cache and what is written are different rows.  Up to about 128 paths it is bound by latency (length, path,
// page table, rows, one behind the other): 2.7 us for one path in a run of calls, 3.5 for 64, 3.8 for 128; behind that by
// rounds of CTAs, of which a sequence has as many as its tree could touch pages: 5.9 for 256 paths out of 64 nodes, 5.4 out of 8.
#include "common.cuh"
#include "kernels.h"

namespace spd {
namespace {

template <int D>
__global__ void __launch_bounds__(256) append_path_kernel(AppendPathArgs p) {
    constexpr int LPR = D * 2 / 16;  // lanes of a row (16 bytes each)
    constexpr int RPI = 32 / LPR;    // rows of a warp's access
    const AppendArgs& a = p.append;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
    const int b = blockIdx.x, T = a.T;
    pdl_wait();
    pdl_trigger();
    const int len = a.seq_lens[b], count = p.n_path[b];
    const int at = lane < T ? p.path[(long long)b * T + lane] : -1;
    const int at2 = lane + 32 < T ? p.path[(long long)b * T + lane + 32] : -1;
    const bool bad_path = count < 0 || count > T ||
                          __any_sync(0xffffffffu, (lane < count && (at < 0 || at >= T)) || (lane + 32 < count && (at2 < 0 || at2 >= T)));
    const bool bad_len = len < 0 || (long long)len + count > min((long long)a.max_pages * a.ps, 0x7fffffffLL);
    if (blockIdx.y == 0 && threadIdx.x == 0) {
        if (bad_path) raise_status(a.status, SPD_DEV_BAD_TREE);
        else if (bad_len) raise_status(a.status, SPD_DEV_BAD_LEN);
        p.new_lens[b] = bad_path || bad_len ? len : len + count;
    }
    if (bad_path || bad_len || count == 0) return;
    const int end = len + count;
    const int page = len / a.ps + (int)blockIdx.y;
    const long long base = (long long)page * a.ps;  // position of the page's first slot
    if (base >= end) return;
    const int valid = (int)min((long long)a.ps, end - base);
    const int nold = (int)max(0LL, len - base);
    const long long phys = a.page_table[(long long)b * a.max_pages + page];
    if (phys < 0 || phys >= a.num_phys) {
        if (threadIdx.x == 0) raise_status(a.status, SPD_DEV_BAD_PAGE);
        return;
    }
    const int r0 = lane / LPR, ch = lane % LPR;
    const __nv_bfloat162 pinf = __floats2bfloat162_rn(__int_as_float(0x7f800000), __int_as_float(0x7f800000));
    const __nv_bfloat162 ninf = __floats2bfloat162_rn(__int_as_float(0xff800000), __int_as_float(0xff800000));
    for (int h = warp; h < a.H_kv; h += nwarps) {
        const long long row0 = (phys * a.H_kv + h) * a.ps;
        uint4* kt = reinterpret_cast<uint4*>(a.K + row0 * D);
        uint4* vt = reinterpret_cast<uint4*>(a.V + row0 * D);
        __nv_bfloat162 mn[4], mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mn[i] = pinf;
            mx[i] = ninf;
        }
        auto fold = [&](const uint4& k) {
            const __nv_bfloat162* e = reinterpret_cast<const __nv_bfloat162*>(&k);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mn[i] = __hmin2(mn[i], e[i]);
                mx[i] = __hmax2(mx[i], e[i]);
            }
        };
        // all rows of the page in batches, so that a page costs one or two round trips
        for (int t0 = 0; t0 < valid; t0 += kAppendBatch * RPI) {  // the same for the whole warp
            uint4 k[kAppendBatch], v[kAppendBatch];
#pragma unroll
            for (int u = 0; u < kAppendBatch; ++u) {
                const int t = t0 + u * RPI + r0;
                const int i = (int)(base + t - len);  // its place on the path
                const int src = i < 0 ? 0 : i;
                const int lo = __shfl_sync(0xffffffffu, at, src & 31), hi = __shfl_sync(0xffffffffu, at2, src & 31);
                const long long node = (long long)b * T + (src < 32 ? lo : hi);
                if (t < nold) {
                    k[u] = kt[t * LPR + ch];
                } else if (t < valid) {
                    k[u] = __ldg(reinterpret_cast<const uint4*>(a.k_new + node * p.k_stride + h * D) + ch);
                    v[u] = __ldg(reinterpret_cast<const uint4*>(a.v_new + node * p.v_stride + h * D) + ch);
                }
            }
#pragma unroll
            for (int u = 0; u < kAppendBatch; ++u) {
                const int t = t0 + u * RPI + r0;
                if (t >= valid) continue;
                if (t >= nold) {
                    kt[t * LPR + ch] = k[u];
                    vt[t * LPR + ch] = v[u];
                }
                fold(k[u]);
            }
        }
#pragma unroll
        for (int off = LPR; off < 32; off <<= 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t*>(&mn[i]), off);
                const uint32_t y = __shfl_xor_sync(0xffffffffu, *reinterpret_cast<uint32_t*>(&mx[i]), off);
                mn[i] = __hmin2(mn[i], *reinterpret_cast<const __nv_bfloat162*>(&x));
                mx[i] = __hmax2(mx[i], *reinterpret_cast<const __nv_bfloat162*>(&y));
            }
        }
        if (r0 == 0) {
            uint4* out = reinterpret_cast<uint4*>(a.summ + (((long long)b * a.H_kv + h) * a.max_pages + page) * 2LL * D);
            out[ch] = *reinterpret_cast<uint4*>(mn);
            out[LPR + ch] = *reinterpret_cast<uint4*>(mx);
        }
    }
}

}  // namespace

cudaError_t launch_append_path(const AppendPathArgs& p, cudaStream_t st) {
    if (p.append.B <= 0) return cudaSuccess;
    const int warps = p.append.H_kv < 8 ? p.append.H_kv : 8;
    const dim3 grid((unsigned)p.append.B, (unsigned)append_touched(p.append.T, p.append.ps, p.append.max_pages)), block(32 * warps);
    return launch_pdl(p.append.D == 128 ? append_path_kernel<128> : append_path_kernel<64>, grid, block, 0, st, p);
}

}  // namespace spd
