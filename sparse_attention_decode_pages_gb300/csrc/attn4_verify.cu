// attn4_verify.cu -- dense causal attention over the 4-bit paged cache for 9 to 64 query
// rows of a KV head (the T drafted positions times the grouped heads).
//
// A unit is a run of at most pages_per_split pages of one (sequence, KV head) row; it
// holds all R = T * G query rows of the KV head.  A CTA of eight warps takes one unit, 128
// tokens (a step: eight 16-token chunks) at a time from a ring that bulk copies fill, and
// computes on the 5th-generation tensor cores (tcgen05, fp16 in, fp32 out)
//
//   S^T = K Q^T        M = 128 tokens, N = query rows (16, 32 or 64), K = channels
//   O^T += V^T P^T     M = 128 channels, N = query rows, K = 128 tokens
//
// with S^T and O^T in tensor memory.  code * scale is exact in fp16, so the products
// are those of the values the cache stands for.  What the threads do is convert:
//   K: warp w converts chunk w in the layout of an mma fragment (lane (g, c) =
//      (lane / 4, lane % 4): tokens g and g + 8, channels c * D / 4 ... -- 16 contiguous
//      bytes a token, free of bank conflicts) and stores them to tensor memory, as the A
//      operand of the first product.  The contraction's order of channels that this gives
//      (position 16 i + 4 c + j is channel c * D / 4 + 4 i + j) is given to Q as well.
//   V: rows of a token's channels to shared memory, as the M-major A operand of the second.
//   P: a warp weighs the 16 tokens of its chunk for every query row, S loaded and the weights,
//      in fp16, stored (8 x 8 matrices, the N-major B operand) as an mma fragment lies.
// A ninth warp issues the copies and, one elected lane, the products, which run while the
// others convert.  mma.sync blocks its SM quarter's issue for 8 cycles each: the same work
// took 502 us with it where this takes 334.
//
// In a step k a converting warp stores K of step k + 1, weighs step k (whose S was begun a step
// ago), says whether a weight is too large for the references (below), waits for O of step
// k - 1, stores P and V of step k, and only then waits for what the others said: no barrier of
// the CTA, and every wait has other work before it.  (Up to 32 query rows: for more, two
// places for K and S exceed tensor memory, so K of step k is stored in step k.)
//
// Queries are scaled by a power of two into fp16's range (the factor goes into the
// logits' scale).  Online softmax in fp32 in base 2; a query row's reference moves only when a
// logit exceeds it by kHead4 (attn4.cuh), for all warps at once.
//
// 64 sequences of 8K-16K tokens, 7 positions, 32 / 8 heads of 128: 334 us, 2.7 TB/s of keys and
// values, 40 % of the measured copy peak.  What it was before, step by step: a barrier for the
// vote and K of its own step 393; K ahead 380; the vote waited for later, and shared memory
// addressed as such, 359; waits that poll, multiply-adds in pairs 347; weights by fragments, their
// factors in registers 337; three splits of a row instead of two 334.  Bound by the latency of a
// step's instructions, 1.3 us for 128 tokens with one CTA on an SM, 1.5 with two (issue slots
// 52 % busy, and a quarter of the instructions hold their pipe for two cycles; shared memory
// 42 %), of which registers allow no third CTA; and by a unit's start and end, 8 to 11 us.
#include <atomic>

#include "attn4.cuh"
#include "tcgen05.cuh"

namespace spd {

namespace {

// CTAs on an SM (registers; shared memory and tensor memory hold them).  The runtime's
// occupancy query answers 1 for any kernel that allocates tensor memory.
constexpr int kVerify4Occ = 2;

template <int D, int N>
struct Verify4Cfg {
    static constexpr int WARPS = 8, THREADS = 32 * (WARPS + 1);  // converting warps, and the issuing one
    static constexpr int NH = N / 2;                      // query rows of a thread
    static constexpr int CHUNKS = 8;                      // of a step
    static constexpr int CHUNK = kv4_tile_bytes(16, D);   // bytes of 16 tokens' keys and values
    static constexpr int STEP = CHUNKS * CHUNK;
    static constexpr int STAGES = N == 64 ? 2 : 3;        // steps in the ring
    // Whether a step's keys are converted, and multiplied, before the softmax of the step before:
    // a second place for K and S in tensor memory, and a third step in the ring
    static constexpr bool AHEAD = N < 64;
    static constexpr int NB = AHEAD ? 2 : 1;              // places of K and S
    // V^T: 64-channel blocks of 128 rows (tokens) of 128 bytes, 128-byte swizzle
    static constexpr int VBLOCK = 128 * 128;
    static constexpr int OFF_V = 0;
    // Q: 64-position blocks of N rows of 128 bytes, 128-byte swizzle
    static constexpr int OFF_Q = OFF_V + D / 64 * VBLOCK;
    // P: 128 rows (tokens) of N fp16, swizzled over the row's 32, 64 or 128 bytes
    static constexpr int OFF_P = OFF_Q + N * D * 2;
    static constexpr int OFF_RING = OFF_P + 128 * N * 2;
    static constexpr int OFF_FR = OFF_RING + STAGES * STEP;  // float [N]: logit scales, then [N]: -references
    static constexpr int OFF_RED = OFF_FR + N * 8;           // float [WARPS][N]: maxima, then sums
    static constexpr int OFF_CORR = OFF_RED + WARPS * N * 4;  // float [N]
    static constexpr int OFF_OUT = OFF_CORR + N * 4;          // long long [N]: output rows
    static constexpr int OFF_LIM = OFF_OUT + N * 8;           // int [N]: the last position that a row sees
    static constexpr int OFF_BAR = OFF_LIM + N * 4;           // uint64 [STAGES] and eight more
    static constexpr int OFF_META = OFF_BAR + (STAGES + 8) * 8;  // int [STAGES][CHUNKS]: first positions or -1
    static constexpr int BODY = OFF_META + STAGES * CHUNKS * 4;
    // tensor memory: K, S, O
    static constexpr int COL_S = NB * D / 2, COL_O = COL_S + NB * N;
    static constexpr int COLUMNS = COL_O + N <= 128 ? 128 : 256;
    // at most 512 / COLUMNS CTAs fit on an SM (227 KB), so that none waits for columns
    static constexpr int LEAST = 227 * 1024 / (512 / COLUMNS + 1);
    static constexpr int SMEM = 1024 + (BODY > LEAST ? BODY : LEAST);
    static_assert(OFF_LIM % 8 == 0 && OFF_BAR % 8 == 0, "aligned");
    static constexpr int P_ROW = N * 2;
    static constexpr uint64_t P_SWIZZLE = N == 16 ? kSwizzle32 : N == 32 ? kSwizzle64 : kSwizzle128;
    static_assert(kVerify4Occ * (SMEM + 2048) <= 228 * 1024 && kVerify4Occ * COLUMNS <= 512, "they fit on an SM");
    static_assert(STAGES <= 4, "the first steps are resolved at once");
};

// Tensor-memory lane of S (and row of V and P) of token i of chunk q: a warp reaches the 32
// lanes of its number modulo 4, so warp q's chunk lies in those.
__device__ __forceinline__ int token_row(int q, int i) { return 32 * (q & 3) + 16 * (q >> 2) + i; }

__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

template <int N>
__device__ __forceinline__ void load_columns(uint32_t taddr, uint32_t (&v)[N]) {
    __syncwarp();
    tmem_ld(taddr, v);
    tmem_wait_ld();
}

template <int N>
__device__ __forceinline__ void load_frag(uint32_t taddr, uint32_t (&v)[N]) {
    __syncwarp();
    tmem_ld_frag(taddr, v);
    tmem_wait_ld();
}

// Four 8 x 8 matrices of 16-bit elements, as mma accumulators lie in a warp; lane i gives the
// address of row i % 8 of matrix i / 8.
__device__ __forceinline__ void store_matrices(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w)
                 : "memory");
}

__device__ __forceinline__ void store_columns(uint32_t taddr, const uint32_t (&v)[8]) {
    __syncwarp();
    tmem_st(taddr, v);
    tmem_wait_st();
}

// A place in a ring of S slots: the slot and the parity of its current round.
template <int S>
struct RingPos {
    int slot = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void advance() {
        if (++slot == S) {
            slot = 0;
            parity ^= 1u;
        }
    }
};

// A barrier of the T converting threads.
template <int T>
__device__ __forceinline__ void converters_sync() {
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(T) : "memory");
}

template <int D, int N>
__global__ void __launch_bounds__(Verify4Cfg<D, N>::THREADS, kVerify4Occ) verify4_kernel(const Attn4Args a) {
    using C = Verify4Cfg<D, N>;
    constexpr int STAGES = C::STAGES, WARPS = C::WARPS, CHUNKS = C::CHUNKS, NH = C::NH;
    constexpr int CODES = kv4_codes_bytes(16, D), HALF = kv4_half_bytes(16, D);  // of a chunk
    extern __shared__ uint8_t smem_raw[];
    __shared__ int s_last, s_move[2];  // s_move: a weight is too large, in an even or an odd step
    __shared__ uint32_t s_tmem;
    // (an offset to the array, not a rounded address: its accesses stay shared-memory ones)
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    float* s_fac = reinterpret_cast<float*>(smem + C::OFF_FR);
    float* s_neg = s_fac + N;
    float* s_red = reinterpret_cast<float*>(smem + C::OFF_RED);
    float* s_corr = reinterpret_cast<float*>(smem + C::OFF_CORR);
    long long* s_out = reinterpret_cast<long long*>(smem + C::OFF_OUT);
    int* s_lim = reinterpret_cast<int*>(smem + C::OFF_LIM);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* k_ready = full + STAGES;  // [2] K of a step is in tensor memory (of even and of odd steps)
    uint64_t* p_ready = k_ready + 2;    // V and P are in shared memory, and the step's codes are read
    uint64_t* voted = p_ready + 1;      // every warp has said whether its weights are too large
    uint64_t* level = voted + 1;        // and is as far as the others, where references move
    uint64_t* s_done = level + 1;       // [2] S is there
    uint64_t* o_done = s_done + 2;      // O is there; V and P may be overwritten
    int* meta = reinterpret_cast<int*>(smem + C::OFF_META);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int g = lane >> 2, c = lane & 3;
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
        for (int i = 0; i < STAGES + 8; ++i) mbar_init(full + i, i >= STAGES && i < STAGES + 5 ? WARPS : 1);
        mbar_fence_init();
        s_move[0] = s_move[1] = 0;
    }
    pdl_wait();
    pdl_trigger();

    // this warp's query rows, read together with the length
    constexpr int RW = (N + WARPS) / (WARPS + 1);
    uint32_t qx[RW][D / 64];
#pragma unroll
    for (int j = 0; j < RW; ++j) {
        const int r = warp + (WARPS + 1) * j;
        const long long at = out_index(r < R ? r : 0) * D + 2 * lane;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) qx[j][i] = r < R ? *reinterpret_cast<const uint32_t*>(a.q + at + 64 * i) : 0u;
    }
    const int start = split * a.pages_per_split;
    const int cpp = a.ps >> 4;  // chunks per page
    // the issuing warp's lane i resolves chunk 32 j + i of the unit, for four steps at a time
    int lp_next = -1, ph_next = -1;  // the next four steps' logical pages and page-table entries, unchecked
    const int len = a.seq_lens[b];
    int P = seq_pages(len, a.ps, a.max_pages);
    if (P < 0) {
        if (tid == 0) raise_status(a.status, SPD_DEV_BAD_LEN);
        P = 0;
    }
    const int n_items = P;
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
    const int steps = (chunks + CHUNKS - 1) / CHUNKS;

    auto next_pages = [&](int j) {
        const int ci = 32 * j + lane;
        lp_next = -1;
        if (ci < chunks) lp_next = start + ci / cpp;
    };
    auto next_entries = [&]() {
        ph_next = lp_next >= 0 ? a.page_table[(long long)b * a.max_pages + lp_next] : -1;
    };
    int ph_cur = -1, pos_cur = -1;  // physical page and first position (-1: nothing to read)
    auto take_next = [&](int j) {
        const int ci = 32 * j + lane;
        ph_cur = pos_cur = -1;
        if (ci < chunks) {
            if (ph_next < 0 || ph_next >= a.num_phys) {
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
    // issues step k's copies: lane 4 q + i copies piece i of chunk q (keys' codes and
    // scales, values' codes and scales), or lane 4 q the whole chunk where a page is one
    const int codes = kv4_codes_bytes(a.ps, D), half = kv4_half_bytes(a.ps, D);
    auto issue = [&](int k) {
        const int slot = k % STAGES, from = (k & 3) * 8;
        const int phys = __shfl_sync(0xffffffffu, ph_cur, from + (lane >> 2));
        const int pos = __shfl_sync(0xffffffffu, pos_cur, from + (lane >> 2));
        const unsigned there = __ballot_sync(0xffffffffu, pos >= 0 && (lane & 3) == 0);
        if ((lane & 3) == 0) meta[slot * CHUNKS + (lane >> 2)] = pos;
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full + slot, __popc(there) * C::CHUNK);
        __syncwarp();
        if (pos >= 0) {
            const int i = lane & 3;
            const uint8_t* tile = a.kv4 + ((long long)phys * a.H_kv + h) * (2LL * half);
            uint8_t* dst = smem + C::OFF_RING + slot * C::STEP + (lane >> 2) * C::CHUNK;
            if (a.ps == 16) {
                if (i == 0) bulk_load(dst, tile, C::CHUNK, full + slot);
            } else {
                const int t0 = pos & (a.ps - 1);
                const uint8_t* src = tile + (i >> 1) * half + (i & 1 ? codes + t0 * (D / 16) : t0 * (D / 2));
                bulk_load(dst + (i >> 1) * HALF + (i & 1) * CODES, src, i & 1 ? HALF - CODES : CODES, full + slot);
            }
        }
    };
    __syncthreads();  // the barriers are initialised
    if (warp == WARPS) {
        next_pages(0);
        next_entries();
        take_next(0);
        for (int k = 0; k < min(STAGES, steps); ++k) issue(k);
        if (steps > 4) next_pages(1);
        tmem_alloc(&s_tmem, C::COLUMNS);
    }

    // the query rows in fp16, each scaled by 2^-e so that its largest channel lies in [1, 2);
    // channel qc * D / 4 + 4 i + j at position 16 i + 4 qc + j
#pragma unroll
    for (int j = 0; j < RW; ++j) {
        const int r = warp + (WARPS + 1) * j;
        if (r >= N) break;
        float2 x[D / 64];
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            x[i] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qx[j][i]));
            amax = fmaxf(amax, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
        }
        const int e = query_exponent(amax);
        const float down = pow2f(-e);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            const int ch = 2 * lane + 64 * i, qc = ch / (D / 4), in = ch % (D / 4);
            const int at = 16 * (in >> 2) + 4 * qc + (in & 3);
            uint8_t* block = smem + C::OFF_Q + (at >> 6) * (N * 128);
            *reinterpret_cast<uint32_t*>(block + r * 128 + (((at & 63) * 2) ^ ((r & 7) << 4))) = pack_f16(x[i].x * down, x[i].y * down);
        }
        if (lane == 0) {
            s_fac[r] = a.scale_log2 * pow2f(e);
            s_neg[r] = -kLow4;
        }
    }
    if (tid < N) {
        s_out[tid] = tid < R ? out_index(tid) : 0;
        s_lim[tid] = tid < R ? len - a.T + tid / G : len - 1;
    }
    async_proxy_fence();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = s_tmem, tm_s = tmem + C::COL_S, tm_o = tmem + C::COL_O;
    const uint32_t my_lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int r0 = (warp >> 2) * NH;                 // this thread's query rows: r0 ... r0 + NH - 1
    const int my_row = (warp & 3) * 32 + lane;       // and its token's row
    const uint32_t v_smem = smem_u32(smem + C::OFF_V), q_smem = smem_u32(smem + C::OFF_Q), p_smem = smem_u32(smem + C::OFF_P);
    constexpr uint32_t kIdescS = umma_idesc_f16(128, N, false, false);
    constexpr uint32_t kIdescO = umma_idesc_f16(128, N, true, true);

    if (warp == WARPS) {
        // ============================================================ copies and products
        int issued = min(STAGES, steps), s_issued = 0, o_issued = 0;  // steps copied, and multiplied
        auto multiply_keys = [&](int k) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(k_ready + (k & 1), (uint32_t)k >> 1 & 1u, a.status, a.wait_ns))) return false;
            tmem_fence_after();
            s_issued = k + 1;
            if (elect_one()) {
                const int place = k & (C::NB - 1);
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
                    umma_f16_ts(tm_s + place * N, tmem + place * (D / 2) + 8 * i,
                                umma_desc(q_smem + (i >> 2) * (N * 128) + (i & 3) * 32, 0, 1024, kSwizzle128), kIdescS, i > 0);
                umma_commit(s_done + (k & 1));
            }
            __syncwarp();
            return true;
        };
        for (int k = C::AHEAD ? -1 : 0; k < steps; ++k) {
            const int ahead = k + (C::AHEAD ? 1 : 0);
            if (ahead < steps && !multiply_keys(ahead)) break;
            if (k < 0) continue;
            const int kn = k + STAGES;  // the next step into this one's slot
            if (kn < steps && (kn & 3) == 0) {
                next_entries();
                take_next(kn >> 2);
                next_pages((kn >> 2) + 1);
            }
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(p_ready, (uint32_t)k & 1u, a.status, a.wait_ns))) break;
            tmem_fence_after();
            o_issued = k + 1;
            if (elect_one()) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    umma_f16_ss(tm_o, umma_desc(v_smem + i * 2048, D == 128 ? C::VBLOCK : 0, 1024, kSwizzle128),
                                umma_desc(p_smem + i * 16 * C::P_ROW, 0, 8 * C::P_ROW, C::P_SWIZZLE), kIdescO, k > 0 || i > 0);
                umma_commit(o_done);
            }
            __syncwarp();
            if (kn < steps) {
                issue(kn);
                issued = kn + 1;
            }
        }
        // the copies in flight land, and the products end, before their memory is given back
        for (int j = max(0, issued - STAGES); j < issued; ++j)
            mbar_wait_bounded(full + j % STAGES, (uint32_t)(j / STAGES) & 1u, a.status, drain_limit(a));
        if (s_issued > 0) mbar_wait_bounded(s_done + (s_issued - 1 & 1), (uint32_t)(s_issued - 1) >> 1 & 1u, a.status, drain_limit(a));
        if (o_issued > 0) mbar_wait_bounded(o_done, (uint32_t)(o_issued - 1) & 1u, a.status, drain_limit(a));
    } else {
    // ================================================================ conversions and softmax
    // V of this warp's chunk: this lane's token (and the one 8 behind) and 32 channels; the eight
    // lanes that store together cover every bank
    const int piece = D == 128 ? (lane >> 2 & 1) + 2 * ((lane >> 3 ^ lane >> 1) & 1) : lane >> 2 & 1;
    const int v_token = D == 128 ? (lane & 3) + 4 * (lane >> 4) : (lane & 3) + 4 * (lane >> 3);
    const int v_src = warp * C::CHUNK + HALF + v_token * (D / 2) + piece * 16;
    const int v_scale_src = warp * C::CHUNK + HALF + CODES + v_token * (D / 16) + piece * 2;
    const uint32_t v_dst = v_smem + (piece >> 1) * C::VBLOCK + token_row(warp, v_token) * 128 +
                           ((((piece & 1) * 4) ^ (v_token & 7)) << 4);
    // P: matrices of 8 tokens by 8 query rows, four a store, a row of one a lane: tokens 0 to 7 and
    // 8 to 15 of the warp's chunk, two 16-byte pieces, in the rows' swizzled order
    const int p_row = token_row(warp, lane & 15);
    const int p_xor = N == 16 ? p_row >> 2 & 1 : N == 32 ? p_row >> 1 & 3 : p_row & 7;
    const uint32_t p_dst = p_smem + p_row * C::P_ROW + (((lane >> 4) ^ p_xor) << 4);

    // this thread has tokens g and g + 8 of the warp's chunk and query rows 8 j + 2 c, 8 j + 2 c + 1
    float2 l[N / 8];  // sums of the rows' weights
#pragma unroll
    for (int j = 0; j < N / 8; ++j) l[j] = make_float2(0.f, 0.f);
    float2 fac[N / 8], neg[N / 8];
    int done = 0;       // steps whose second product was issued
    RingPos<STAGES> ring;  // of the next step whose keys are converted

    // K of step k: this warp's chunk to tensor memory (one that is not there: whatever the ring
    // holds; its tokens are hidden)
    auto convert_keys = [&](int k) {
        const bool there = mbar_wait_bounded(full + ring.slot, ring.parity, a.status, a.wait_ns);
        {
            const uint8_t* kt = smem + C::OFF_RING + ring.slot * C::STEP + warp * C::CHUNK;
            ring.advance();
            uint32_t f[D / 4];  // [column group][row g: two columns, row g + 8: two]
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = g + 8 * j;
                uint32_t w[D / 32], s;
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4*>(kt + t * 64 + c * 16);
                    w[0] = x.x;
                    w[1] = x.y;
                    w[D / 32 - 2] = x.z;
                    w[D / 32 - 1] = x.w;
                    s = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(kt + CODES + t * 8 + 2 * c));
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(kt + t * 32 + c * 8);
                    w[0] = x.x;
                    w[1] = x.y;
                    s = e4m3x2_to_f16(kt[CODES + t * 4 + c]);
                }
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    uint32_t v[4];
                    e2m1x8_to_f16(w[x], v);
                    const uint32_t s2 = __byte_perm(s, 0, x < 2 ? 0x1010 : 0x3232);
                    f[8 * x + 2 * j] = hmul2(v[0], s2);
                    f[8 * x + 2 * j + 1] = hmul2(v[1], s2);
                    f[8 * x + 4 + 2 * j] = hmul2(v[2], s2);
                    f[8 * x + 4 + 2 * j + 1] = hmul2(v[3], s2);
                }
            }
            __syncwarp();
            tmem_st_frag(tmem + ((uint32_t)token_row(warp, 0) << 16) + (k & (C::NB - 1)) * (D / 2), f);
        }
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_ready + (k & 1));
        return there;
    };
    // A barrier of the converting warps that no warp can be held at: false where the wait ran out.
    uint32_t level_parity = 0;
    auto all_level = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(level);
        const bool there = __all_sync(0xffffffffu, mbar_wait_bounded(level, level_parity, a.status, a.wait_ns));
        level_parity ^= 1u;
        return there;
    };
    bool ok = true;
    int slot = 0;  // of step k

    for (int k = C::AHEAD ? -1 : 0; k < steps; ++k) {
        const uint8_t* stage = smem + C::OFF_RING + slot * C::STEP;
        const int ahead = k + (C::AHEAD ? 1 : 0);
        if (ahead < steps) ok &= convert_keys(ahead);
        if (k < 0) continue;

        // softmax of this thread's token, for its query rows
        ok &= mbar_wait_bounded(s_done + (k & 1), (uint32_t)k >> 1 & 1u, a.status, a.wait_ns);
        tmem_fence_after();
        const uint32_t my_s = tm_s + (k & (C::NB - 1)) * N + ((uint32_t)token_row(warp, 0) << 16);
        const int first = meta[slot * CHUNKS + warp];
        const int pos = first < 0 ? 0x7ffffff0 : first + g;  // of this thread's first token
        const bool all = first >= 0 && first + 15 <= len - a.T;  // every row sees every token of the warp
        float2 p[N / 8][2];
        // (what runs once a unit is kept short: a unit's first pass through straight code is bound by
        // fetching it)
#pragma unroll 1
        for (bool moved = false;; moved = true) {
            {
                uint32_t s[N / 2];
                load_frag(my_s, s);
#pragma unroll
                for (int j = 0; j < N / 8; ++j) {
                    if (N == 64 || moved || k == 0) {
                        fac[j] = *reinterpret_cast<const float2*>(s_fac + 8 * j + 2 * c);
                        neg[j] = *reinterpret_cast<const float2*>(s_neg + 8 * j + 2 * c);
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const float2 y = fma2(make_float2(__uint_as_float(s[4 * j + 2 * t]), __uint_as_float(s[4 * j + 2 * t + 1])), fac[j], neg[j]);
                        p[j][t] = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                    }
                }
            }
            if (!all) {
#pragma unroll
                for (int j = 0; j < N / 8; ++j) {
                    const int2 lim = *reinterpret_cast<const int2*>(s_lim + 8 * j + 2 * c);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (pos + 8 * t > lim.x) p[j][t].x = 0.f;
                        if (pos + 8 * t > lim.y) p[j][t].y = 0.f;
                    }
                }
            }
            if (!moved) {
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < N / 8; ++j)
                    top = fmaxf(fmaxf(top, fmaxf(p[j][0].x, p[j][0].y)), fmaxf(p[j][1].x, p[j][1].y));
                const bool large = __any_sync(0xffffffffu, top > kMost4);  // some weight is too large
                if (lane == 0) {
                    if (large) s_move[k & 1] = 1;
                    mbar_arrive(voted);
                }
                if (k > 0) ok &= mbar_wait_bounded(o_done, (uint32_t)(k - 1) & 1u, a.status, a.wait_ns);
                __syncwarp();
            }
#pragma unroll
            for (int j = 0; j < N / 8; j += 2)
                store_matrices(p_dst ^ (j << 4), pack_f16(p[j][0].x, p[j][0].y), pack_f16(p[j][1].x, p[j][1].y),
                               pack_f16(p[j + 1][0].x, p[j + 1][0].y), pack_f16(p[j + 1][1].x, p[j + 1][1].y));
            if (moved) break;

            // V: this warp's chunk to shared memory, 32 channels of a token at a time
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const uint8_t* vt = stage + v_src + i * (8 * (D / 2));
                const uint4 x = *reinterpret_cast<const uint4*>(vt);
                uint32_t two = *reinterpret_cast<const uint16_t*>(stage + v_scale_src + i * (8 * (D / 16)));
                if (first < 0 || first + v_token + 8 * i >= len) two = 0u;  // no token: its bytes may be anything, its scale counts as 0
                const uint32_t s = e4m3x2_to_f16(two);
                const uint32_t s_lo = __byte_perm(s, 0, 0x1010), s_hi = __byte_perm(s, 0, 0x3232);
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t v[4];
                    e2m1x8_to_f16(w[j], v);
                    const uint32_t s2 = j < 2 ? s_lo : s_hi;
                    st_shared16((v_dst ^ (j << 4)) + i * 1024, hmul2(v[0], s2), hmul2(v[1], s2), hmul2(v[2], s2), hmul2(v[3], s2));
                }
            }
            ok &= mbar_wait_bounded(voted, (uint32_t)k & 1u, a.status, a.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok || !*reinterpret_cast<volatile int*>(s_move + (k & 1))) break;
            // the references move to the largest logit of each row among this step's tokens
            {
                uint32_t s[N / 2];
                load_frag(my_s, s);
#pragma unroll
                for (int j = 0; j < N / 8; ++j) {
                    const float2 f = *reinterpret_cast<const float2*>(s_fac + 8 * j + 2 * c);
                    const int2 lim = *reinterpret_cast<const int2*>(s_lim + 8 * j + 2 * c);
                    float2 m = make_float2(NEG_INF, NEG_INF);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (pos + 8 * t <= lim.x) m.x = fmaxf(m.x, __uint_as_float(s[4 * j + 2 * t]) * f.x);
                        if (pos + 8 * t <= lim.y) m.y = fmaxf(m.y, __uint_as_float(s[4 * j + 2 * t + 1]) * f.y);
                    }
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) {
                        m.x = fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, off));
                        m.y = fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, off));
                    }
                    if (g == 0) *reinterpret_cast<float2*>(s_red + warp * N + 8 * j + 2 * c) = m;
                }
            }
            ok = all_level();
            if (!ok) break;
            if (tid < N) {
                float x = NEG_INF;
#pragma unroll
                for (int i = 0; i < WARPS; ++i) x = fmaxf(x, s_red[i * N + tid]);
                const float old = -s_neg[tid], now = fmaxf(old, x - kBias4);
                s_corr[tid] = fast_exp2(old - now);
                s_neg[tid] = -now;
            }
            if (tid == 0) s_move[k & 1] = 0;  // every warp has read it
            ok = all_level();
            if (!ok) break;
            if (k > 0) {
                tmem_fence_after();  // O of step k - 1, whose end this thread has waited for above
#pragma unroll 1
                for (int r = 0; r < NH; r += 8) {
                    uint32_t o[8];
                    load_columns<8>(tm_o + r0 + r + my_lanes, o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * s_corr[r0 + r + i]);
                    store_columns(tm_o + r0 + r + my_lanes, o);
                }
            }
#pragma unroll
            for (int j = 0; j < N / 8; ++j) {
                const float2 corr = *reinterpret_cast<const float2*>(s_corr + 8 * j + 2 * c);
                l[j].x *= corr.x;
                l[j].y *= corr.y;
            }
        }
        if (!ok) break;  // a wait ran out: the others' waits for this warp will, too
        async_proxy_fence();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready);
        done = k + 1;
        slot = slot + 1 == STAGES ? 0 : slot + 1;
#pragma unroll
        for (int j = 0; j < N / 8; ++j) l[j] = add2(l[j], add2(p[j][0], p[j][1]));
    }

    if (done > 0) mbar_wait_bounded(o_done, (uint32_t)(done - 1) & 1u, a.status, a.wait_ns);
    tmem_fence_after();
    uint32_t o[NH];
    load_columns<NH>(tm_o + r0 + my_lanes, o);  // channel my_row of this thread's query rows
    tmem_fence_before();
    // the sums of the rows, over the eight lanes of a warp and the warps that hold parts of each
#pragma unroll
    for (int j = 0; j < N / 8; ++j) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l[j].x += __shfl_xor_sync(0xffffffffu, l[j].x, off);
            l[j].y += __shfl_xor_sync(0xffffffffu, l[j].y, off);
        }
        if (g == 0) *reinterpret_cast<float2*>(s_red + warp * N + 8 * j + 2 * c) = l[j];
    }
    converters_sync<32 * WARPS>();
    if (tid < N) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) sum += s_red[i * N + tid];
        s_corr[tid] = sum == 0.f ? 0.f : a.v_scale / sum;
        const float lse = sum == 0.f ? NEG_INF : (log2f(sum) - s_neg[tid]) * kLn2;
        const long long at = ((long long)row * a.parts + split) * R + tid;
        if (tid < R && nsplit > 1) a.part_lse[at] = lse;
        if (tid < R && nsplit == 1 && a.lse) a.lse[s_out[tid]] = lse;
    }
    converters_sync<32 * WARPS>();
    if (my_row < D) {
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            const int r = r0 + i;
            const float inv = s_corr[r], x = inv == 0.f ? 0.f : __uint_as_float(o[i]) * inv;
            if (r < R) {
                if (nsplit == 1)
                    reinterpret_cast<bf16*>(a.o)[s_out[r] * D + my_row] = __float2bfloat16_rn(x);
                else
                    a.part_o[(((long long)row * a.parts + split) * R + r) * D + my_row] = x;
            }
        }
    }
    }
    __syncthreads();
    tmem_fence_after();
    if (warp == WARPS) tmem_free(tmem, C::COLUMNS);
    join_splits<D, C::THREADS, true>(a, row, split, nsplit, R, &s_last, out_index);
}

typedef void (*Verify4Fn)(const Attn4Args);

template <int D>
void pick(int R, Verify4Fn* fn, int* smem) {
    *fn = R <= 16 ? verify4_kernel<D, 16> : R <= 32 ? verify4_kernel<D, 32> : verify4_kernel<D, 64>;
    *smem = R <= 16 ? Verify4Cfg<D, 16>::SMEM : R <= 32 ? Verify4Cfg<D, 32>::SMEM : Verify4Cfg<D, 64>::SMEM;
}

}  // namespace

int occ_attn4_verify() { return kVerify4Occ; }

cudaError_t launch_attn4_verify(const Attn4Args& a, cudaStream_t st) {
    // the kernel's attributes for its shared memory, set once for a device and a variant
    constexpr int kDevices = 64, kVariants = 6;
    static std::atomic<bool> known[kDevices][kVariants];
    const int R = a.T * (a.H_q / a.H_kv);
    Verify4Fn fn;
    int smem, dev = 0;
    if (a.D == 128) pick<128>(R, &fn, &smem);
    else pick<64>(R, &fn, &smem);
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int v = (a.D == 128 ? 3 : 0) + (R <= 16 ? 0 : R <= 32 ? 1 : 2);
    if (dev >= kDevices || !known[dev][v].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
        if (e != cudaSuccess) return e;
        if (dev < kDevices) known[dev][v].store(true, std::memory_order_release);
    }
    return launch_pdl(fn, dim3((unsigned)((long long)a.B * a.H_kv * a.num_splits)), dim3(Verify4Cfg<128, 16>::THREADS), smem, st, a);
}

}  // namespace spd
