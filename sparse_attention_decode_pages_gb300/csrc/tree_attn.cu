// tree_attn.cu -- attention of the nodes of a tree of drafted tokens over the paged cache, their
// ancestors and themselves.
//
// The R = T * G query rows of a (sequence, KV head) see the same cached tokens, so they are the rows of two
// products on the 5th-generation tensor cores (tcgen05, bf16 in, fp32 out in tensor memory)
//
//   S = Q K^T      M = 128 rows, N = 128 tokens, K = channels;  Q and K in shared memory
//   O += P V       M = 128 rows, N = channels, K = 128 tokens;  P in tensor memory, in S's place
//
// over tiles of 128 tokens, the tree's own nodes as the last one.  A thread of a softmax
// warp has one row (a lane of tensor memory): its maximum, its sum and its weights need no other
// thread.  Two streams of 128 rows take turns, so that one's softmax runs under the other's
// products: more than 128 rows of a KV head are two row tiles over the same tokens, fewer are one row
// tile whose streams take the even and the odd tiles of tokens and are joined at the end, in tensor
// memory.
//
// The softmax goes by a reference that follows the row's maximum only when that has grown by 2^8 beyond it, so O
// is rarely rescaled; sums are fp32, a tile's by itself first, the weights that multiply V are rounded to bf16 (V's type,
// as the products want them), 2^-8 of a weight at most and of either sign.  O adds up in tensor memory for 65,536 tokens of a stream and
// then in an fp32 sum in the workspace, or what the tensor cores cut grows with the length (means of 2^20 tokens were up to 0.4 % low,
// of 2^24 6 %; now 0.01 %, at no cost: a pass over O in 512 tiles).
//
// One CTA an SM: two warpgroups for the softmax, and a warp each for the keys' copies, the values' copies, the products
// and the nodes' values.  A page's keys or values of a KV head are one TMA box.  A sequence that ends inside a page has that page
// copied eight slots at a time, by boxes that start above it: what lies before the page arrives as zeros, so its valid
// tokens come to lie at the end of its place in the tile and nothing past the sequence is ever read.
//
// The tiles of all (sequence, KV head, pair of row tiles) units in a row are cut into equal shares, one a CTA (the GPU knows
// the lengths, the host does not); a unit that a border cuts leaves unnormalised partials, at most two a CTA, for
// a second kernel to join.
//
// What bounds it (32 / 8 heads of 128 channels): memory up to 128 rows a KV head (64 sequences of 8K-16K tokens, 15 nodes:
// 467 to 476 us, the measured copy rate).  With 256 rows (64 nodes) the hand-overs between softmax and products: a pair of tiles takes
// 3,325 cycles, its products 2,048 of them, and their operands and copies keep shared memory busy for as many.  598 to 633 us in a
// run of ten calls, 634 to 683 in longer ones, where the power limit takes the SM clock to 1.46 to 1.6 GHz as well; at that clock a large
// library product does 1,718 TFLOP/s, this 1,243.  One sequence of 131,001 tokens, 61 nodes: 102 us, 108
// with cold inputs, 110 to 116 in long runs; of 1,003, 8 nodes: 11.5 us, 15 cold, the latency of the two kernels.  With heads of 64
// channels a tile's softmax is as long and its products half: 64 nodes 430 to 437 us (bytes: 239), 15 nodes 262, 131,001 tokens 84.
#include <atomic>

#include "common.cuh"
#include "kernels.h"
#include "tcgen05.cuh"
#include "tree.cuh"

namespace spd {
namespace {

constexpr int kRows = 128;          // of a row tile
constexpr int kTokens = 128;        // of a tile of tokens
constexpr int kThreads = 384;       // two softmax warpgroups and four warps
// Registers: 168 a thread at launch (64,512 of the SM's 65,536); of these the softmax warpgroups take 208 a
// thread, the third keeps 80: 2 * 128 * 208 + 128 * 80 = 63,488.
constexpr int kSoftmaxRegs = 208, kOtherRegs = 80;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "what the block was launched with");
constexpr int kInfos = 16;          // tiles whose visible tokens are written down
constexpr int kOdd = 8;             // pieces whose nodes with odd values are
// Units of which the SMs hold this many times as many are cut into parts of their own, so that no CTA has parts of two
// (3 sequences of 14,000 tokens, 61 nodes: 46 us against 51); more units than this leave parts of too different lengths, or CTAs
// without one (8 sequences of 8,000, 8 nodes: 55.6 us so, 51.2 in equal shares).
constexpr int kFewUnits = 4;
// What a unit costs a CTA beside its tiles (queries, first products, results), in tiles: so many are counted in front of its own
// where equal shares are cut, or a CTA with many short units would hold up the others (12 sequences of 0 to 16,000 tokens, 61 nodes:
// 119 -> 88 us; 64 of 0 to 2,000, 64 nodes: 121 -> 88; with five instead of three the same).
constexpr int kUnitTiles = 3;
constexpr float kLag = 8.f;         // powers of two that a maximum may lie above the reference
// Tiles of a stream whose products add up in tensor memory (a power of two).  The tensor cores cut what lies about 2^-25 below a sum,
// so O goes to an fp32 sum in the workspace every so many and starts again.
constexpr int kAside = 512;

template <int D>
struct Cfg {
    static constexpr int HALVES = D / 64;
    static constexpr int HALF = kTokens * 128;  // 64 channels of a tile
    static constexpr int TILE = HALVES * HALF;
    // A tile of tokens: atoms of 8 tokens by 64 channels (1,024 bytes, 128-byte swizzle), a page's of all channels together, so
    // that a page is one box: 8 tokens on and 64 channels on are these many bytes on.  Queries and the tree's nodes lie
    // by 64 channels: [half][row].
    static constexpr int GROUP = HALVES * 1024;
    static constexpr int STAGES = D == 128 ? 5 : 10;
    static constexpr int OFF_Q = 0;             // two row tiles
    static constexpr int OFF_RING = 2 * TILE;
    static constexpr int OFF_INFO = OFF_RING + STAGES * TILE;  // uint16 [kInfos][8]: visible tokens of a tile
    static constexpr int OFF_ML = OFF_INFO + kInfos * 16;      // float2 [128]: a stream's references and sums
    static constexpr int OFF_BAR = OFF_ML + kRows * 8;         // uint64: full, empty, v_tree [STAGES], and ten more
    static constexpr int SMEM = 1024 + OFF_BAR + (3 * STAGES + 10) * 8;
    static_assert(SMEM <= 227 * 1024 && SMEM > 114 * 1024, "one CTA an SM");
    // tensor memory: S (and P) and O of each stream
    static constexpr int COL_S = 0, COL_O = 256, COLUMNS = 512;
};

// What a CTA leaves for the joining kernel: a unit that begins in its share and ends in another's (one for a CTA, or, where units are
// few, for a unit).
struct Cut {
    int b, sub, pieces, cta;
};

// Partials: [slot][D / 4][256 rows] float4, then [slot][256 rows] (reference, sum); two slots a CTA, one for the unit
// that its share begins in and one for the unit that it ends in.  A reference that is NaN: the CTA gave up, and the unit's rows
// are left as they were.
constexpr int kSlotRows = 256;
__host__ __device__ constexpr size_t slot_bytes(int D) { return (size_t)kSlotRows * (D * 4 + 8); }
__device__ __forceinline__ float* part_o_of(void* ws, int ctas) {
    return reinterpret_cast<float*>(static_cast<char*>(ws) + ((size_t)ctas * sizeof(Cut) + 255) / 256 * 256);
}
__device__ __forceinline__ float2* part_ml_of(void* ws, int ctas, int D) {
    return reinterpret_cast<float2*>(part_o_of(ws, ctas) + (size_t)2 * ctas * kSlotRows * D);
}

// What follows from T, G and the page size, worked out once by the host (a division costs a CTA's start more than it looks).
struct Shape {
    int G, tpt, row_tiles, pairs;  // heads of a group, nodes of a row tile, row tiles (up to 4), units of a (sequence, KV head) (1 or 2)
    int lg_ps;                     // log2 of the page size
    __device__ __forceinline__ int pages(int len, int max_pages) const {  // as seq_pages
        if (len < 0 || (long long)len > (long long)max_pages << lg_ps) return -1;
        return (int)(((unsigned)len + (1u << lg_ps) - 1) >> lg_ps);
    }
    __device__ __forceinline__ int head(int sub) const { return sub >> (pairs - 1); }
    __device__ __forceinline__ int first_tile(int sub) const { return 2 * (sub & (pairs - 1)); }
};
inline Shape shape_of(int T, int G, int ps) {
    Shape s;
    s.G = G;
    s.tpt = kRows / G < T ? kRows / G : T;
    s.row_tiles = (T + s.tpt - 1) / s.tpt;
    s.pairs = (s.row_tiles + 1) / 2;
    s.lg_ps = ps == 16 ? 4 : ps == 32 ? 5 : 6;
    return s;
}

// The part of a unit that lies in a CTA's share: tiles t0 .. t1 - 1 of its nt.
struct Piece {
    int b, sub, len, nt, t0, t1;
    bool bad;  // a length that the page table has no room for: no tokens, no nodes
};

// Where a CTA's share begins, counted with kUnitTiles in front of each unit's, and what it is of: tile `at` of `total`, or (few
// units) the first of a unit's parts, which `follow` CTAs hold the rest of.
struct Share {
    int b, sub, t0, len;
    long long left, at, total;
    int follow;
};

// Goes through the pieces of a share, one sequence's units after the other's (t0 and left counted as the share).
struct Walk {
    int b, sub, t0, len, nt;
    bool bad;
    long long left;
    __device__ __forceinline__ void look(const TreeAttnArgs& a, const Shape& sh, int raw) {
        bad = sh.pages(raw, a.max_pages) < 0;
        len = bad ? 0 : raw;
        nt = (len + kTokens - 1) / kTokens + 1;
    }
    __device__ __forceinline__ bool next(const TreeAttnArgs& a, const Shape& sh, Piece& p) {
        while (left > 0) {
            p.b = b;
            p.sub = sub;
            p.len = len;
            p.nt = nt;
            p.bad = bad;
            const int end = (int)min((long long)nt + kUnitTiles, t0 + left);
            p.t0 = max(0, t0 - kUnitTiles);
            p.t1 = max(0, end - kUnitTiles);
            left -= end - t0;
            t0 = 0;
            if (++sub == a.H_kv * sh.pairs) {
                sub = 0;
                if (left > 0) look(a, sh, a.seq_lens[++b]);
            }
            if (p.t0 < p.t1) return true;
        }
        return false;
    }
};

__device__ __forceinline__ void other_regs() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs)); }

// Where share i of `total` tiles begins: the first total % ctas shares have a tile more.
struct Shares {
    long long each;
    int more;
    __device__ __forceinline__ Shares(long long total, int ctas) {
        if (total < 0x7fffffff) {
            each = (int)total / ctas;
            more = (int)total - (int)each * ctas;
        } else {
            each = total / ctas;
            more = (int)(total - each * ctas);
        }
    }
    __device__ __forceinline__ long long begin(int i) const { return each * i + min(i, more); }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const TreeAttnArgs a, const __grid_constant__ TreeMaps maps, const Shape sh, const bool few) {
    using C = Cfg<D>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long s_scan[kThreads / 32];
    __shared__ Share s_share;
    __shared__ uint32_t s_tmem;
    __shared__ unsigned long long s_odd[kOdd];  // nodes of a piece's tree whose values are not all finite
    __shared__ int s_asked;                     // tiles whose values have been asked for
    __shared__ int s_gave_up;                   // a softmax warp's wait has run out
    uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* empty = full + STAGES;
    uint64_t* v_tree = empty + STAGES;  // the nodes' values have come; then they are looked over
    uint64_t* q_full = v_tree + STAGES;
    uint64_t* q_empty = q_full + 1;
    uint64_t* s_full = q_empty + 1;  // [2] S is there, and the tile's visible tokens are written down
    uint64_t* p_full = s_full + 2;   // [2] P is there
    uint64_t* o_done = p_full + 2;   // [2] a piece's last product is done
    uint64_t* level = o_done + 2;    // the softmax warps are as far as the others, where streams are joined
    uint64_t* drain = level + 1;
    uint16_t* info = reinterpret_cast<uint16_t*>(smem + C::OFF_INFO);
    float2* s_ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int subs = a.H_kv * sh.pairs;
    const float NEG_INF = __int_as_float(0xff800000);
    const unsigned long long drain_ns = a.wait_ns > kDefaultWaitNs ? a.wait_ns : kDefaultWaitNs;

    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(full + i, 1);
            mbar_init(empty + i, 1);
            mbar_init(v_tree + i, 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 2);  // the product's completion, and the issuing thread
            mbar_init(p_full + i, 4);
            mbar_init(o_done + i, 2);  // as s_full
        }
        mbar_init(level, 8);
        mbar_init(drain, 1);
        mbar_fence_init();
        s_asked = 0;
        s_gave_up = 0;
    }
    if (warp == 8 && elect_one()) {
        tma_prefetch_desc(&maps.q);
        tma_prefetch_desc(&maps.k);
        tma_prefetch_desc(&maps.k_edge);
        tma_prefetch_desc(&maps.kt);
    }
    if (warp == 11 && elect_one()) {
        tma_prefetch_desc(&maps.v);
        tma_prefetch_desc(&maps.v_edge);
        tma_prefetch_desc(&maps.vt);
    }
    pdl_wait();
    pdl_trigger();

    // This CTA's share: where it begins (unit and tile) and how many tiles, in shared memory (what every role would carry in
    // registers otherwise costs the softmax its own).
    {
        auto tiles_of = [&](int len) { return sh.pages(len, a.max_pages) < 0 ? 1 : (len + kTokens - 1) / kTokens + 1; };
        if (warp == 9) tmem_alloc(&s_tmem, C::COLUMNS);
        if (few) {
            // A unit's tiles are cut into equal parts, none of more tiles than there have to be for all parts to find a CTA, so
            // that no CTA goes from one unit to the next: one warp, a sequence a lane.
            if (warp == 0) {
                int len = 0, nt = 0;
                if (lane < a.B) {
                    len = a.seq_lens[lane];
                    nt = tiles_of(len);
                }
                int most = max(1, (__reduce_add_sync(0xffffffffu, nt) * subs + (int)gridDim.x - 1) / (int)gridDim.x), parts;
                for (;; most += 1 + (most >> 4)) {  // (ends where every unit is one part at the latest: there are more CTAs)
                    parts = (nt + most - 1) / most;
                    if (__reduce_add_sync(0xffffffffu, parts) * subs <= (int)gridDim.x) break;
                }
                int incl = parts * subs;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, off);
                    if (lane >= off) incl += y;
                }
                const unsigned mine = __ballot_sync(0xffffffffu, lane < a.B && (int)blockIdx.x < incl);
                if (lane == (mine ? __ffs((int)mine) - 1 : 0)) {
                    const int off = (int)blockIdx.x - (incl - parts * subs);
                    Share x = {lane, 0, 0, len, 0, 0, 0, 0};
                    if (mine) {
                        x.sub = off / parts;
                        const int part = off - x.sub * parts;
                        const int t0 = (int)((unsigned)nt * part / parts);  // (at most 2^23 tiles, 256 parts)
                        x.t0 = t0 + kUnitTiles;
                        x.left = (int)((unsigned)nt * (part + 1) / parts) - t0;
                        x.follow = part == 0 ? parts - 1 : 0;
                    }
                    s_share = x;
                }
            }
        } else {
            // all tiles in a row, in equal shares
            auto cost_of = [&](int len) { return tiles_of(len) + kUnitTiles; };
            const int per = (a.B + kThreads - 1) / kThreads;
            const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
            int len = 0;  // of this thread's last sequence
            long long mine = 0;
            for (int b = b0; b < b1; ++b) {
                len = a.seq_lens[b];
                mine += (long long)cost_of(len) * subs;
            }
            long long incl = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += y;
            }
            if (lane == 31) s_scan[warp] = incl;
            __syncthreads();
            long long sums = lane < kThreads / 32 ? s_scan[lane] : 0;
#pragma unroll
            for (int off = 1; off < 16; off <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, sums, off);
                if (lane >= off) sums += y;
            }
            const long long total = __shfl_sync(0xffffffffu, sums, kThreads / 32 - 1);
            long long before = __shfl_sync(0xffffffffu, sums, warp > 0 ? warp - 1 : 0);
            before = (warp > 0 ? before : 0) + incl - mine;
            const int ctas = (int)min((long long)gridDim.x, total);
            const bool any = (int)blockIdx.x < ctas;
            const Shares shares(total, ctas);
            const long long g0 = any ? shares.begin(blockIdx.x) : 0;
            if (before <= g0 && g0 < before + mine) {  // one thread's
                int b = b0;
                if (per > 1) len = a.seq_lens[b];
                long long at = before;
                while (g0 - at >= (long long)cost_of(len) * subs) {
                    at += (long long)cost_of(len) * subs;
                    len = a.seq_lens[++b];
                }
                const long long off = g0 - at;
                const int nt = cost_of(len);
                Share x = {b, 0, 0, len, any ? shares.begin(blockIdx.x + 1) - g0 : 0, g0, total, 0};
                x.sub = off < 0x7fffffff ? (int)off / nt : (int)(off / nt);
                x.t0 = (int)(off - (long long)x.sub * nt);
                s_share = x;
            }
        }
        tmem_fence_before();
        __syncthreads();
        tmem_fence_after();
        Walk w;
        w.b = s_share.b;
        w.sub = s_share.sub;
        w.t0 = s_share.t0;
        w.left = s_share.left;
        w.look(a, sh, s_share.len);
        float* part_o = part_o_of(a.ws, (int)gridDim.x);
        float2* part_ml = part_ml_of(a.ws, (int)gridDim.x, D);
        const uint32_t tmem = s_tmem;
        const uint32_t q_smem = smem_u32(smem + C::OFF_Q), ring_smem = smem_u32(smem + C::OFF_RING);

        if (warp < 8) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
            // ======================================================== softmax
            const int s = warp >> 2;               // the stream
            const int row = (warp & 3) * 32 + lane;  // of its row tile
            const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
            const uint32_t tm_s = tmem + C::COL_S + s * 128 + lanes, tm_o = tmem + C::COL_O + lanes;
            const float scale = fmaxf(fabsf(a.scale_log2), 1e-37f);  // (0 would make -inf, a hidden token, a NaN)
            const bool flip = a.scale_log2 < 0.f;
            uint32_t s_parity = 0, o_parity = 0, level_parity = 0;
            int tiles_done = 0, piece = -1;  // of the pieces before: their visible tokens' places
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, a.status, a.wait_ns));
                return ok;
            };
            // a barrier of the eight softmax warps that no warp can be held at (a warp that has given up is counted no more)
            auto all_level = [&]() {
                if (!ok) return;
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(level);
                wait(level, level_parity);
                level_parity ^= 1u;
                tmem_fence_after();
            };
            int tree_b = -1;
            unsigned long long tree[2] = {0, 0};
            Piece p;
            while (ok && w.next(a, sh, p)) {
                const int h = sh.head(p.sub), mt = sh.first_tile(p.sub);
                const bool two = mt + 1 < sh.row_tiles;
                const int n = p.t1 - p.t0, step = two ? 1 : 2;
                ++piece;
                if (p.b != tree_b) {
                    tree_masks(a.parents + (long long)p.b * a.T, a.T, tree);
                    if (p.bad) tree[0] = tree[1] = 0;
                    tree_b = p.b;
                }
                const int node = (mt + (two ? s : 0)) * sh.tpt + row / sh.G;
                const bool there = row < sh.tpt * sh.G && node < a.T;
                const unsigned long long m_lo = __shfl_sync(0xffffffffu, tree[0], node & 31), m_hi = __shfl_sync(0xffffffffu, tree[1], node & 31);
                const unsigned long long mask = !there ? 0 : node < 32 ? m_lo : m_hi;
                float ref = NEG_INF, sum = 0.f;
                // outputs, or the partial of slot 2 i (a unit that began before this share) or 2 i + 1; until then what this row has put aside
                const int slot = 2 * (int)blockIdx.x + (p.t0 == 0 ? 1 : 0);
                auto aside = [&]() { return reinterpret_cast<float4*>(part_o) + (size_t)slot * kSlotRows * (D / 4) + s * kRows + row; };
                auto aside_ml = [&]() { return part_ml + (size_t)slot * kSlotRows + s * kRows + row; };
                for (int j = two ? 0 : s; j < n; j += step) {
                    const int t = p.t0 + j;
                    if (!wait(s_full + s, s_parity)) break;
                    s_parity ^= 1u;
                    tmem_fence_after();
                    uint32_t x[4][32];
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_ld(tm_s + 32 * i, x[i]);
                    uint4 seen = *reinterpret_cast<const uint4*>(info + ((tiles_done + j) & (kInfos - 1)) * 8);
                    if (t == p.nt - 1) seen = make_uint4((uint32_t)mask, (uint32_t)(mask >> 32), 0u, 0u);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 4; ++i) tmem_loaded(x[i]);
                    if (flip) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int c = 0; c < 32; ++c) x[i][c] ^= 0x80000000u;
                    }
                    if (__any_sync(0xffffffffu, (seen.x & seen.y & seen.z & seen.w) != 0xffffffffu)) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t bits = i == 0 ? seen.x : i == 1 ? seen.y : i == 2 ? seen.z : seen.w;
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                if (!(bits >> c & 1u)) x[i][c] = 0xff800000u;
                        }
                    }
                    float top[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        top[i] = __uint_as_float(x[i][0]);
#pragma unroll
                        for (int c = 1; c < 31; c += 2) top[i] = fmaxf(top[i], fmaxf(__uint_as_float(x[i][c]), __uint_as_float(x[i][c + 1])));
                        top[i] = fmaxf(top[i], __uint_as_float(x[i][31]));
                    }
                    const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
                    const bool moves = most > ref + kLag;
                    const int i_s = j >> (step - 1);  // the stream's tile
                    const bool full_up = i_s > 0 && (i_s & (kAside - 1)) == 0;
                    if (full_up || __any_sync(0xffffffffu, moves)) {
                        const float now = moves ? most : ref;
                        const float corr = moves ? fast_exp2(ref - now) : 1.f;
                        ref = now;
                        sum *= corr;
                        if (full_up) {  // put aside, at the new reference; the next product starts from nothing
                            const bool more = i_s > kAside;
                            const float2 ml = more ? *aside_ml() : make_float2(NEG_INF, 0.f);
                            const float w = ml.x == NEG_INF ? 0.f : fast_exp2(ml.x - ref);
                            *aside_ml() = make_float2(ref, sum + (ml.x == NEG_INF ? ml.y : ml.y * w));
                            sum = 0.f;
                            float4* at = aside();
#pragma unroll 1
                            for (int i = 0; i < D; i += 16) {
                                uint32_t o[16];
                                tmem_ld(tm_o + s * 128 + i, o);
                                tmem_wait_ld();
                                tmem_loaded(o);
#pragma unroll
                                for (int c = 0; c < 16; c += 4, at += kSlotRows) {
                                    const float4 x = more ? *at : make_float4(0.f, 0.f, 0.f, 0.f);
                                    *at = make_float4(fmaf(__uint_as_float(o[c]), corr, x.x * w), fmaf(__uint_as_float(o[c + 1]), corr, x.y * w),
                                                      fmaf(__uint_as_float(o[c + 2]), corr, x.z * w), fmaf(__uint_as_float(o[c + 3]), corr, x.w * w));
                                }
                            }
                        } else if (j >= step) {  // O of the tiles before; their products are done, as S's is
#pragma unroll 1
                            for (int i = 0; i < D; i += 16) {
                                uint32_t o[16];
                                tmem_ld(tm_o + s * 128 + i, o);
                                tmem_wait_ld();
                                tmem_loaded(o);
#pragma unroll
                                for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * corr);
                                tmem_st(tm_o + s * 128 + i, o);
                            }
                        }
                    }
                    const float neg = ref == NEG_INF ? 0.f : -ref;
                    const float2 scale2 = make_float2(scale, scale), neg2 = make_float2(neg, neg);
                    float2 l0 = make_float2(0.f, 0.f), l1 = l0;  // of this tile
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t w16[16];
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float2 y = fma2(make_float2(__uint_as_float(x[i][2 * c]), __uint_as_float(x[i][2 * c + 1])), scale2, neg2);
                            const float2 e = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                            if (c & 1) l1 = add2(l1, e);
                            else l0 = add2(l0, e);
                            w16[c] = pack_bf16(e.x, e.y);
                        }
                        tmem_st(tm_s + 16 * i, w16);
                    }
                    tmem_wait_st();
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_full + s);
                    sum += l0.x + l0.y + (l1.x + l1.y);
                }
                if (!ok) break;
                tiles_done += n;
                const bool whole = p.t0 == 0 && p.t1 == p.nt;
                const long long out = ((long long)p.b * a.T + node) * a.H_q + h * sh.G + row % sh.G;
                bf16* o_row = reinterpret_cast<bf16*>(a.o) + out * D;
                float4* part = reinterpret_cast<float4*>(part_o) + (size_t)slot * kSlotRows * (D / 4) + (two ? s * kRows : 0) + row;
                // values that are not finite, of the nodes that this row sees: added to columns c0 ... c0 + 15
                auto give_back = [&](float (&o)[16], int c0) {
                    unsigned long long odd = p.t1 == p.nt ? *reinterpret_cast<volatile unsigned long long*>(s_odd + (piece & (kOdd - 1))) & mask : 0;
                    while (odd) {
                        const int u = __ffsll((long long)odd) - 1;
                        odd &= odd - 1;
                        const bf16* v = reinterpret_cast<const bf16*>(a.v_tree) + ((long long)p.b * a.T + u) * a.v_stride + h * D + c0;
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const float x = __bfloat162float(v[c]);
                            if (!(fabsf(x) <= 3.4e38f)) o[c] += x;
                        }
                    }
                };
                // 16 columns of this row's result, from column c0
                auto put = [&](const float (&o)[16], int c0, float inv) {
                    if (whole) {
                        if (there) {
#pragma unroll
                            for (int c = 0; c < 16; c += 8) {
                                uint4 v;
                                v.x = pack_bf16(o[c] * inv, o[c + 1] * inv);
                                v.y = pack_bf16(o[c + 2] * inv, o[c + 3] * inv);
                                v.z = pack_bf16(o[c + 4] * inv, o[c + 5] * inv);
                                v.w = pack_bf16(o[c + 6] * inv, o[c + 7] * inv);
                                *reinterpret_cast<uint4*>(o_row + c0 + c) = v;
                            }
                        }
                    } else if (there) {
#pragma unroll
                        for (int c = 0; c < 16; c += 4) part[(size_t)((c0 + c) / 4) * kSlotRows] = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                    }
                };
                if (s < n || two) {  // (the other stream's end is known behind the barrier below)
                    if (!wait(o_done + s, o_parity)) break;
                    o_parity ^= 1u;
                }
                tmem_fence_after();
                if ((two ? n : (n - s + 1) >> 1) > kAside) {  // what was put aside, back to O
                    const float2 ml = *aside_ml();
                    const float w = ml.x == NEG_INF ? 0.f : fast_exp2(ml.x - ref);
                    sum += ml.x == NEG_INF ? ml.y : ml.y * w;
                    const float4* at = aside();
#pragma unroll 1
                    for (int i = 0; i < D; i += 16) {
                        uint32_t o[16];
                        tmem_ld(tm_o + s * 128 + i, o);
                        tmem_wait_ld();
                        tmem_loaded(o);
#pragma unroll
                        for (int c = 0; c < 16; c += 4, at += kSlotRows) {
                            const float4 x = *at;
                            o[c] = __float_as_uint(fmaf(x.x, w, __uint_as_float(o[c])));
                            o[c + 1] = __float_as_uint(fmaf(x.y, w, __uint_as_float(o[c + 1])));
                            o[c + 2] = __float_as_uint(fmaf(x.z, w, __uint_as_float(o[c + 2])));
                            o[c + 3] = __float_as_uint(fmaf(x.w, w, __uint_as_float(o[c + 3])));
                        }
                        tmem_st(tm_o + s * 128 + i, o);
                    }
                    tmem_wait_st();
                }
                // the row's parts: this stream's, or both streams', of which this warpgroup joins half of the channels
                float w0 = 1.f, w1 = 0.f;
                if (!two) {
                    if (s == 1) s_ml[row] = make_float2(ref, sum);
                    all_level();
                    float2 ml0 = make_float2(ref, sum), ml1 = ml0;
                    if (s == 0) {  // the other's, and in its place this one's
                        ml1 = s_ml[row];
                        s_ml[row] = ml0;
                    }
                    all_level();
                    if (!ok) break;
                    if (s == 1) ml0 = s_ml[row];
                    ref = fmaxf(ml0.x, ml1.x);
                    w0 = ml0.x == NEG_INF ? 0.f : fast_exp2(ml0.x - ref);
                    w1 = ml1.x == NEG_INF ? 0.f : fast_exp2(ml1.x - ref);
                    // (a row of NaN logits alone has a sum of NaN and no reference)
                    sum = (ml0.x == NEG_INF ? ml0.y : ml0.y * w0) + (ml1.x == NEG_INF ? ml1.y : ml1.y * w1);
                }
                if (mask == 0) {
                    sum = 0.f;
                    ref = NEG_INF;
                }
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                const uint32_t tm_a = tm_o + (two ? s * 128 : 0);
                const int c_end = two ? D : (s + 1) * (D / 2);
#pragma unroll 1
                for (int c0 = two ? 0 : s * (D / 2); c0 < c_end; c0 += 16) {
                    uint32_t oa[16], ob[16];
                    tmem_ld(tm_a + c0, oa);
                    if (!two && n > 1) tmem_ld(tm_o + 128 + c0, ob);
                    tmem_wait_ld();
                    tmem_loaded(oa);
                    float v[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) v[c] = __uint_as_float(oa[c]) * w0;
                    if (!two && n > 1) {
                        tmem_loaded(ob);
#pragma unroll
                        for (int c = 0; c < 16; ++c) v[c] = fmaf(__uint_as_float(ob[c]), w1, v[c]);
                    }
                    if (mask == 0) {
#pragma unroll
                        for (int c = 0; c < 16; ++c) v[c] = 0.f;
                    }
                    give_back(v, c0);
                    put(v, c0, inv);
                }
                if ((two || s == 0) && there) {
                    if (whole) {
                        if (a.lse) a.lse[out] = sum == 0.f ? NEG_INF : (ref + log2f(sum)) * kLn2;
                    } else {
                        part_ml[(size_t)slot * kSlotRows + (two ? s * kRows : 0) + row] = make_float2(ref, sum);
                    }
                }
                if (two) tmem_fence_before();
                else all_level();  // both have read O and the references
            }
            if (!ok && lane == 0) *reinterpret_cast<volatile int*>(&s_gave_up) = 1;
        } else if (warp == 8 || warp == 11) {
            other_regs();
            // ======================================================== copies: keys and queries, or values
            const bool value = warp == 11;
            const int lg_ps = sh.lg_ps, ppt = kTokens >> lg_ps;  // pages of a tile
            const int lg_batch = lg_ps - 2;                      // 32 page-table entries are 2^lg_batch tiles
            const int oob = (int)max(1LL, a.num_phys * a.H_kv);      // a row of pages that is not there
            const CUtensorMap* map = value ? &maps.v : &maps.k;
            const CUtensorMap* map_edge = value ? &maps.v_edge : &maps.k_edge;
            uint32_t q_parity = 1, v_parity = 0;                // v_parity: of each slot's next nodes, bits
            uint32_t asked = 0, asked_nodes = 0, asked_parity = 0;  // this warp's last copy to each slot, bits
            int base = 0, n_info = 0;                            // items, and tiles, of the pieces before
            int asked_item = 0;                                  // lane i: of slot i
            bool ok = true, q_asked = false;
            Piece p;
            while (ok && w.next(a, sh, p)) {
                const int h = sh.head(p.sub), mt = sh.first_tile(p.sub);
                const bool two = mt + 1 < sh.row_tiles;
                const int n = p.t1 - p.t0;
                const int P = (p.len + a.ps - 1) >> lg_ps;
                // page-table entries, 32 at a time, asked for before the queries
                const int32_t* table = a.page_table + (long long)p.b * a.max_pages;
                auto ask = [&](int batch) {
                    const int e = batch * 32 + lane;
                    return e < P ? table[e] : -1;
                };
                auto checked = [&](int batch, int phys) {
                    if (batch * 32 + lane < P && (phys < 0 || phys >= a.num_phys)) {
                        raise_status(a.status, SPD_DEV_BAD_PAGE);
                        phys = -1;
                    }
                    return phys;
                };
                int batch = p.t0 >> lg_batch;
                int ids = ask(batch), nxt = ask(batch + 1);
                if (!value) {
                    if (p.bad && p.sub == 0 && lane == 0) raise_status(a.status, SPD_DEV_BAD_LEN);
                    // queries
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(q_empty, q_parity, a.status, a.wait_ns));
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(q_full, (two ? 2 : 1) * C::HALVES * sh.tpt * sh.G * 128);
                        for (int s = 0; s < (two ? 2 : 1); ++s)
                            for (int x = 0; x < C::HALVES; ++x)
                                tma_load_4d(smem + C::OFF_Q + s * C::TILE + x * C::HALF, &maps.q, 0, h * sh.G, p.b * a.T + (mt + s) * sh.tpt, x, q_full);
                    }
                    q_asked = true;
                    q_parity ^= 1u;
                }
                ids = checked(batch, ids);
                for (int j = 0; j < n; ++j) {
                    // the items' order, as the products take them: two row tiles K0 V0 K1 V1 ...; one K0 K1 V0 K2 V1 ...
                    const int item = base + (two ? 2 * j + (value ? 1 : 0) : value ? min(2 * j + 2, 2 * n - 1) : max(0, 2 * j - 1));
                    const int t = p.t0 + j, slot = item % STAGES;
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(empty + slot, ((uint32_t)(item / STAGES) & 1u) ^ 1u, a.status, a.wait_ns));
                    if (!ok) break;
                    uint8_t* dst = smem + C::OFF_RING + slot * C::TILE;
                    uint64_t* bar = full + slot;
                    if (t < p.nt - 1) {
                        if (t >> lg_batch > batch) {
                            ++batch;
                            ids = checked(batch, nxt);
                            nxt = ask(batch + 1);
                        }
                        // lane i copies page i
                        const int i = lane & (ppt - 1);
                        const int page = t * ppt + i;
                        const int phys = __shfl_sync(0xffffffffu, ids, page & 31);
                        const int valid = min(a.ps, p.len - (page << lg_ps));  // its tokens (below 1: none)
                        if (!value) {
                            // 16 tokens a lane: a page's valid tokens are the last of its place in the tile
                            const int gi = lane & 7, own = gi * 16 >> lg_ps;
                            const int op = __shfl_sync(0xffffffffu, phys, own), ov = __shfl_sync(0xffffffffu, valid, own);
                            const int hidden = (op < 0 || ov < 1 ? a.ps : a.ps - ov) - (gi * 16 & (a.ps - 1));
                            const uint16_t bits = (uint16_t)(hidden <= 0 ? 0xffffu : hidden >= 16 ? 0u : 0xffffu << hidden);
                            if (lane < 8) info[(n_info & (kInfos - 1)) * 8 + gi] = bits;
                            ++n_info;
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive_expect_tx(bar, C::TILE);
                        __syncwarp();
                        const bool there = phys >= 0 && valid > 0;
                        const unsigned cut = __ballot_sync(0xffffffffu, lane < ppt && there && valid < a.ps);
                        if (lane < ppt && !(there && valid < a.ps))
                            tma_load_5d(dst + (i << lg_ps) * (D * 2), map, 0, 0, 0, 0, there ? phys * a.H_kv + h : oob, bar);
                        if (cut) {  // the sequence's last page, eight slots and 64 channels at a time
                            const int e = __ffs((int)cut) - 1;
                            const int ep = __shfl_sync(0xffffffffu, phys, e), ev = __shfl_sync(0xffffffffu, valid, e);
                            const int grp = lane / C::HALVES, half = lane % C::HALVES;
                            if (grp < a.ps >> 3)
                                tma_load_4d(dst + (e << lg_ps) * (D * 2) + lane * 1024, map_edge, 0, grp * 8 + ev - a.ps, half, ep * a.H_kv + h, bar);
                        }
                        asked_nodes &= ~(1u << slot);
                    } else {
                        // the nodes: 64 rows, zeros behind the last
                        uint64_t* to = value ? v_tree + slot : bar;
                        ++n_info;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(to, C::HALVES * 64 * 128);
                            for (int half = 0; half < C::HALVES; ++half)
                                tma_load_5d(dst + half * C::HALF, value ? &maps.vt : &maps.kt, 0, 0, p.b, h, half, to);
                        }
                        if (value) {
                            asked_nodes |= 1u << slot;
                            v_parity ^= 1u << slot;
                        }
                    }
                    asked |= 1u << slot;
                    if (value && lane == 0) *reinterpret_cast<volatile int*>(&s_asked) = base / 2 + j + 1;
                    if (lane == slot) asked_item = item;
                    asked_parity = (asked_parity & ~(1u << slot)) | ((uint32_t)(item / STAGES) & 1u) << slot;
                }
                base += 2 * n;
            }
            // copies land before their memory is given back, also where the products no longer wait for them.  (Where all have
            // been asked for, the other warp's later item in a slot has this one's behind it, and the barrier two phases on.)
            for (int i = 0; i < STAGES; ++i) {
                if (!(asked >> i & 1u) || (ok && __shfl_sync(0xffffffffu, asked_item, i) < base - STAGES)) continue;
                if (asked_nodes >> i & 1u) mbar_wait_bounded(v_tree + i, ~v_parity >> i & 1u, a.status, drain_ns);
                else mbar_wait_bounded(full + i, asked_parity >> i & 1u, a.status, drain_ns);
            }
            if (q_asked) mbar_wait_bounded(q_full, q_parity, a.status, drain_ns);
        } else if (warp == 9) {
            other_regs();
            // ======================================================== products
            constexpr uint32_t kIdescS = umma_idesc_bf16(kRows, kTokens, false, false);
            constexpr uint32_t kIdescO = umma_idesc_bf16(kRows, D, false, true);
            uint32_t q_parity = 0, p_parity = 0;  // (of both streams: bits)
            int base = 0;  // items of the ring before this piece
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, a.status, a.wait_ns));
                return ok;
            };
            auto wait_item = [&](int item) { return wait(full + item % STAGES, (uint32_t)(item / STAGES) & 1u); };
            // S of stream s with row tile q and the keys of an item
            // (Descriptors count in 16 bytes: the steps' are sums.  Loops rolled but for two steps: unrolled at every place, what they share is kept
            // in registers that the softmax then spills, 571 us against 565.)
            auto keys = [&](int s, int q, int item, bool tree) {
                tmem_fence_after();
                if (elect_one()) {
                    const uint32_t half = (tree ? C::HALF : 1024) >> 4;
                    const uint64_t dq = umma_desc(q_smem + q * C::TILE, 0, 1024, kSwizzle128);
                    const uint64_t dk = umma_desc(ring_smem + item % STAGES * C::TILE, 0, tree ? 1024 : C::GROUP, kSwizzle128);
#pragma unroll (D / 64)
                    for (int i = 0; i < D / 16; ++i)
                        umma_f16_ss(tmem + C::COL_S + s * 128, dq + (((i >> 2) * C::HALF + (i & 3) * 32) >> 4), dk + ((i >> 2) * half + (i & 3) * 2),
                                    kIdescS, i > 0);
                    umma_commit(s_full + s);
                    mbar_arrive(s_full + s);
                }
                __syncwarp();
            };
            auto values = [&](int s, int item, bool first, bool tree) {
                tmem_fence_after();
                if (elect_one()) {
                    const uint32_t group = tree ? 1024 : C::GROUP;
                    const uint64_t dv = umma_desc(ring_smem + item % STAGES * C::TILE, tree ? C::HALF : 1024, group, kSwizzle128);
                    const int steps = tree ? 4 : 8;
#pragma unroll 2
                    for (int i = 0; i < steps; ++i)
                        umma_f16_ts(tmem + C::COL_O + s * 128, tmem + C::COL_S + s * 128 + 8 * i, dv + i * (2 * group >> 4), kIdescO, !first || i > 0);
                }
                __syncwarp();
            };
            auto commit = [&](uint64_t* bar) {
                if (elect_one()) umma_commit(bar);
                __syncwarp();
            };
            auto last_product = [&](int s) {
                if (elect_one()) {
                    umma_commit(o_done + s);
                    mbar_arrive(o_done + s);
                }
                __syncwarp();
            };
            auto wait_p = [&](int s) {
                wait(p_full + s, p_parity >> s & 1u);
                p_parity ^= 1u << s;
                return ok;
            };
            Piece p;
            while (ok && w.next(a, sh, p)) {
                const int h = sh.head(p.sub), mt = sh.first_tile(p.sub);
                const bool two = mt + 1 < sh.row_tiles;
                const int n = p.t1 - p.t0;
                if (!wait(q_full, q_parity)) break;
                q_parity ^= 1u;
                if (two) {
                    if (!wait_item(base)) break;
                    keys(0, 0, base, p.t0 == p.nt - 1);
                    keys(1, 1, base, p.t0 == p.nt - 1);
                    commit(empty + base % STAGES);
                    if (n == 1) commit(q_empty);
                    for (int i = 0; i < n && ok; ++i) {
                        const int kn = base + 2 * i + 2, vi = base + 2 * i + 1;
                        const bool tree = p.t0 + i == p.nt - 1;
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            if (!wait_p(s)) break;
                            if (s == 0 && !wait_item(vi)) break;
                            values(s, vi, (i & (kAside - 1)) == 0, tree);
                            if (s == 1) commit(empty + vi % STAGES);
                            if (i + 1 < n) {
                                if (s == 0 && !wait_item(kn)) break;
                                keys(s, s, kn, p.t0 + i + 1 == p.nt - 1);
                                if (s == 1) {
                                    commit(empty + kn % STAGES);
                                    if (i + 2 == n) commit(q_empty);
                                }
                            } else {
                                last_product(s);
                            }
                        }
                    }
                } else {
                    for (int j = 0; j < min(n, 2) && ok; ++j) {
                        if (!wait_item(base + j)) break;
                        keys(j, 0, base + j, p.t0 + j == p.nt - 1);
                        commit(empty + (base + j) % STAGES);
                        if (j + 1 == n) commit(q_empty);
                    }
                    for (int i = 0; i < n && ok; ++i) {
                        const int s = i & 1, vi = base + min(2 * i + 2, 2 * n - 1), kn = base + 2 * i + 3;  // keys of tile i + 2
                        if (!wait_p(s) || !wait_item(vi)) break;
                        values(s, vi, ((i >> 1) & (kAside - 1)) == 0, p.t0 + i == p.nt - 1);
                        commit(empty + vi % STAGES);
                        if (i + 2 < n) {
                            if (!wait_item(kn)) break;
                            keys(s, 0, kn, p.t0 + i + 2 == p.nt - 1);
                            commit(empty + kn % STAGES);
                            if (i + 3 == n) commit(q_empty);
                        } else {
                            last_product(s);
                        }
                    }
                }
                base += 2 * n;
            }
            if (!ok) {  // products in flight end before their memory is given back
                commit(drain);
                mbar_wait_bounded(drain, 0, a.status, drain_ns);
            }
        } else if (warp == 10) {
            other_regs();
            // ======================================================== the nodes' values
            // first, a unit that begins here and ends behind the share is the joining kernel's work
            if (lane == 0) {
                Cut* cuts = reinterpret_cast<Cut*>(a.ws);
                if (few) {
                    if (w.left > 0 && w.t0 == kUnitTiles) {
                        const int parts = s_share.follow + 1;
                        cuts[w.b * subs + w.sub] = {w.b, w.sub, parts > 1 ? parts : 0, (int)blockIdx.x};
                    }
                } else {
                    Cut cut = {0, 0, 0, (int)blockIdx.x};
                    Walk x = w;
                    Piece p;
                    const Shares shares(s_share.total, (int)min((long long)gridDim.x, s_share.total));
                    while (x.next(a, sh, p)) {
                        if (p.t0 == 0 && p.t1 < p.nt) {
                            const long long end = s_share.at + (w.left - x.left) + (p.nt - p.t1);  // of the unit
                            int c = blockIdx.x;
                            while (shares.begin(c + 1) < end) ++c;
                            cut = {p.b, p.sub, c - (int)blockIdx.x + 1, (int)blockIdx.x};
                        }
                    }
                    cuts[blockIdx.x] = cut;
                }
            }
            __syncwarp();
            // A weight of 0 times an infinity or a NaN would reach rows that do not see the node: rows of what is
            // no node (which may hold anything) and values that are not finite become 0 here, and the rows that see
            // the latter get them back at the end.
            uint32_t v_parity = 0;  // of each slot: bits
            int base = 0, piece = 0;
            // A piece's nodes come behind all of its tiles: the limit counts from the last tile that was asked for.
            auto wait_nodes = [&](uint64_t* bar, uint32_t parity) {
                int asked = -1;
                unsigned long long since = 0;
                while (!mbar_try_wait(bar, parity)) {
                    const int now_asked = *reinterpret_cast<volatile int*>(&s_asked);
                    const unsigned long long now = globaltimer_ns();
                    if (now_asked != asked) {
                        asked = now_asked;
                        since = now;
                    } else if (now - since > a.wait_ns) {
                        raise_status(a.status, SPD_DEV_TIMEOUT);
                        return false;
                    }
                }
                return true;
            };
            Piece p;
            while (w.next(a, sh, p)) {
                base += 2 * (p.t1 - p.t0);
                if (p.t1 == p.nt) {
                    const int slot = (base - 1) % STAGES;
                    unsigned long long m[2];
                    if (!tree_masks(a.parents + (long long)p.b * a.T, a.T, m) && lane == 0 && p.sub == 0) raise_status(a.status, SPD_DEV_BAD_TREE);
                    const unsigned long long gone = (unsigned long long)__ballot_sync(0xffffffffu, m[1] == 0) << 32 | __ballot_sync(0xffffffffu, m[0] == 0);
                    if (!__all_sync(0xffffffffu, wait_nodes(v_tree + slot, v_parity >> slot & 1u))) break;
                    v_parity ^= 1u << slot;
                    uint8_t* rows = smem + C::OFF_RING + slot * C::TILE;
                    unsigned long long odd = 0;
#pragma unroll 4
                    for (int i = 0; i < 2 * C::HALVES * 8; ++i) {
                        // 16 bytes a lane: four rows an access
                        const int y = i * 32 + lane, row = y >> 3 & 63;
                        uint32_t* at = reinterpret_cast<uint32_t*>(rows + (y >> 9) * C::HALF + row * 128 + (y & 7) * 16);
                        uint4 v = *reinterpret_cast<uint4*>(at);
                        // an exponent of ones carries into the sign's place
                        auto bad = [](uint32_t x) { return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
                        const bool none = gone >> row & 1;
                        const uint32_t any = bad(v.x) | bad(v.y) | bad(v.z) | bad(v.w);
                        if (none || any) {
                            auto clear = [&](uint32_t x) {
                                const uint32_t b = bad(x);
                                return none ? 0u : x & ~((b >> 15) * 0xffffu);
                            };
                            *reinterpret_cast<uint4*>(at) = make_uint4(clear(v.x), clear(v.y), clear(v.z), clear(v.w));
                            if (!none) odd |= 1ull << row;
                        }
                    }
                    odd = (unsigned long long)__reduce_or_sync(0xffffffffu, (uint32_t)(odd >> 32)) << 32 | __reduce_or_sync(0xffffffffu, (uint32_t)odd);
                    if (lane == 0) s_odd[piece & (kOdd - 1)] = odd;
                    async_proxy_fence();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full + slot);
                }
                ++piece;
            }
        }
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == 9) tmem_free(s_tmem, C::COLUMNS);
    if (s_gave_up && tid < kSlotRows) {  // what is in this CTA's slots is not joined
        float2* ml = part_ml_of(a.ws, (int)gridDim.x, D) + (size_t)2 * blockIdx.x * kSlotRows + tid;
        ml[0] = ml[kSlotRows] = make_float2(__int_as_float(0x7fffffff), 0.f);
    }
}

// Joins the partials of the units that shares' borders cut.  A thread has eight channels of a row and asks for eight partials at
// once.  A CTA has 2^lg_rows rows, `chunks` of which cover a unit; what is left of its threads goes over the partials in turn
// (SPLIT: few units, in many parts each) or has other channels.  (One sequence of 23,545 tokens with two KV heads, in 76 parts
// each: 16.6 us for the whole call, 27.5 where a thread goes over all partials of a row; 64 sequences of 1,024, 15 nodes, in two
// or three parts: 60 us, 5 more with splits.)
constexpr int kJoinChannels = 8, kJoinAhead = 8, kJoinThreads = 256;
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kJoinThreads, SPLIT ? 3 : 4) join_kernel(const TreeAttnArgs a, const Shape sh, int ctas, int lg_rows, int chunks) {
    __shared__ float4 s_o[SPLIT ? kJoinThreads : 1][2];
    __shared__ float2 s_ml[SPLIT ? kJoinThreads : 1];
    const float NEG_INF = __int_as_float(0xff800000);
    const int rows = 1 << lg_rows, others = kJoinThreads >> lg_rows, other = threadIdx.x >> lg_rows;
    const int splits = SPLIT ? others : 1, split = SPLIT ? other : 0;
    const int groups = SPLIT ? 1 : others;  // eight channels each
    const int blocks = D / kJoinChannels / groups, chunk = blockIdx.x % (unsigned)chunks, block = blockIdx.x / (unsigned)chunks;
    const int unit = block / blocks, group = (block - unit * blocks) * groups + (SPLIT ? 0 : other);
    const int at = (chunk << lg_rows) + (int)(threadIdx.x & (rows - 1));  // of the unit's two row tiles
    const float2* part_ml = part_ml_of(a.ws, ctas, D) + at;
    const float4* part = reinterpret_cast<const float4*>(part_o_of(a.ws, ctas)) + group * 2 * kSlotRows + at;
    pdl_wait();
    pdl_trigger();
    const Cut cut = reinterpret_cast<const Cut*>(a.ws)[unit];
    if (cut.pieces == 0) return;
    const int h = sh.head(cut.sub), mt = sh.first_tile(cut.sub);
    const int row = at & (kRows - 1), node = (mt + at / kRows) * sh.tpt + row / sh.G;
    const bool valid = mt + at / kRows < sh.row_tiles && row < sh.tpt * sh.G && node < a.T;
    float r = NEG_INF, total = 0.f;
    bool gone = false;  // a part is not there
    float4 o0 = make_float4(0.f, 0.f, 0.f, 0.f), o1 = o0;
    auto add = [&](float now, float m, float l, float4 x, float4 y) {
        const float w = m == NEG_INF ? 0.f : fast_exp2(m - now);
        total += m == NEG_INF ? l : l * w;  // (a row of NaN logits alone has no reference)
        o0 = make_float4(fmaf(x.x, w, o0.x), fmaf(x.y, w, o0.y), fmaf(x.z, w, o0.z), fmaf(x.w, w, o0.w));
        o1 = make_float4(fmaf(y.x, w, o1.x), fmaf(y.y, w, o1.y), fmaf(y.z, w, o1.z), fmaf(y.w, w, o1.w));
    };
    auto follow = [&](float now) {
        const float corr = r == NEG_INF ? 0.f : fast_exp2(r - now);
        total = r == NEG_INF ? total : total * corr;
        r = now;
        o0 = make_float4(o0.x * corr, o0.y * corr, o0.z * corr, o0.w * corr);
        o1 = make_float4(o1.x * corr, o1.y * corr, o1.z * corr, o1.w * corr);
    };
    for (int i0 = split; valid && i0 < cut.pieces; i0 += kJoinAhead * splits) {
        float2 ml[kJoinAhead];
        float4 x[kJoinAhead], y[kJoinAhead];
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
            const int i = i0 + k * splits;
            // a unit's first partial is its CTA's second slot, the others are their CTAs' first
            const size_t slot = (size_t)(2 * (cut.cta + i) + (i == 0 ? 1 : 0));
            ml[k] = make_float2(NEG_INF, 0.f);
            x[k] = y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < cut.pieces) {
                ml[k] = part_ml[slot * kSlotRows];
                x[k] = part[slot * (D / 4) * kSlotRows];
                y[k] = part[(slot * (D / 4) + 1) * kSlotRows];
            }
        }
        float now = r;
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) {
            now = fmaxf(now, ml[k].x);
            gone |= ml[k].x != ml[k].x;
        }
        follow(now);
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k) add(now, ml[k].x, ml[k].y, x[k], y[k]);
    }
    if (SPLIT) {
        if (split > 0) {
            s_o[threadIdx.x][0] = o0;
            s_o[threadIdx.x][1] = o1;
            s_ml[threadIdx.x] = make_float2(gone ? __int_as_float(0x7fffffff) : r, total);
        }
        __syncthreads();
        if (split > 0) return;
        float now = r;
        for (int i = threadIdx.x + rows; i < kJoinThreads; i += rows) {
            now = fmaxf(now, s_ml[i].x);
            gone |= s_ml[i].x != s_ml[i].x;
        }
        follow(now);
        for (int i = threadIdx.x + rows; i < kJoinThreads; i += rows) add(now, s_ml[i].x, s_ml[i].y, s_o[i][0], s_o[i][1]);
    }
    if (!valid || gone) return;
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const long long out = ((long long)cut.b * a.T + node) * a.H_q + h * sh.G + row % sh.G;
    *reinterpret_cast<uint4*>(reinterpret_cast<bf16*>(a.o) + out * D + group * kJoinChannels) =
        make_uint4(pack_bf16(o0.x * inv, o0.y * inv), pack_bf16(o0.z * inv, o0.w * inv), pack_bf16(o1.x * inv, o1.y * inv),
                   pack_bf16(o1.z * inv, o1.w * inv));
    if (group == 0 && a.lse) a.lse[out] = total == 0.f ? NEG_INF : (r + log2f(total)) * kLn2;
}

template <int D>
cudaError_t launch(const TreeAttnArgs& a, const TreeMaps& m, int ctas, cudaStream_t st) {
    static std::atomic<bool> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !known[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(tree_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::SMEM);
        if (e != cudaSuccess) return e;
        if (dev < 64) known[dev].store(true, std::memory_order_release);
    }
    const Shape sh = shape_of(a.T, a.H_q / a.H_kv, a.ps);
    const long long units = (long long)a.B * a.H_kv * sh.pairs;
    const bool few = a.B <= 32 && units * kFewUnits <= ctas;
    e = launch_pdl(tree_kernel<D>, dim3((unsigned)ctas), dim3(kThreads), Cfg<D>::SMEM, st, a, m, sh, few);
    if (e != cudaSuccess) return e;
    const long long cuts = few ? units : ctas;
    // no more rows a CTA than there are; and where units are few, splits until a thread has eight partials or the GPU is full
    const int rows = sh.row_tiles == 1 ? sh.tpt * sh.G : kSlotRows;
    int lg = 5;
    auto chunks = [&] { return (rows + (1 << lg) - 1) >> lg; };
    auto blocks = [&] { return cuts * chunks() * (D / kJoinChannels) / (few ? 1 : kJoinThreads >> lg); };
    while (lg < 8 && chunks() > 1 && (!few || blocks() > 4 * a.num_sms || ctas <= units * kJoinAhead * (kJoinThreads >> (lg + 1)))) ++lg;
    return launch_pdl(few ? join_kernel<D, true> : join_kernel<D, false>, dim3((unsigned)blocks()), dim3(kJoinThreads), 0, st, a, sh, ctas, lg, chunks());
}

// CTAs: one an SM, or as many as there can be tiles.
int grid_of(int B, int H_kv, int G, int T, int max_pages, int ps, int num_sms) {
    const long long most = ((long long)max_pages * ps + kTokens - 1) / kTokens + 1;
    const long long tiles = most * B * H_kv * shape_of(T, G, ps).pairs;
    return (int)(tiles < num_sms ? tiles : num_sms);
}

}  // namespace

int tree_nodes_per_tile(int T, int G) { return shape_of(T, G, 16).tpt; }

size_t tree_attn_ws(int D, int num_sms) {
    return ((size_t)num_sms * sizeof(Cut) + 255) / 256 * 256 + 2 * num_sms * slot_bytes(D);
}

cudaError_t launch_tree_attn(const TreeAttnArgs& a, const TreeMaps& m, cudaStream_t st) {
    const int ctas = grid_of(a.B, a.H_kv, a.H_q / a.H_kv, a.T, a.max_pages, a.ps, a.num_sms);
    return a.D == 128 ? launch<128>(a, m, ctas, st) : launch<64>(a, m, ctas, st);
}

}  // namespace spd
