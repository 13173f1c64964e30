// spd_api.cu -- the C ABI of libspd (declared in include/spd.h): argument
// validation, workspace carving, TMA tensor-map encoding, launch-shape choice
// and dispatch to the kernels.  Nothing here allocates device memory or
// synchronises (except spd_device_status).
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>

#include "kernels.h"

#define SPD_API extern "C" __attribute__((visibility("default")))

namespace spd {
namespace {

thread_local std::string g_err;

// Device status word (SPD_DEV_* bits), one per device that loads the library.
__device__ unsigned g_status;

spd_status fail(spd_status s, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_err = buf;
    return s;
}

spd_status cuda_fail(cudaError_t e, const char* what) {
    return fail(SPD_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

constexpr int kMaxDevices = 64;
constexpr float kLog2e = 1.4426950408889634f;

struct DevInfo {
    std::once_flag once;
    unsigned* status = nullptr;
    int sms = 0;
    cudaError_t err = cudaSuccess;
};
DevInfo g_dev[kMaxDevices];

DevInfo* dev_info(spd_status* st) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) {
        *st = cuda_fail(e, "cudaGetDevice");
        return nullptr;
    }
    if (dev < 0 || dev >= kMaxDevices) {
        *st = fail(SPD_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
        return nullptr;
    }
    DevInfo* d = &g_dev[dev];
    std::call_once(d->once, [d, dev]() {
        void* p = nullptr;
        d->err = cudaGetSymbolAddress(&p, g_status);
        if (d->err == cudaSuccess) d->status = static_cast<unsigned*>(p);
        if (d->err == cudaSuccess) d->err = cudaDeviceGetAttribute(&d->sms, cudaDevAttrMultiProcessorCount, dev);
    });
    if (d->err != cudaSuccess) {
        *st = cuda_fail(d->err, "device set-up");
        return nullptr;
    }
    return d;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn(spd_status* st) {
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    static cudaError_t err = cudaSuccess;
    std::call_once(once, []() {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        err = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        if (err == cudaSuccess && q == cudaDriverEntryPointSuccess) fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    if (!fn) *st = fail(SPD_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable (%s)", cudaGetErrorString(err));
    return fn;
}

// 3-D view of a paged K or V cache: x = 64 channels (128 bytes), y = rows
// (num_phys * H_kv * ps of D bf16, stride 2D bytes), z = the D / 64 halves of a
// row (stride 128 bytes).  One box = a page's ps rows of one KV head (or `rows` of
// them), laid out in shared memory as [half][row][64] with the 128-byte swizzle.
spd_status kv_map(CUtensorMap* m, const void* base, const spd_dims* d, int rows = 0) {
    spd_status st = SPD_OK;
    EncodeTiledFn fn = encode_fn(&st);
    if (!fn) return st;
    cuuint64_t gdim[3] = {64, (cuuint64_t)d->num_phys_pages * d->H_kv * d->page_size, (cuuint64_t)d->D / 64};
    cuuint64_t gstride[2] = {(cuuint64_t)d->D * 2, 128};
    cuuint32_t box[3] = {64, (cuuint32_t)(rows ? rows : d->page_size), (cuuint32_t)d->D / 64};
    cuuint32_t estride[3] = {1, 1, 1};
    CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), gdim, gstride, box, estride,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(SPD_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return SPD_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

namespace {
std::atomic<unsigned long long> g_wait_ns{kDefaultWaitNs};
}  // namespace

unsigned long long wait_limit_ns() { return g_wait_ns.load(std::memory_order_relaxed); }

// Per-device set-up of the current device (status word, SM count), done once.
spd_status device_ready() {
    spd_status st = SPD_OK;
    return dev_info(&st) ? SPD_OK : st;
}

spd_status set_error(spd_status s, const char* msg) { return fail(s, "%s", msg); }

namespace {

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

spd_status check_dims(const spd_dims* d) {
    if (!d) return fail(SPD_ERR_INVALID_ARG, "dims is NULL");
    if (d->B < 0 || d->H_q <= 0 || d->H_kv <= 0 || d->max_pages_per_seq <= 0 || d->num_phys_pages < 0)
        return fail(SPD_ERR_INVALID_ARG, "bad dims (B=%d H_q=%d H_kv=%d max_pages=%d num_phys=%lld)", d->B,
                    d->H_q, d->H_kv, d->max_pages_per_seq, (long long)d->num_phys_pages);
    if (d->H_q % d->H_kv) return fail(SPD_ERR_INVALID_ARG, "H_q (%d) is not a multiple of H_kv (%d)", d->H_q, d->H_kv);
    if (d->H_q / d->H_kv > 8) return fail(SPD_ERR_UNSUPPORTED, "GQA group %d > 8", d->H_q / d->H_kv);
    if (d->D != 64 && d->D != 128) return fail(SPD_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", d->D);
    if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64)
        return fail(SPD_ERR_UNSUPPORTED, "page size %d (supported: 16, 32, 64)", d->page_size);
    if ((long long)d->num_phys_pages * d->H_kv * d->page_size >= (1LL << 31))
        return fail(SPD_ERR_UNSUPPORTED, "num_phys_pages * H_kv * page_size must be < 2^31");
    if ((long long)d->B * d->max_pages_per_seq >= (1LL << 31))
        return fail(SPD_ERR_UNSUPPORTED, "B * max_pages_per_seq must be < 2^31");
    return SPD_OK;
}

int pages_per_split_floor(int ps) { return ps >= 64 ? 2 : (ps == 32 ? 4 : 8); }

// Splits per row.  Sparse rows are short and about equal (k_max pages), so a
// row is one unit unless there are too few rows to occupy the persistent
// workers (a whole-row unit needs no partials or merge).  Dense rows differ in
// length by up to 2x, so they are cut into about units_per_worker units per
// worker for the queue to balance.  Each unit keeps at least floor_items pages.
int splits_for(long long rows, int items, long long workers, int floor_items, int units_per_worker,
               int req) {
    int S = req;
    if (S <= 0) {
        S = 1;
        const long long want = units_per_worker * workers;
        if (rows > 0 && (units_per_worker > 1 ? rows < want : 2 * rows < want)) {
            S = (int)((want + rows - 1) / rows);
            const int max_s = (items + floor_items - 1) / floor_items;
            if (S > max_s) S = max_s;
        }
    }
    if (S > items) S = items;
    if (S < 1) S = 1;
    const int ips = (items + S - 1) / S;
    return (items + ips - 1) / ips;
}

int sparse_splits(const spd_dims* d, int k_max, int req, int sms) {
    const long long rows = (long long)d->B * d->H_kv;
    const long long workers = (long long)sms * occ_sparse_attn(d->D, d->page_size);
    return splits_for(rows, k_max, workers, pages_per_split_floor(d->page_size), 1, req);
}

int dense_splits(const spd_dims* d, int T, int req, int sms) {
    const long long rows = (long long)d->B * d->H_kv;
    const int mt = attn_mtiles(T, d->H_q / d->H_kv);
    const long long workers = (long long)sms * occ_dense_attn(d->D, d->page_size, mt);
    return splits_for(rows, d->max_pages_per_seq, workers, 2 * pages_per_split_floor(d->page_size), 4, req);
}

struct AttnWs {
    int* queue;
    int* counters;
    float* part_lse;
    float* part_o;
    size_t bytes;
};

// [queue: 16 B][row tickets][partial lse][partial o]; the first two must start zeroed.
// Bytes of the queue and the tickets of these rows alone, as in scratch that no other call shares.
size_t ticket_bytes(long long rows) { return align256(16 + (size_t)rows * sizeof(int)); }

// The same in a caller's workspace: the place of every call's queue and tickets (those of the
// 4-bit attention and of token_logprobs too), which scores and partials of any call stay clear
// of, so it stays zero and one buffer serves calls of any kind and size in turn.
size_t ws_prefix(long long rows) {
    const size_t own = ticket_bytes(rows);
    return own > kTicketBytes ? own : kTicketBytes;
}

AttnWs attn_ws_layout(void* ws, long long rows, int S, int R, int D, size_t prefix) {
    AttnWs w;
    size_t off = prefix;
    char* base = static_cast<char*>(ws);
    w.queue = reinterpret_cast<int*>(base);
    w.counters = reinterpret_cast<int*>(base + 16);
    w.part_lse = reinterpret_cast<float*>(base + off);
    off += align256((size_t)rows * S * R * sizeof(float));
    w.part_o = reinterpret_cast<float*>(base + off);
    off += (size_t)rows * S * R * D * sizeof(float);
    w.bytes = off;
    return w;
}

// Bytes of attn_ws_layout the kernel touches: with one unit per row (S = 1) only
// the queue and the tickets (no partials).
size_t attn_ws_needed(long long rows, int S, int R, int D, size_t prefix) {
    if (S == 1) return ticket_bytes(rows);
    return attn_ws_layout(nullptr, rows, S, R, D, prefix).bytes;
}

}  // namespace
}  // namespace spd

using namespace spd;

SPD_API int32_t spd_version(void) { return 100; }

SPD_API const char* spd_last_error(void) { return g_err.c_str(); }

SPD_API spd_status spd_set_wait_limit_ns(uint64_t ns) {
    if (ns == 0) return fail(SPD_ERR_INVALID_ARG, "wait limit 0");
    g_wait_ns.store(ns, std::memory_order_relaxed);
    return SPD_OK;
}

SPD_API uint64_t spd_wait_limit_ns(void) { return wait_limit_ns(); }

SPD_API spd_status spd_device_status(uint32_t* out, int32_t clear) {
    if (!out) return fail(SPD_ERR_INVALID_ARG, "out is NULL");
    spd_status st = SPD_OK;
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    unsigned v = 0;
    cudaError_t e = cudaMemcpy(&v, d->status, sizeof v, cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e, "reading the device status");
    *out = v;
    if (clear) {
        e = cudaMemset(d->status, 0, sizeof(unsigned));
        if (e == cudaSuccess) e = cudaDeviceSynchronize();
        if (e != cudaSuccess) return cuda_fail(e, "clearing the device status");
    }
    return SPD_OK;
}

SPD_API size_t spd_score_select_workspace_size(const spd_dims* dims) {
    if (check_dims(dims) != SPD_OK) return 0;
    const long long rows = (long long)dims->B * dims->H_kv;
    return ws_prefix(rows) + (size_t)rows * dims->max_pages_per_seq * sizeof(float);
}

SPD_API size_t spd_sparse_decode_workspace_size(const spd_dims* dims, int32_t k_max, int32_t num_splits) {
    if (check_dims(dims) != SPD_OK) return 0;
    if (k_max < 1) {
        fail(SPD_ERR_INVALID_ARG, "k_max < 1");
        return 0;
    }
    spd_status st = SPD_OK;
    DevInfo* d = dev_info(&st);
    if (!d) return 0;
    const int S = sparse_splits(dims, k_max, num_splits, d->sms);
    const long long rows = (long long)dims->B * dims->H_kv;
    return attn_ws_layout(nullptr, rows, S, dims->H_q / dims->H_kv, dims->D, ws_prefix(rows)).bytes;
}

SPD_API size_t spd_dense_verify_workspace_size(const spd_dims* dims, int32_t T, int32_t num_splits) {
    if (check_dims(dims) != SPD_OK) return 0;
    if (T < 1 || T * (dims->H_q / dims->H_kv) > 64) {
        fail(SPD_ERR_UNSUPPORTED, "T=%d with G=%d (need 1 <= T and T*G <= 64)", T, dims->H_q / dims->H_kv);
        return 0;
    }
    spd_status st = SPD_OK;
    DevInfo* d = dev_info(&st);
    if (!d) return 0;
    const int S = dense_splits(dims, T, num_splits, d->sms);
    const long long rows = (long long)dims->B * dims->H_kv;
    return attn_ws_layout(nullptr, rows, S, T * (dims->H_q / dims->H_kv), dims->D, ws_prefix(rows)).bytes;
}

SPD_API spd_status pages_summarize(const spd_dims* dims, const spd_bf16* K, const int32_t* page_table,
                                   const int32_t* seq_lens, const int32_t* only_pages, int32_t n_only,
                                   spd_bf16* summ, void* stream) {
    spd_status st = check_dims(dims);
    if (st != SPD_OK) return st;
    if (dims->B == 0 || (only_pages && n_only == 0)) return SPD_OK;
    if (!K || !page_table || !seq_lens || !summ) return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (only_pages && n_only < 0) return fail(SPD_ERR_INVALID_ARG, "n_only < 0");
    if (!aligned16(K) || !aligned16(summ)) return fail(SPD_ERR_INVALID_ARG, "K and summ must be 16-byte aligned");
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    SummarizeArgs a;
    a.K = K;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.only_pages = only_pages;
    a.n_only = n_only;
    a.summ = summ;
    a.B = dims->B;
    a.H_kv = dims->H_kv;
    a.D = dims->D;
    a.ps = dims->page_size;
    a.max_pages = dims->max_pages_per_seq;
    a.num_phys = dims->num_phys_pages;
    a.status = d->status;
    cudaError_t e = launch_summarize(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "pages_summarize launch");
}

SPD_API spd_status kv_append_refresh(const spd_dims* dims, int32_t T, spd_bf16* K, spd_bf16* V,
                                     const int32_t* page_table, const int32_t* seq_lens,
                                     const spd_bf16* k_new, const spd_bf16* v_new, spd_bf16* summ,
                                     void* stream) {
    spd_status st = check_dims(dims);
    if (st != SPD_OK) return st;
    if (T < 1 || T > 4096) return fail(SPD_ERR_INVALID_ARG, "T = %d outside [1, 4096]", T);
    if (dims->B == 0) return SPD_OK;
    if (!K || !V || !page_table || !seq_lens || !k_new || !v_new || !summ)
        return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(K) || !aligned16(V) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(summ))
        return fail(SPD_ERR_INVALID_ARG, "K, V, k_new, v_new and summ must be 16-byte aligned");
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    AppendArgs a;
    a.K = K;
    a.V = V;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.k_new = k_new;
    a.v_new = v_new;
    a.summ = summ;
    a.B = dims->B;
    a.T = T;
    a.H_kv = dims->H_kv;
    a.D = dims->D;
    a.ps = dims->page_size;
    a.max_pages = dims->max_pages_per_seq;
    a.num_phys = dims->num_phys_pages;
    a.status = d->status;
    cudaError_t e = launch_append_refresh(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "kv_append_refresh launch");
}

SPD_API spd_status spec_accept(int32_t B, int32_t k, int32_t n_vocab, const float* p_draft,
                               const float* q_target, const int32_t* draft, const float* u_acc,
                               const float* u_res, int32_t* n_accepted, int32_t* tokens, void* stream) {
    if (B < 0) return fail(SPD_ERR_INVALID_ARG, "B < 0");
    if (k < 1 || k > 32) return fail(SPD_ERR_UNSUPPORTED, "k = %d outside [1, 32]", k);
    if (n_vocab < 1 || n_vocab > (1 << 21)) return fail(SPD_ERR_UNSUPPORTED, "n_vocab = %d outside [1, 2^21]", n_vocab);
    if (B == 0) return SPD_OK;
    if (!p_draft || !q_target || !draft || !u_acc || !u_res || !n_accepted || !tokens)
        return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(p_draft) || !aligned16(q_target))
        return fail(SPD_ERR_INVALID_ARG, "p_draft and q_target must be 16-byte aligned");
    spd_status st;
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    SpecArgs a;
    a.p = p_draft;
    a.q = q_target;
    a.draft = draft;
    a.u_acc = u_acc;
    a.u_res = u_res;
    a.n_accepted = n_accepted;
    a.tokens = tokens;
    a.B = B;
    a.k = k;
    a.n = n_vocab;
    a.status = d->status;
    a.wait_ns = wait_limit_ns();
    cudaError_t e = launch_spec_accept(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "spec_accept launch");
}

static spd_status score_select_setup(const spd_dims* dims, const spd_bf16* q, const spd_bf16* summ,
                                     const int32_t* seq_lens, const spd_budget_policy* policy, int32_t* sel,
                                     int32_t* nsel, int32_t k_max, float* scores, void* ws, size_t ws_bytes,
                                     ScoreSelectArgs& a, DevInfo** dev) {
    spd_status st = check_dims(dims);
    if (st != SPD_OK) return st;
    if (!policy) return fail(SPD_ERR_INVALID_ARG, "policy is NULL");
    const spd_budget_policy& p = *policy;
    if (p.mode < 0 || p.mode > 3) return fail(SPD_ERR_INVALID_ARG, "unknown budget mode %d", p.mode);
    if (p.mode == SPD_BUDGET_TOP_P &&
        (!(p.top_p >= 0.f && p.top_p <= 1.f) || !(p.score_scale > 0.f) || !(p.score_scale < 1e30f)))
        return fail(SPD_ERR_INVALID_ARG, "top_p must be in [0, 1] and score_scale > 0 and finite");
    if (p.sink_pages < 0 || p.local_pages < 0) return fail(SPD_ERR_INVALID_ARG, "negative sink/local pages");
    if (p.mode == SPD_BUDGET_FIXED_PAGES && p.fixed_pages < 0) return fail(SPD_ERR_INVALID_ARG, "fixed_pages < 0");
    if (p.mode == SPD_BUDGET_LINEAR_TOKENS && (p.slope_den <= 0 || p.slope_num < 0 || p.min_tokens < 0))
        return fail(SPD_ERR_INVALID_ARG, "bad linear budget parameters");
    if (p.mode == SPD_BUDGET_FRACTION && (p.frac_den <= 0 || p.frac_num < 0))
        return fail(SPD_ERR_INVALID_ARG, "bad fraction budget parameters");
    if (k_max < 1 || (long long)k_max < (long long)p.sink_pages + p.local_pages)
        return fail(SPD_ERR_INVALID_ARG, "k_max (%d) must be >= 1 and >= sink_pages + local_pages", k_max);
    if (dims->max_pages_per_seq > 32768)
        return fail(SPD_ERR_UNSUPPORTED, "max_pages_per_seq %d > 32768", dims->max_pages_per_seq);
    if (dims->B > 16384) return fail(SPD_ERR_UNSUPPORTED, "pages_score_select supports B <= 16384");
    if (dims->B == 0) return SPD_OK;
    if (!q || !summ || !seq_lens || !sel || !nsel)
        return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(q) || !aligned16(summ)) return fail(SPD_ERR_INVALID_ARG, "q and summ must be 16-byte aligned");
    const size_t need = spd_score_select_workspace_size(dims);
    if (!ws || ws_bytes < need) return fail(SPD_ERR_WORKSPACE, "workspace %zu bytes < %zu", ws_bytes, need);
    if (!aligned16(ws)) return fail(SPD_ERR_INVALID_ARG, "ws must be 16-byte aligned");
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    a = ScoreSelectArgs{};
    a.q = q;
    a.summ = summ;
    a.seq_lens = seq_lens;
    a.pol = p;
    a.sel = sel;
    a.nsel = nsel;
    a.k_max = k_max;
    a.scores = scores ? scores : reinterpret_cast<float*>(static_cast<char*>(ws) + ws_prefix((long long)dims->B * dims->H_kv));
    a.B = dims->B;
    a.H_q = dims->H_q;
    a.H_kv = dims->H_kv;
    a.D = dims->D;
    a.ps = dims->page_size;
    a.max_pages = dims->max_pages_per_seq;
    a.num_phys = dims->num_phys_pages;
    a.status = d->status;
    a.wait_ns = wait_limit_ns();
    *dev = d;
    return SPD_OK;
}

SPD_API spd_status pages_score_select(const spd_dims* dims, const spd_bf16* q, const spd_bf16* summ,
                                      const int32_t* seq_lens,
                                      const spd_budget_policy* policy, int32_t* sel, int32_t* nsel, int32_t k_max,
                                      float* scores, void* ws, size_t ws_bytes, void* stream) {
    ScoreSelectArgs a;
    DevInfo* d = nullptr;
    spd_status st = score_select_setup(dims, q, summ, seq_lens, policy, sel, nsel, k_max, scores, ws, ws_bytes, a, &d);
    if (st != SPD_OK || dims->B == 0) return st;
    cudaError_t e = launch_score_select(a, d->sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "pages_score_select launch");
}

SPD_API spd_status pages_append_score_select(const spd_dims* dims, spd_bf16* K, spd_bf16* V,
                                             const int32_t* page_table, const int32_t* seq_lens,
                                             const spd_bf16* k_new, const spd_bf16* v_new, const spd_bf16* q,
                                             spd_bf16* summ, const spd_budget_policy* policy, int32_t* sel,
                                             int32_t* nsel, int32_t k_max, float* scores, void* ws,
                                             size_t ws_bytes, void* stream) {
    ScoreSelectArgs a;
    DevInfo* d = nullptr;
    spd_status st = score_select_setup(dims, q, summ, seq_lens, policy, sel, nsel, k_max, scores, ws, ws_bytes, a, &d);
    if (st != SPD_OK || dims->B == 0) return st;
    if (!K || !V || !page_table || !k_new || !v_new) return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(K) || !aligned16(V) || !aligned16(k_new) || !aligned16(v_new))
        return fail(SPD_ERR_INVALID_ARG, "K, V, k_new and v_new must be 16-byte aligned");
    a.K = K;
    a.V = V;
    a.page_table = page_table;
    a.k_new = k_new;
    a.v_new = v_new;
    a.summ_w = summ;
    cudaError_t e = launch_score_select(a, d->sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "pages_append_score_select launch");
}

static spd_status attn_common(const spd_dims* dims, const spd_bf16* q, const spd_bf16* K, const spd_bf16* V,
                              const int32_t* page_table, const int32_t* seq_lens, spd_bf16* o) {
    if (!q || !K || !V || !page_table || !seq_lens || !o) return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(q) || !aligned16(K) || !aligned16(V) || !aligned16(o))
        return fail(SPD_ERR_INVALID_ARG, "q, K, V and o must be 16-byte aligned");
    if (dims->num_phys_pages < 1) return fail(SPD_ERR_INVALID_ARG, "num_phys_pages < 1");
    return SPD_OK;
}

// Validates and launches the sparse attention kernel with S units per row (S >= 1
// already chosen) and `prefix` bytes for the queue and the tickets; sel_done != NULL chains
// it behind the selection of each row.
static spd_status sparse_attn_launch(const spd_dims* dims, const spd_bf16* q, const spd_bf16* K, const spd_bf16* V,
                                     const int32_t* page_table, const int32_t* seq_lens, const int32_t* sel,
                                     const int32_t* nsel, int32_t k_max, int S, float softmax_scale, spd_bf16* o,
                                     float* lse, void* ws, size_t ws_bytes, size_t prefix, unsigned* sel_done,
                                     const int32_t* sel_phys, DevInfo* d, void* stream) {
    spd_status st;
    const int G = dims->H_q / dims->H_kv;
    const long long rows = (long long)dims->B * dims->H_kv;
    AttnWs w = attn_ws_layout(ws, rows, S, G, dims->D, prefix);
    const size_t need = attn_ws_needed(rows, S, G, dims->D, prefix);
    if (!ws || ws_bytes < need) return fail(SPD_ERR_WORKSPACE, "workspace %zu bytes < %zu", ws_bytes, need);
    if (!aligned16(ws)) return fail(SPD_ERR_INVALID_ARG, "ws must be 16-byte aligned");
    CUtensorMap tk, tv;
    if ((st = kv_map(&tk, K, dims)) != SPD_OK || (st = kv_map(&tv, V, dims)) != SPD_OK) return st;
    AttnArgs a{};
    a.q = q;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.sel = sel;
    a.nsel = nsel;
    a.k_max = k_max;
    a.B = dims->B;
    a.H_q = dims->H_q;
    a.H_kv = dims->H_kv;
    a.D = dims->D;
    a.ps = dims->page_size;
    a.max_pages = dims->max_pages_per_seq;
    a.T = 1;
    a.num_phys = dims->num_phys_pages;
    a.items_per_split = (k_max + S - 1) / S;
    a.num_splits = S;
    a.scale_log2 = softmax_scale * kLog2e;
    a.o = o;
    a.lse = lse;
    a.part_o = w.part_o;
    a.part_lse = w.part_lse;
    a.counters = w.counters;
    a.queue = w.queue;
    a.num_sms = d->sms;
    a.status = d->status;
    a.wait_ns = wait_limit_ns();
    a.sel_done = sel_done;
    a.sel_phys = sel_phys;
    cudaError_t e = launch_sparse_attn(a, tk, tv, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "sparse attention launch");
}

SPD_API spd_status sparse_decode_attn(const spd_dims* dims, const spd_bf16* q, const spd_bf16* K,
                                      const spd_bf16* V, const int32_t* page_table, const int32_t* seq_lens,
                                      const int32_t* sel, const int32_t* nsel, int32_t k_max, int32_t num_splits,
                                      float softmax_scale, spd_bf16* o, float* lse, void* ws, size_t ws_bytes,
                                      void* stream) {
    spd_status st = check_dims(dims);
    if (st != SPD_OK) return st;
    if (k_max < 1) return fail(SPD_ERR_INVALID_ARG, "k_max < 1");
    if (num_splits < 0) return fail(SPD_ERR_INVALID_ARG, "num_splits < 0");
    if (dims->B == 0) return SPD_OK;
    if ((st = attn_common(dims, q, K, V, page_table, seq_lens, o)) != SPD_OK) return st;
    if (!sel || !nsel) return fail(SPD_ERR_INVALID_ARG, "NULL selection");
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    return sparse_attn_launch(dims, q, K, V, page_table, seq_lens, sel, nsel, k_max,
                              sparse_splits(dims, k_max, num_splits, d->sms), softmax_scale, o, lse, ws, ws_bytes,
                              ws_prefix((long long)dims->B * dims->H_kv), nullptr, nullptr, d, stream);
}

// The chained step's workspace: [score / select][chain: two tile counters, warps
// done, selection claims, tiles_done[rows], sel_done[rows], (256-aligned) keys[rows][max_pages],
// (256-aligned) sel_phys[rows][k_max]][attention].
struct StepWs {
    size_t score, chain, keys, phys, attn, bytes;
};

// The chained selection also writes each selected page's physical page (from a copy
// of the row's page table in shared memory) when that copy fits comfortably.
static bool step_sel_phys(const spd_dims* dims, const spd_budget_policy* policy) {
    const size_t words = ((size_t)dims->max_pages_per_seq + 31) / 32;
    const size_t per = (policy && policy->mode == SPD_BUDGET_TOP_P) ? 3 : 2;
    return ((size_t)dims->max_pages_per_seq * per + 2 * words) * sizeof(uint32_t) <= 96 * 1024;
}

static bool step_ws_layout(const spd_dims* dims, int32_t k_max, StepWs* w, DevInfo* d) {
    const long long rows = (long long)dims->B * dims->H_kv;
    const int S = sparse_splits(dims, k_max, 0, d->sms);
    w->score = align256(spd_score_select_workspace_size(dims));
    w->keys = align256(32 + 2 * (size_t)rows * sizeof(unsigned));  // offset of the keys in the chain part
    w->phys = w->keys + align256((size_t)rows * dims->max_pages_per_seq * sizeof(unsigned));
    w->chain = w->phys + align256((size_t)rows * k_max * sizeof(int32_t));
    w->attn = attn_ws_layout(nullptr, rows, S, dims->H_q / dims->H_kv, dims->D, ticket_bytes(rows)).bytes;
    w->bytes = w->score + w->chain + w->attn;
    return w->score != 0;
}

SPD_API size_t spd_sparse_decode_step_workspace_size(const spd_dims* dims, int32_t k_max) {
    if (check_dims(dims) != SPD_OK) return 0;
    if (k_max < 1) {
        fail(SPD_ERR_INVALID_ARG, "k_max < 1");
        return 0;
    }
    spd_status st = SPD_OK;
    DevInfo* d = dev_info(&st);
    if (!d) return 0;
    StepWs w;
    return step_ws_layout(dims, k_max, &w, d) ? w.bytes : 0;
}

SPD_API spd_status sparse_decode_step(const spd_dims* dims, spd_bf16* K, spd_bf16* V, const int32_t* page_table,
                                      const int32_t* seq_lens, const spd_bf16* k_new, const spd_bf16* v_new,
                                      const spd_bf16* q, spd_bf16* summ, const spd_budget_policy* policy,
                                      int32_t* sel, int32_t* nsel, int32_t k_max, float softmax_scale,
                                      spd_bf16* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
    spd_status st = check_dims(dims);
    if (st != SPD_OK) return st;
    if (k_max < 1) return fail(SPD_ERR_INVALID_ARG, "k_max < 1");
    if (dims->B == 0) return SPD_OK;
    if ((k_new == nullptr) != (v_new == nullptr)) return fail(SPD_ERR_INVALID_ARG, "k_new and v_new: both or neither");
    if ((st = attn_common(dims, q, K, V, page_table, seq_lens, o)) != SPD_OK) return st;
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    StepWs w;
    if (!step_ws_layout(dims, k_max, &w, d)) return fail(SPD_ERR_INVALID_ARG, "bad dims");
    if (!ws || ws_bytes < w.bytes) return fail(SPD_ERR_WORKSPACE, "workspace %zu bytes < %zu", ws_bytes, w.bytes);
    if (!aligned16(ws)) return fail(SPD_ERR_INVALID_ARG, "ws must be 16-byte aligned");
    char* base = static_cast<char*>(ws);
    ScoreSelectArgs a;
    DevInfo* d2 = nullptr;
    st = score_select_setup(dims, q, summ, seq_lens, policy, sel, nsel, k_max, nullptr, base, w.score, a, &d2);
    if (st != SPD_OK) return st;
    if (k_new) {
        if (!aligned16(k_new) || !aligned16(v_new)) return fail(SPD_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
        a.K = K;
        a.V = V;
        a.page_table = page_table;
        a.k_new = k_new;
        a.v_new = v_new;
        a.summ_w = summ;
    }
    // Chained row by row: the selection of a row starts as soon as its tiles are
    // scored, and each of its attention units as soon as it is selected.
    const int S = sparse_splits(dims, k_max, 0, d->sms);
    char* chain = base + w.score;
    const long long rows = (long long)dims->B * dims->H_kv;
    a.tile_ctr = reinterpret_cast<unsigned long long*>(chain);
    a.warps_done = reinterpret_cast<unsigned*>(chain + 16);
    a.sel_claims = reinterpret_cast<unsigned*>(chain + 20);
    a.tiles_done = reinterpret_cast<unsigned*>(chain + 32);
    a.sel_done = a.tiles_done + rows;
    a.keys = reinterpret_cast<unsigned*>(chain + w.keys);
    if (step_sel_phys(dims, policy)) {
        a.page_table = page_table;
        a.sel_phys = reinterpret_cast<int32_t*>(chain + w.phys);
    }
    unsigned* sel_done = a.sel_done;
    cudaError_t e = launch_score_select(a, d->sms, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "sparse_decode_step scoring launch");
    return sparse_attn_launch(dims, q, K, V, page_table, seq_lens, sel, nsel, k_max, S, softmax_scale, o, lse,
                              base + w.score + w.chain, w.attn, ticket_bytes(rows), sel_done, a.sel_phys, d, stream);
}

SPD_API spd_status dense_verify_attn(const spd_dims* dims, int32_t T, const spd_bf16* q, const spd_bf16* K,
                                     const spd_bf16* V, const int32_t* page_table, const int32_t* seq_lens,
                                     int32_t num_splits, float softmax_scale, spd_bf16* o, float* lse, void* ws,
                                     size_t ws_bytes, void* stream) {
    spd_status st = check_dims(dims);
    if (st != SPD_OK) return st;
    const int G = dims->H_q / dims->H_kv;
    if (T < 1 || T * G > 64) return fail(SPD_ERR_UNSUPPORTED, "T=%d with G=%d (need 1 <= T and T*G <= 64)", T, G);
    if (num_splits < 0) return fail(SPD_ERR_INVALID_ARG, "num_splits < 0");
    if (dims->B == 0) return SPD_OK;
    if ((st = attn_common(dims, q, K, V, page_table, seq_lens, o)) != SPD_OK) return st;
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    const int S = dense_splits(dims, T, num_splits, d->sms);
    const long long rows = (long long)dims->B * dims->H_kv;
    AttnWs w = attn_ws_layout(ws, rows, S, T * G, dims->D, ws_prefix(rows));
    if (!ws || ws_bytes < w.bytes) return fail(SPD_ERR_WORKSPACE, "workspace %zu bytes < %zu", ws_bytes, w.bytes);
    if (!aligned16(ws)) return fail(SPD_ERR_INVALID_ARG, "ws must be 16-byte aligned");
    CUtensorMap tk, tv;
    if ((st = kv_map(&tk, K, dims)) != SPD_OK || (st = kv_map(&tv, V, dims)) != SPD_OK) return st;
    AttnArgs a{};
    a.q = q;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.sel = nullptr;
    a.nsel = nullptr;
    a.k_max = 0;
    a.B = dims->B;
    a.H_q = dims->H_q;
    a.H_kv = dims->H_kv;
    a.D = dims->D;
    a.ps = dims->page_size;
    a.max_pages = dims->max_pages_per_seq;
    a.T = T;
    a.num_phys = dims->num_phys_pages;
    a.items_per_split = (dims->max_pages_per_seq + S - 1) / S;
    a.num_splits = S;
    a.scale_log2 = softmax_scale * kLog2e;
    a.o = o;
    a.lse = lse;
    a.part_o = w.part_o;
    a.part_lse = w.part_lse;
    a.counters = w.counters;
    a.queue = w.queue;
    a.num_sms = d->sms;
    a.status = d->status;
    a.wait_ns = wait_limit_ns();
    cudaError_t e = launch_dense_attn(a, tk, tv, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "dense_verify_attn launch");
}

SPD_API spd_status lse_merge(int32_t S, int32_t rows, int32_t D, const float* part_o, const float* part_lse,
                             spd_bf16* o, float* lse, void* stream) {
    if (S < 1 || rows < 0) return fail(SPD_ERR_INVALID_ARG, "bad S (%d) or rows (%d)", S, rows);
    if (D != 64 && D != 128) return fail(SPD_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", D);
    if (rows == 0) return SPD_OK;
    if (!part_o || !part_lse || !o) return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    cudaError_t e = launch_lse_merge(S, rows, D, part_o, part_lse, o, lse, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "lse_merge launch");
}

// ---------------------------------------------------------------------------
// sparse_decode_attn_noalloc: the same launch with its scratch in a fixed
// device array instead of a caller workspace (see include/spd.h).

namespace spd {
namespace {

__device__ __align__(256) unsigned char g_noalloc_scratch[SPD_NOALLOC_SCRATCH_BYTES];

struct NoAllocDev {
    std::once_flag once;
    void* ptr = nullptr;
    cudaError_t err = cudaSuccess;
};
NoAllocDev g_noalloc[kMaxDevices];

// Device address of the fixed scratch array for the current device (looked up
// once per device; in host code the array's name is only a host-side handle).
void* noalloc_scratch(spd_status* st) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) {
        *st = cuda_fail(e, "cudaGetDevice");
        return nullptr;
    }
    if (dev < 0 || dev >= kMaxDevices) {
        *st = fail(SPD_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
        return nullptr;
    }
    NoAllocDev* n = &g_noalloc[dev];
    std::call_once(n->once, [n]() { n->err = cudaGetSymbolAddress(&n->ptr, g_noalloc_scratch); });
    if (n->err != cudaSuccess || !n->ptr) {
        *st = cuda_fail(n->err, "looking up the fixed scratch array");
        return nullptr;
    }
    return n->ptr;
}

}  // namespace
}  // namespace spd

SPD_API spd_status sparse_decode_attn_noalloc(const spd_dims* dims, const spd_bf16* q, const spd_bf16* K,
                                              const spd_bf16* V, const int32_t* page_table, const int32_t* seq_lens,
                                              const int32_t* sel, const int32_t* nsel, int32_t k_max,
                                              int32_t num_splits, float softmax_scale, spd_bf16* o, float* lse,
                                              void* stream) {
    spd_status st = check_dims(dims);
    if (st != SPD_OK) return st;
    if (k_max < 1) return fail(SPD_ERR_INVALID_ARG, "k_max < 1");
    if (num_splits < 0) return fail(SPD_ERR_INVALID_ARG, "num_splits < 0");
    if (dims->B == 0) return SPD_OK;
    if ((st = attn_common(dims, q, K, V, page_table, seq_lens, o)) != SPD_OK) return st;
    if (!sel || !nsel) return fail(SPD_ERR_INVALID_ARG, "NULL selection");
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    void* scratch = noalloc_scratch(&st);
    if (!scratch) return st;
    const int G = dims->H_q / dims->H_kv;
    const long long rows = (long long)dims->B * dims->H_kv;
    const size_t prefix = ticket_bytes(rows);
    int S = sparse_splits(dims, k_max, num_splits, d->sms);
    if (num_splits == 0) {
        // automatic: the usual split count, or fewer until the partials fit
        while (S > 1 && attn_ws_needed(rows, S, G, dims->D, prefix) > SPD_NOALLOC_SCRATCH_BYTES)
            S = sparse_splits(dims, k_max, S - 1, d->sms);
    }
    const size_t need = attn_ws_needed(rows, S, G, dims->D, prefix);
    if (need > SPD_NOALLOC_SCRATCH_BYTES)
        return fail(SPD_ERR_UNSUPPORTED,
                    "sparse_decode_attn_noalloc needs %zu bytes of scratch for %d split(s); the fixed array holds %zu",
                    need, S, (size_t)SPD_NOALLOC_SCRATCH_BYTES);
    // the queue and the split tickets must start at zero
    cudaError_t e = cudaMemsetAsync(scratch, 0, prefix, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "clearing the fixed scratch array");
    return sparse_attn_launch(dims, q, K, V, page_table, seq_lens, sel, nsel, k_max, S, softmax_scale, o, lse,
                              scratch, SPD_NOALLOC_SCRATCH_BYTES, prefix, nullptr, nullptr, d, stream);
}

// ---------------------------------------------------------------- head norms and rotation

// Checks a rotation's description and fills the kernel's arguments from it.
static spd_status rope_setup(const spd_rope* rope, int32_t D, int32_t H_q, int32_t H_kv, const spd_bf16* q,
                             int64_t q_stride, const spd_bf16* k, int64_t k_stride, RopeArgs& a) {
    if (!rope) return fail(SPD_ERR_INVALID_ARG, "rope is NULL");
    if (D != 64 && D != 128) return fail(SPD_ERR_UNSUPPORTED, "head dim %d (supported: 64, 128)", D);
    if (rope->rot_dim < 0 || rope->rot_dim > D || rope->rot_dim % 8)
        return fail(SPD_ERR_UNSUPPORTED, "rot_dim %d (need a multiple of 8 in [0, %d])", rope->rot_dim, D);
    if (!(rope->eps >= 0.f) || !(rope->eps <= 3.4e38f)) return fail(SPD_ERR_INVALID_ARG, "eps must be >= 0 and finite");
    if (rope->rot_dim > 0 && (!rope->table || rope->n_pos < 1 || !aligned16(rope->table)))
        return fail(SPD_ERR_INVALID_ARG, "the angle table must be 16-byte aligned and hold at least one position");
    if ((reinterpret_cast<uintptr_t>(rope->q_weight) | reinterpret_cast<uintptr_t>(rope->k_weight)) & 7u)
        return fail(SPD_ERR_INVALID_ARG, "norm weights must be 8-byte aligned");
    if ((q && (H_q < 1 || q_stride < (int64_t)H_q * D || q_stride % 8)) ||
        (k && (H_kv < 1 || k_stride < (int64_t)H_kv * D || k_stride % 8)))
        return fail(SPD_ERR_INVALID_ARG, "bad heads or row strides (H_q=%d q_stride=%lld H_kv=%d k_stride=%lld)", H_q,
                    (long long)q_stride, H_kv, (long long)k_stride);
    a = RopeArgs{};
    a.q = q;
    a.k = k;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.H_q = q ? H_q : 0;
    a.H_kv = k ? H_kv : 0;
    a.D = D;
    a.table = rope->table;
    a.n_pos = rope->n_pos;
    a.rot = rope->rot_dim;
    a.interleaved = rope->interleaved != 0;
    a.q_weight = q ? rope->q_weight : nullptr;
    a.k_weight = k ? rope->k_weight : nullptr;
    a.eps = rope->eps;
    return SPD_OK;
}

SPD_API spd_status qk_norm_rope(int64_t rows, int32_t H_q, int32_t H_kv, int32_t D, const spd_rope* rope,
                                const spd_bf16* q, int64_t q_stride, const spd_bf16* k, int64_t k_stride,
                                const int32_t* positions, spd_bf16* q_out, spd_bf16* k_out, void* stream) {
    RopeArgs a;
    spd_status st = rope_setup(rope, D, H_q, H_kv, q, q_stride, k, k_stride, a);
    if (st != SPD_OK) return st;
    if (rows < 0) return fail(SPD_ERR_INVALID_ARG, "rows < 0");
    if (rows == 0 || (!q && !k)) return SPD_OK;
    if ((q && !q_out) || (k && !k_out) || (a.rot > 0 && !positions))
        return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out))
        return fail(SPD_ERR_INVALID_ARG, "q, k, q_out and k_out must be 16-byte aligned");
    if (rows >= (1LL << 31) || a.H_q > 65536 || a.H_kv > 65536)
        return fail(SPD_ERR_UNSUPPORTED, "too many rows or heads (rows=%lld H_q=%d H_kv=%d)", (long long)rows, a.H_q, a.H_kv);
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    a.rows = rows;
    a.positions = positions;
    a.q_out = q_out;
    a.k_out = k_out;
    a.status = d->status;
    cudaError_t e = launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "qk_norm_rope launch");
}

SPD_API spd_status kv_append_rope(const spd_dims* dims, int32_t T, const spd_rope* rope, spd_bf16* K, spd_bf16* V,
                                  const int32_t* page_table, const int32_t* seq_lens, const spd_bf16* q,
                                  int64_t q_stride, const spd_bf16* k, int64_t k_stride, const spd_bf16* v,
                                  int64_t v_stride, spd_bf16* q_out, spd_bf16* summ, void* stream) {
    spd_status st = check_dims(dims);
    if (st != SPD_OK) return st;
    if (T < 1 || T > 4096) return fail(SPD_ERR_INVALID_ARG, "T = %d outside [1, 4096]", T);
    AppendRopeArgs p;
    st = rope_setup(rope, dims->D, dims->H_q, dims->H_kv, q, q_stride, k, k_stride, p.rope);
    if (st != SPD_OK) return st;
    if (dims->B == 0) return SPD_OK;
    if (!K || !V || !page_table || !seq_lens || !k || !v || !summ || (q != nullptr) != (q_out != nullptr))
        return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument (q and q_out go together)");
    if (v_stride < (int64_t)dims->H_kv * dims->D || v_stride % 8)
        return fail(SPD_ERR_INVALID_ARG, "bad v_stride %lld", (long long)v_stride);
    if (!aligned16(K) || !aligned16(V) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) ||
        !aligned16(summ))
        return fail(SPD_ERR_INVALID_ARG, "K, V, q, k, v, q_out and summ must be 16-byte aligned");
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    AppendArgs& a = p.append;
    a = AppendArgs{};
    a.K = K;
    a.V = V;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.summ = summ;
    a.B = dims->B;
    a.T = T;
    a.H_kv = dims->H_kv;
    a.D = dims->D;
    a.ps = dims->page_size;
    a.max_pages = dims->max_pages_per_seq;
    a.num_phys = dims->num_phys_pages;
    a.status = d->status;
    p.rope.rows = (long long)dims->B * T;
    p.rope.q_out = q_out;
    p.rope.status = d->status;
    p.v = v;
    p.v_stride = v_stride;
    p.touched = 0;
    if (append_rope_ctas(p) >= (1LL << 28) || p.rope.rows >= (1LL << 31)) return fail(SPD_ERR_UNSUPPORTED, "B * T * H_q too large");
    cudaError_t e = launch_append_rope(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "kv_append_rope launch");
}

// ---------------------------------------------------------------- the 4-bit cache

static spd_status kv4_exps(int32_t k_exp, int32_t v_exp) {
    if (k_exp < -64 || k_exp > 64 || v_exp < -64 || v_exp > 64)
        return fail(SPD_ERR_INVALID_ARG, "k_exp (%d) and v_exp (%d) must lie in [-64, 64]", k_exp, v_exp);
    return SPD_OK;
}

static spd_status kv4_rows_setup(const spd_dims* dims, int32_t T, const uint8_t* kv4, int32_t k_exp, int32_t v_exp,
                                 const int32_t* page_table, const int32_t* seq_lens, const void* k, const void* v,
                                 Kv4Args& a) {
    spd_status st = check_dims(dims);
    if (st != SPD_OK) return st;
    if (T < 1 || T > 4096) return fail(SPD_ERR_INVALID_ARG, "T = %d outside [1, 4096]", T);
    st = kv4_exps(k_exp, v_exp);
    if (st != SPD_OK || dims->B == 0) return st;
    if (!kv4 || !page_table || !seq_lens || !k || !v) return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(kv4) || !aligned16(k) || !aligned16(v))
        return fail(SPD_ERR_INVALID_ARG, "the cache and the rows must be 16-byte aligned");
    if ((long long)dims->B * T * dims->H_kv >= (1LL << 31)) return fail(SPD_ERR_UNSUPPORTED, "B * T * H_kv must be < 2^31");
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    a = Kv4Args{};
    a.kv4 = const_cast<uint8_t*>(kv4);
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.B = dims->B;
    a.T = T;
    a.H_kv = dims->H_kv;
    a.D = dims->D;
    a.ps = dims->page_size;
    a.max_pages = dims->max_pages_per_seq;
    a.num_phys = dims->num_phys_pages;
    a.k_exp = k_exp;
    a.v_exp = v_exp;
    a.status = d->status;
    return SPD_OK;
}

SPD_API spd_status kv4_append(const spd_dims* dims, int32_t T, uint8_t* kv4, int32_t k_exp, int32_t v_exp,
                              const int32_t* page_table, const int32_t* seq_lens, const spd_bf16* k_new,
                              const spd_bf16* v_new, spd_bf16* summ, void* stream) {
    Kv4Args a;
    spd_status st = kv4_rows_setup(dims, T, kv4, k_exp, v_exp, page_table, seq_lens, k_new, v_new, a);
    if (st != SPD_OK || dims->B == 0) return st;
    if (!summ || !aligned16(summ)) return fail(SPD_ERR_INVALID_ARG, "summ must be 16-byte aligned and not NULL");
    a.k_new = k_new;
    a.v_new = v_new;
    a.summ = summ;
    cudaError_t e = launch_kv4_append(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "kv4_append launch");
}

SPD_API spd_status kv4_read(const spd_dims* dims, int32_t T, const uint8_t* kv4, int32_t k_exp, int32_t v_exp,
                            const int32_t* page_table, const int32_t* seq_lens, spd_bf16* k_out, spd_bf16* v_out,
                            void* stream) {
    Kv4Args a;
    spd_status st = kv4_rows_setup(dims, T, kv4, k_exp, v_exp, page_table, seq_lens, k_out, v_out, a);
    if (st != SPD_OK || dims->B == 0) return st;
    a.k_out = k_out;
    a.v_out = v_out;
    cudaError_t e = launch_kv4_read(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "kv4_read launch");
}

// Splits of a row of the 4-bit attention.  Its CTAs take one unit each, `slots` at a time, in
// turns of 128 tokens, and a unit costs about `fixed` turns besides its own (the lengths, the
// queries, the first copies, the join).  Up to half a GPU of rows is cut into one round of
// units, or, with more than eight query rows, into fewer where the join would take longer (one KV
// head, 64 query rows, 131,000 / 20,000 tokens: 304 / 157 units 95.6 / 68.0 us, 161 / 46 units 79.6 /
// 49.3 us).  More rows, selections (about equal): the count that takes the least rounds *
// (turns + fixed).  More rows, whole sequences (their lengths differ, and only the GPU knows
// them): units + the longest one's tail, rows * S * (turns / S + fixed) / slots + turns / S, is
// least at S = sqrt(turns * slots / (rows * fixed)).  Measured: 64 sequences of 8K-16K tokens, 8 KV heads,
// 28 query rows: S = 1 / 2 / 3 / 4 / 8: 344 / 337 / 333 / 342 / 377 us (3 taken); 40 of
// 2K-6K, 64 query rows: 1 / 2 / 3: 136 / 150 / 159 us (1 taken); 64 selections of 64
// pages of 16: 1 / 2 / 4: 23 / 32 / 40 us (1 taken); one sequence of 131,072 tokens, 8 KV heads: 25 / 38 / 44 / 57 /
// 76 / 90: 57 / 42 / 55 / 46 / 40 / 52 us (76 taken: 38, 57 and 76 are two, three and four units on each of 152 SMs,
// the counts between them leave some SMs one unit more than others, and 90 takes a second round); 8 selections of
// 256 pages of 32: 4 / 7 / 9 / 14: 29 / 30 / 26 / 33 us (9 taken).
// A dense row's units are planned by the page table's width, since only the GPU knows the length; in a table
// much wider than the sequence fewer of them have work (one of 2,048 / 16,384 / 65,536 tokens in a table for 131,072
// against one of its own width: 19 / 26 / 37 us against 8 / 17 / 27).
constexpr long long kJoinBytes = 256 << 10;

static int kv4_splits(const spd_dims* d, int T, int items, bool sparse, int req, int sms) {
    const long long rows = (long long)d->B * d->H_kv;
    if (rows > kTickets) return 1;  // many times the rows that fill the GPU
    const int R = T * (d->H_q / d->H_kv);
    const bool few = R <= kAttn4DecodeRows;
    const double fixed = few ? 6 : R <= 32 ? 10 : 20;
    const long long slots = (long long)sms * (few ? occ_attn4_decode() : occ_attn4_verify());
    int S = req;
    if (S <= 0) {
        S = 1;
        const int floor_items = 128 / d->page_size;
        const int most = (items + floor_items - 1) / floor_items;
        const double turns = (double)items * d->page_size / 128;
        if (rows > 0 && 2 * rows <= slots) {
            S = (int)(slots / rows);
            if (!few) {
                // turns / S * 1.3 us + 2 sqrt(S) partials of the join at 50 GB/s
                const double part = (double)R * d->D * 4 / 50e3;
                const int least = (int)cbrt(turns * 1.3 / part * (turns * 1.3 / part)) + 1;
                if (S > least) S = least;
            }
        } else if (rows > 0 && !sparse) {
            S = (int)(sqrt(turns * slots / (rows * fixed)) + 0.5);
        } else if (rows > 0) {
            double best = 1e300;
            for (int s = 1; s <= 16 && s <= most; ++s) {
                const double cost = (double)((rows * s + slots - 1) / slots) * (turns / s + fixed);
                if (cost < best) {
                    best = cost;
                    S = s;
                }
            }
        }
        if (S > most) S = most;
    }
    if (S > items) S = items;
    if (S < 1) S = 1;
    const int ips = (items + S - 1) / S;
    return (items + ips - 1) / ips;
}

// Groups of splits that are joined first.  One CTA reads a row's partials at ~50 GB/s, so the join
// of many splits of many query rows goes in two steps of about sqrt(S) partials where they
// are more than 256 KB.  One sequence of 131,000 tokens, one KV head, 64 / 24 / 8 query rows:
// 232 / 92 / 77 us in one step, 96 / 46 / 22 in two (304 splits each); 8 KV heads of 4 rows (156 KB): 39.0 in one, 38.2
// to 40.1 in two.
struct Kv4Groups {
    int group, groups;  // splits of a group; groups of a row (0: no groups)
};
static Kv4Groups kv4_groups(long long rows, int S, int R, int D) {
    Kv4Groups g = {S, 0};
    if ((long long)S * R * D * 4 <= kJoinBytes) return g;
    const int group = (int)ceil(sqrt((double)S)), groups = (S + group - 1) / group;
    if (rows * (1 + groups) > kTickets) return g;
    g.group = group;
    g.groups = groups;
    return g;
}

// The workspace: tickets at its start, the rows' where the bf16 attention's are and the groups'
// behind them, within the place that no call's scores or partials reach (ws_prefix).
static AttnWs kv4_ws_layout(void* ws, long long rows, int S, int R, int D) {
    S += kv4_groups(rows, S, R, D).groups;
    AttnWs w;
    char* base = static_cast<char*>(ws);
    w.queue = nullptr;
    w.counters = reinterpret_cast<int*>(base + 16);
    size_t off = kTicketBytes;
    w.part_lse = reinterpret_cast<float*>(base + off);
    if (S > 1) off += align256((size_t)rows * S * R * sizeof(float));
    w.part_o = reinterpret_cast<float*>(base + off);
    if (S > 1) off += (size_t)rows * S * R * D * sizeof(float);
    w.bytes = off;
    return w;
}

static size_t kv4_attn_ws(const spd_dims* dims, int T, int items, bool sparse, int32_t num_splits) {
    spd_status st = SPD_OK;
    DevInfo* d = dev_info(&st);
    if (!d) return 0;
    const int S = kv4_splits(dims, T, items, sparse, num_splits, d->sms);
    return kv4_ws_layout(nullptr, (long long)dims->B * dims->H_kv, S, T * (dims->H_q / dims->H_kv), dims->D).bytes;
}

static spd_status kv4_check_T(const spd_dims* dims, int32_t T) {
    if (T < 1 || (long long)T * (dims->H_q / dims->H_kv) > 64)
        return fail(SPD_ERR_UNSUPPORTED, "T=%d with G=%d (need 1 <= T and T*G <= 64)", T, dims->H_q / dims->H_kv);
    return SPD_OK;
}

SPD_API size_t spd_kv4_sparse_decode_workspace_size(const spd_dims* dims, int32_t k_max, int32_t num_splits) {
    if (check_dims(dims) != SPD_OK) return 0;
    if (k_max < 1) {
        fail(SPD_ERR_INVALID_ARG, "k_max < 1");
        return 0;
    }
    return kv4_attn_ws(dims, 1, k_max, true, num_splits);
}

SPD_API size_t spd_kv4_dense_verify_workspace_size(const spd_dims* dims, int32_t T, int32_t num_splits) {
    if (check_dims(dims) != SPD_OK || kv4_check_T(dims, T) != SPD_OK) return 0;
    return kv4_attn_ws(dims, T, dims->max_pages_per_seq, false, num_splits);
}

// The common body of the two calls (sel NULL: dense).  dims and T are checked.
static spd_status kv4_attn(const spd_dims* dims, int32_t T, const spd_bf16* q, const uint8_t* kv4, int32_t k_exp,
                           int32_t v_exp, const int32_t* page_table, const int32_t* seq_lens, const int32_t* sel,
                           const int32_t* nsel, int32_t items, int32_t num_splits, float scale, spd_bf16* o,
                           float* lse, void* ws, size_t ws_bytes, void* stream) {
    const bool sparse = sel != nullptr;
    spd_status st = kv4_exps(k_exp, v_exp);
    if (st != SPD_OK) return st;
    const double scale_log2 = (double)scale * 1.4426950408889634 * (double)exp2f((float)k_exp);
    if (!(scale_log2 >= -3.4e38 && scale_log2 <= 3.4e38))
        return fail(SPD_ERR_INVALID_ARG, "softmax_scale (times 2^k_exp) is not finite in 32 bits");
    if (num_splits < 0) return fail(SPD_ERR_INVALID_ARG, "num_splits < 0");
    if (!q || !kv4 || !page_table || !seq_lens || !o) return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(q) || !aligned16(kv4) || !aligned16(o))
        return fail(SPD_ERR_INVALID_ARG, "q, kv4 and o must be 16-byte aligned");
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    const int R = T * (dims->H_q / dims->H_kv);
    const int S = kv4_splits(dims, T, items, sparse, num_splits, d->sms);
    const long long rows = (long long)dims->B * dims->H_kv;
    if (rows * S >= (1LL << 31)) return fail(SPD_ERR_UNSUPPORTED, "B * H_kv * num_splits must be < 2^31");
    const AttnWs w = kv4_ws_layout(ws, rows, S, R, dims->D);
    if (!ws || ws_bytes < w.bytes) return fail(SPD_ERR_WORKSPACE, "workspace %zu bytes < %zu", ws_bytes, w.bytes);
    if (!aligned16(ws)) return fail(SPD_ERR_INVALID_ARG, "ws must be 16-byte aligned");
    Attn4Args a = {};
    a.q = q;
    a.kv4 = kv4;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.sel = sel;
    a.nsel = nsel;
    a.k_max = items;
    a.B = dims->B;
    a.H_q = dims->H_q;
    a.H_kv = dims->H_kv;
    a.D = dims->D;
    a.ps = dims->page_size;
    a.max_pages = dims->max_pages_per_seq;
    a.T = T;
    a.num_phys = dims->num_phys_pages;
    a.pages_per_split = (items + S - 1) / S;
    a.num_splits = S;
    const Kv4Groups g = kv4_groups(rows, S, R, dims->D);
    a.group = g.group;
    a.parts = S + g.groups;
    a.scale_log2 = (float)scale_log2;
    a.v_scale = exp2f((float)v_exp);
    a.o = o;
    a.lse = lse;
    a.part_o = w.part_o;
    a.part_lse = w.part_lse;
    a.counters = w.counters;
    a.status = d->status;
    a.wait_ns = wait_limit_ns();
    cudaError_t e = R <= kAttn4DecodeRows ? launch_attn4_decode(a, sparse, static_cast<cudaStream_t>(stream))
                                          : launch_attn4_verify(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, sparse ? "kv4_sparse_decode_attn launch" : "kv4_dense_verify_attn launch");
}

SPD_API spd_status kv4_sparse_decode_attn(const spd_dims* dims, const spd_bf16* q, const uint8_t* kv4, int32_t k_exp,
                                          int32_t v_exp, const int32_t* page_table, const int32_t* seq_lens,
                                          const int32_t* sel, const int32_t* nsel, int32_t k_max, int32_t num_splits,
                                          float softmax_scale, spd_bf16* o, float* lse, void* ws, size_t ws_bytes,
                                          void* stream) {
    spd_status st = check_dims(dims);
    if (st != SPD_OK) return st;
    if (k_max < 1) return fail(SPD_ERR_INVALID_ARG, "k_max < 1");
    if (dims->B == 0) return SPD_OK;
    if (!sel || !nsel) return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    return kv4_attn(dims, 1, q, kv4, k_exp, v_exp, page_table, seq_lens, sel, nsel, k_max, num_splits, softmax_scale, o,
                    lse, ws, ws_bytes, stream);
}

SPD_API spd_status kv4_dense_verify_attn(const spd_dims* dims, int32_t T, const spd_bf16* q, const uint8_t* kv4,
                                         int32_t k_exp, int32_t v_exp, const int32_t* page_table,
                                         const int32_t* seq_lens, int32_t num_splits, float softmax_scale, spd_bf16* o,
                                         float* lse, void* ws, size_t ws_bytes, void* stream) {
    spd_status st = check_dims(dims);
    if (st != SPD_OK) return st;
    st = kv4_check_T(dims, T);
    if (st != SPD_OK || dims->B == 0) return st;
    return kv4_attn(dims, T, q, kv4, k_exp, v_exp, page_table, seq_lens, nullptr, nullptr, dims->max_pages_per_seq,
                    num_splits, softmax_scale, o, lse, ws, ws_bytes, stream);
}

// ---------------------------------------------------------------- token log probabilities

static spd_status logprob_shape(int64_t rows, int32_t n_vocab, int32_t top_k) {
    if (rows < 0 || rows >= (1LL << 31)) return fail(SPD_ERR_INVALID_ARG, "rows = %lld outside [0, 2^31)", (long long)rows);
    if (n_vocab < 1 || n_vocab > (1 << 21)) return fail(SPD_ERR_UNSUPPORTED, "n_vocab = %d outside [1, 2^21]", n_vocab);
    if (top_k < 0 || top_k > 32) return fail(SPD_ERR_UNSUPPORTED, "top_k = %d outside [0, 32]", top_k);
    if (rows * ((n_vocab >> 10) + 1) >= (1LL << 31)) return fail(SPD_ERR_UNSUPPORTED, "rows * n_vocab too large");
    return SPD_OK;
}

SPD_API size_t spd_token_logprobs_workspace_size(int64_t rows, int32_t n_vocab, int32_t top_k) {
    spd_status st = logprob_shape(rows, n_vocab, top_k);
    if (st != SPD_OK) return 0;
    DevInfo* d = dev_info(&st);
    return d ? token_logprobs_ws(rows, n_vocab, top_k, d->sms) : 0;
}

SPD_API spd_status token_logprobs(int64_t rows, int32_t n_vocab, const void* logits, int32_t logits_bf16,
                                  int64_t row_stride, const int32_t* targets, float inv_temperature, float* logprob,
                                  float* entropy, float* lse, int32_t top_k, int32_t* top_ids, float* top_logprobs,
                                  void* ws, size_t ws_bytes, void* stream) {
    spd_status st = logprob_shape(rows, n_vocab, top_k);
    if (st != SPD_OK) return st;
    if (row_stride < n_vocab) return fail(SPD_ERR_INVALID_ARG, "row_stride %lld < n_vocab %d", (long long)row_stride, n_vocab);
    if (!(inv_temperature > 0.f && inv_temperature * kLog2e <= 3.4e38f))
        return fail(SPD_ERR_INVALID_ARG, "inv_temperature must be > 0 and finite, times log2(e) too");
    if (rows == 0) return SPD_OK;
    if (!logits || (logprob && !targets) || (top_k > 0 && (!top_ids || !top_logprobs)))
        return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (reinterpret_cast<uintptr_t>(logits) % (logits_bf16 ? 2 : 4))
        return fail(SPD_ERR_INVALID_ARG, "logits are not aligned to their type");
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    const size_t need = token_logprobs_ws(rows, n_vocab, top_k, d->sms);
    if (!ws || ws_bytes < need) return fail(SPD_ERR_WORKSPACE, "workspace %zu bytes < %zu", ws_bytes, need);
    if (!aligned16(ws)) return fail(SPD_ERR_INVALID_ARG, "ws must be 16-byte aligned");
    LogprobArgs a = {};
    a.logits = logits;
    a.bf16 = logits_bf16 != 0;
    a.rows = rows;
    a.row_stride = row_stride;
    a.n = n_vocab;
    a.targets = targets;
    a.inv_t = inv_temperature;
    a.logprob = logprob;
    a.entropy = entropy;
    a.lse = lse;
    a.top_k = top_k;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.ws = ws;
    a.status = d->status;
    cudaError_t e = launch_token_logprobs(a, d->sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "token_logprobs launch");
}

// ---------------------------------------------------------------- trees of drafted tokens

// T and the rows of its nodes.
static spd_status tree_rows(const spd_dims* dims, int32_t T, const spd_bf16* k_tree, int64_t k_stride,
                            const spd_bf16* v_tree, int64_t v_stride) {
    if (T < 1 || T > kTreeMax) return fail(SPD_ERR_UNSUPPORTED, "T = %d outside [1, %d]", T, kTreeMax);
    if (dims->B == 0) return SPD_OK;
    const int64_t row = (int64_t)dims->H_kv * dims->D;
    if (!k_tree || !v_tree) return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(k_tree) || !aligned16(v_tree)) return fail(SPD_ERR_INVALID_ARG, "k_tree and v_tree must be 16-byte aligned");
    if (k_stride < row || k_stride % 8 || v_stride < row || v_stride % 8)
        return fail(SPD_ERR_INVALID_ARG, "bad row strides (k_stride=%lld v_stride=%lld)", (long long)k_stride, (long long)v_stride);
    return SPD_OK;
}

// One position for a token: in 32 signed bits, with room for a tile behind the last.
static spd_status position_dims(const spd_dims* dims) {
    if ((long long)dims->max_pages_per_seq * dims->page_size > (1LL << 30))
        return fail(SPD_ERR_UNSUPPORTED, "max_pages_per_seq * page_size must be at most 2^30");
    return SPD_OK;
}

static spd_status tree_attn_dims(const spd_dims* dims, int32_t T) {
    spd_status st = check_dims(dims);
    if (st == SPD_OK) st = position_dims(dims);
    if (st != SPD_OK) return st;
    if (T < 1 || T > kTreeMax) return fail(SPD_ERR_UNSUPPORTED, "T = %d outside [1, %d]", T, kTreeMax);
    if ((long long)dims->B * dims->H_kv > 16384) return fail(SPD_ERR_UNSUPPORTED, "B * H_kv must be at most 16384");
    return SPD_OK;
}

static spd_status tree_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* size, const cuuint64_t* stride,
                           const cuuint32_t* box) {
    spd_status st = SPD_OK;
    EncodeTiledFn fn = encode_fn(&st);
    if (!fn) return st;
    const cuuint32_t step[5] = {1, 1, 1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), size, stride, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SPD_OK : fail(SPD_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
}

// Pages of keys or values as boxes of atoms, 8 slots by 64 channels: [page and KV head][slot / 8][half][slot % 8], n of them.
static spd_status page_map(CUtensorMap* m, const void* base, int D, int ps, cuuint64_t n) {
    const cuuint64_t row = (cuuint64_t)D * 2, halves = (cuuint64_t)D / 64;
    const cuuint64_t size[5] = {64, 8, halves, (cuuint64_t)ps / 8, n}, stride[4] = {row, 128, row * 8, row * ps};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)halves, (cuuint32_t)ps / 8, 1};
    return tree_map(m, base, 5, size, stride, box);
}

// The views that the tree's attention copies boxes of, 64 channels (128 bytes) wide: pages as [page and KV head][slot / 8][half][slot % 8] and [page and KV head][half][slot],
// queries as [half][row][head], nodes as [half][head][sequence][node] (what lies behind the last node arrives as zeros).
static spd_status tree_maps(const TreeAttnArgs& a, TreeMaps* m) {
    const cuuint64_t row = (cuuint64_t)a.D * 2, halves = (cuuint64_t)a.D / 64;
    const cuuint64_t pages = (cuuint64_t)a.num_phys * a.H_kv;
    const cuuint64_t n = pages ? pages : 1;
    const cuuint64_t e_size[4] = {64, (cuuint64_t)a.ps, halves, n}, e_stride[3] = {row, 128, row * a.ps};
    const cuuint32_t e_box[4] = {64, 8, 1, 1};
    spd_status st = page_map(&m->k, a.K, a.D, a.ps, n);
    if (st == SPD_OK) st = page_map(&m->v, a.V, a.D, a.ps, n);
    if (st == SPD_OK) st = tree_map(&m->k_edge, a.K, 4, e_size, e_stride, e_box);
    if (st == SPD_OK) st = tree_map(&m->v_edge, a.V, 4, e_size, e_stride, e_box);
    const int G = a.H_q / a.H_kv;
    const cuuint64_t q_size[4] = {64, (cuuint64_t)a.H_q, (cuuint64_t)a.B * a.T, halves}, q_stride[3] = {row, (cuuint64_t)a.q_stride * 2, 128};
    const cuuint32_t q_box[4] = {64, (cuuint32_t)G, (cuuint32_t)tree_nodes_per_tile(a.T, G), 1};
    if (st == SPD_OK) st = tree_map(&m->q, a.q, 4, q_size, q_stride, q_box);
    const cuuint32_t t_box[5] = {64, kTreeMax, 1, 1, 1};
    for (int i = 0; i < 2 && st == SPD_OK; ++i) {
        const cuuint64_t stride = (cuuint64_t)(i ? a.v_stride : a.k_stride) * 2;
        const cuuint64_t t_size[5] = {64, (cuuint64_t)a.T, (cuuint64_t)a.B, (cuuint64_t)a.H_kv, halves};
        const cuuint64_t t_stride[4] = {stride, stride * a.T, row, 128};
        st = tree_map(i ? &m->vt : &m->kt, i ? a.v_tree : a.k_tree, 5, t_size, t_stride, t_box);
    }
    return st;
}

SPD_API size_t spd_tree_verify_workspace_size(const spd_dims* dims, int32_t T) {
    if (tree_attn_dims(dims, T) != SPD_OK) return 0;
    spd_status st = SPD_OK;
    DevInfo* d = dev_info(&st);
    return d ? kTicketBytes + tree_attn_ws(dims->D, d->sms) : 0;
}

SPD_API spd_status tree_verify_attn(const spd_dims* dims, int32_t T, const spd_bf16* q, int64_t q_stride,
                                    const spd_bf16* K, const spd_bf16* V, const int32_t* page_table,
                                    const int32_t* seq_lens, const spd_bf16* k_tree, int64_t k_stride,
                                    const spd_bf16* v_tree, int64_t v_stride, const int32_t* parents,
                                    float softmax_scale, spd_bf16* o, float* lse, void* ws, size_t ws_bytes,
                                    void* stream) {
    spd_status st = tree_attn_dims(dims, T);
    if (st == SPD_OK) st = tree_rows(dims, T, k_tree, k_stride, v_tree, v_stride);
    if (st != SPD_OK) return st;
    const double scale_log2 = (double)softmax_scale * 1.4426950408889634;
    if (!(fabs(scale_log2) <= 3.4e38)) return fail(SPD_ERR_INVALID_ARG, "softmax_scale must be finite, times log2(e) too");
    if (dims->B == 0) return SPD_OK;
    if (!q || !K || !V || !page_table || !seq_lens || !parents || !o) return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(q) || !aligned16(K) || !aligned16(V) || !aligned16(o))
        return fail(SPD_ERR_INVALID_ARG, "q, K, V and o must be 16-byte aligned");
    if (q_stride < (int64_t)dims->H_q * dims->D || q_stride % 8)
        return fail(SPD_ERR_INVALID_ARG, "bad row stride (q_stride=%lld)", (long long)q_stride);
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    const size_t need = kTicketBytes + tree_attn_ws(dims->D, d->sms);
    if (!ws || ws_bytes < need) return fail(SPD_ERR_WORKSPACE, "workspace %zu bytes < %zu", ws_bytes, need);
    if (!aligned16(ws)) return fail(SPD_ERR_INVALID_ARG, "ws must be 16-byte aligned");
    TreeAttnArgs a = {};
    a.q = q;
    a.K = K;
    a.V = V;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.k_tree = k_tree;
    a.v_tree = v_tree;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.parents = parents;
    a.B = dims->B;
    a.H_q = dims->H_q;
    a.H_kv = dims->H_kv;
    a.D = dims->D;
    a.ps = dims->page_size;
    a.max_pages = dims->max_pages_per_seq;
    a.T = T;
    a.num_phys = dims->num_phys_pages;
    a.scale_log2 = (float)scale_log2;
    a.o = o;
    a.lse = lse;
    a.ws = static_cast<char*>(ws) + kTicketBytes;  // behind the place of every call's tickets
    a.num_sms = d->sms;
    a.status = d->status;
    a.wait_ns = wait_limit_ns();
    TreeMaps m;
    st = tree_maps(a, &m);
    if (st != SPD_OK) return st;
    cudaError_t e = launch_tree_attn(a, m, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "tree_verify_attn launch");
}

SPD_API spd_status spec_accept_tree(int32_t B, int32_t T, int32_t n_vocab, const float* q_target, const int32_t* draft,
                                    const int32_t* parents, const float* u_acc, const float* u_res, int32_t* n_path,
                                    int32_t* path, int32_t* tokens, void* stream) {
    if (B < 0) return fail(SPD_ERR_INVALID_ARG, "B < 0");
    if (T < 1 || T > kTreeMax) return fail(SPD_ERR_UNSUPPORTED, "T = %d outside [1, %d]", T, kTreeMax);
    if (n_vocab < 1 || n_vocab > (1 << 21)) return fail(SPD_ERR_UNSUPPORTED, "n_vocab = %d outside [1, 2^21]", n_vocab);
    if ((int64_t)B * 16 >= (1LL << 31)) return fail(SPD_ERR_UNSUPPORTED, "B = %d is too large", B);
    if (B == 0) return SPD_OK;
    if (!q_target || !draft || !parents || !u_acc || !u_res || !n_path || !path || !tokens)
        return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(q_target)) return fail(SPD_ERR_INVALID_ARG, "q_target must be 16-byte aligned");
    spd_status st;
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    TreeAcceptArgs a = {};
    a.q = q_target;
    a.draft = draft;
    a.parents = parents;
    a.u_acc = u_acc;
    a.u_res = u_res;
    a.n_path = n_path;
    a.path = path;
    a.tokens = tokens;
    a.B = B;
    a.T = T;
    a.n = n_vocab;
    a.status = d->status;
    a.wait_ns = wait_limit_ns();
    cudaError_t e = launch_spec_accept_tree(a, d->sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "spec_accept_tree launch");
}

SPD_API spd_status kv_append_path(const spd_dims* dims, int32_t T, spd_bf16* K, spd_bf16* V, const int32_t* page_table,
                                  const int32_t* seq_lens, const spd_bf16* k_tree, int64_t k_stride,
                                  const spd_bf16* v_tree, int64_t v_stride, const int32_t* path, const int32_t* n_path,
                                  spd_bf16* summ, int32_t* new_lens, void* stream) {
    spd_status st = check_dims(dims);
    if (st != SPD_OK) return st;
    st = tree_rows(dims, T, k_tree, k_stride, v_tree, v_stride);
    if (st != SPD_OK || dims->B == 0) return st;
    if (!K || !V || !page_table || !seq_lens || !path || !n_path || !summ || !new_lens)
        return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(K) || !aligned16(V) || !aligned16(summ))
        return fail(SPD_ERR_INVALID_ARG, "K, V and summ must be 16-byte aligned");
    if (new_lens == seq_lens) return fail(SPD_ERR_INVALID_ARG, "new_lens must not be seq_lens");
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    AppendPathArgs p = {};
    AppendArgs& a = p.append;
    a.K = K;
    a.V = V;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.k_new = k_tree;
    a.v_new = v_tree;
    a.summ = summ;
    a.B = dims->B;
    a.T = T;
    a.H_kv = dims->H_kv;
    a.D = dims->D;
    a.ps = dims->page_size;
    a.max_pages = dims->max_pages_per_seq;
    a.num_phys = dims->num_phys_pages;
    a.status = d->status;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.path = path;
    p.n_path = n_path;
    p.new_lens = new_lens;
    cudaError_t e = launch_append_path(p, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "kv_append_path launch");
}

// ---------------------------------------------------------------- eviction by attention weight

SPD_API spd_status kv_weights_update(const spd_dims* dims, int32_t T, const spd_bf16* q, const float* lse,
                                     const spd_bf16* K, const int32_t* page_table, const int32_t* seq_lens,
                                     const int32_t* path, const int32_t* n_path, const int32_t* sel,
                                     const int32_t* nsel, int32_t k_max, float decay, float softmax_scale,
                                     const float* w_in, float* w_out, void* stream) {
    spd_status st = check_dims(dims);
    if (st == SPD_OK) st = position_dims(dims);
    if (st != SPD_OK) return st;
    if (T < 1 || T > kTreeMax) return fail(SPD_ERR_UNSUPPORTED, "T = %d outside [1, %d]", T, kTreeMax);
    const double scale_log2 = (double)softmax_scale * 1.4426950408889634;
    if (!(fabs(scale_log2) <= 3.4e38) || !(fabsf(decay) <= 3.4e38f))
        return fail(SPD_ERR_INVALID_ARG, "decay and softmax_scale must be finite");
    if ((path != nullptr) != (n_path != nullptr)) return fail(SPD_ERR_INVALID_ARG, "path and n_path go together");
    if ((sel != nullptr) != (nsel != nullptr)) return fail(SPD_ERR_INVALID_ARG, "sel and nsel go together");
    if (sel && k_max < 1) return fail(SPD_ERR_INVALID_ARG, "k_max < 1");
    if ((long long)dims->B * dims->H_kv * (((long long)dims->max_pages_per_seq * dims->page_size >> 9) + 1) >= (1LL << 31))
        return fail(SPD_ERR_UNSUPPORTED, "B * H_kv * max_pages_per_seq is too large");
    if (dims->B == 0) return SPD_OK;
    if (!q || !lse || !K || !page_table || !seq_lens || !w_out) return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(q) || !aligned16(K)) return fail(SPD_ERR_INVALID_ARG, "q and K must be 16-byte aligned");
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    WeightsArgs a = {};
    a.q = q;
    a.lse = lse;
    a.K = K;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.path = path;
    a.n_path = n_path;
    a.sel = sel;
    a.nsel = nsel;
    a.k_max = k_max;
    a.B = dims->B;
    a.H_q = dims->H_q;
    a.H_kv = dims->H_kv;
    a.D = dims->D;
    a.ps = dims->page_size;
    a.max_pages = dims->max_pages_per_seq;
    a.T = T;
    a.num_phys = dims->num_phys_pages;
    a.decay = decay;
    a.scale_log2 = (float)scale_log2;
    a.w_in = w_in;
    a.w_out = w_out;
    a.status = d->status;
    a.wait_ns = wait_limit_ns();
    spd_dims k = *dims;
    if (k.num_phys_pages < 1) k.num_phys_pages = 1;  // (a view of nothing is none; no page of it is read)
    CUtensorMap map;
    st = weights_by_tiles(T, dims->H_q / dims->H_kv, sel != nullptr, (long long)k.max_pages_per_seq * k.page_size)
             ? page_map(&map, K, k.D, k.page_size, dims->num_phys_pages ? (cuuint64_t)k.num_phys_pages * k.H_kv : 1)
                                                                      : kv_map(&map, K, &k, 16);
    if (st != SPD_OK) return st;
    cudaError_t e = launch_weights_update(a, map, d->sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "kv_weights_update launch");
}

SPD_API spd_status kv_evict(const spd_dims* dims, int32_t budget, int32_t n_sink, int32_t n_recent, spd_bf16* K,
                            spd_bf16* V, const int32_t* page_table, const int32_t* seq_lens, const float* weights,
                            const int32_t* dst_table, int32_t* kept, float* weights_out, spd_bf16* summ,
                            int32_t* new_lens, void* stream) {
    spd_status st = check_dims(dims);
    if (st == SPD_OK) st = position_dims(dims);
    if (st != SPD_OK) return st;
    if (budget < 1 || n_sink < 0 || n_recent < 0 || (int64_t)n_sink + n_recent > budget)
        return fail(SPD_ERR_INVALID_ARG, "budget %d must be >= 1 and hold n_sink (%d) and n_recent (%d) tokens", budget, n_sink, n_recent);
    const long long rows = (long long)dims->B * dims->H_kv;
    if (rows * 8 >= (1LL << 31) || rows * dims->max_pages_per_seq >= (1LL << 31))
        return fail(SPD_ERR_UNSUPPORTED, "B * H_kv * max_pages_per_seq is too large");
    if (dims->B == 0) return SPD_OK;
    if (!K || !V || !page_table || !seq_lens || !weights || !dst_table || !kept || !weights_out || !summ || !new_lens)
        return fail(SPD_ERR_INVALID_ARG, "NULL pointer argument");
    if (!aligned16(K) || !aligned16(V) || !aligned16(summ))
        return fail(SPD_ERR_INVALID_ARG, "K, V and summ must be 16-byte aligned");
    if (new_lens == seq_lens || weights_out == weights || dst_table == page_table)
        return fail(SPD_ERR_INVALID_ARG, "new_lens, weights_out and dst_table must not be seq_lens, weights and page_table");
    DevInfo* d = dev_info(&st);
    if (!d) return st;
    EvictArgs a = {};
    a.K = K;
    a.V = V;
    a.page_table = page_table;
    a.seq_lens = seq_lens;
    a.dst_table = dst_table;
    a.w = weights;
    a.w_out = weights_out;
    a.kept = kept;
    a.summ = summ;
    a.new_lens = new_lens;
    a.budget = budget;
    a.n_sink = n_sink;
    a.n_recent = n_recent;
    a.B = dims->B;
    a.H_kv = dims->H_kv;
    a.D = dims->D;
    a.ps = dims->page_size;
    a.max_pages = dims->max_pages_per_seq;
    a.num_phys = dims->num_phys_pages;
    a.status = d->status;
    cudaError_t e = launch_evict(a, d->sms, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPD_OK : cuda_fail(e, "kv_evict launch");
}
