// kernels.h -- host-side launch interface between the C-ABI layer (spd_api.cu)
// and the kernel translation units.  Internal to the library.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spd.h"

#include <utility>

namespace spd {

// Launches a kernel of the library with programmatic stream serialisation
// allowed (see pdl_wait / pdl_trigger): the launch of a kernel overlaps the
// tail of the previous one on the stream.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// The same in clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, unsigned cluster,
                               cudaStream_t st, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

struct SummarizeArgs {
    const uint16_t* K;
    const int32_t* page_table;
    const int32_t* seq_lens;
    const int32_t* only_pages;  // NULL = all pages
    int n_only;
    uint16_t* summ;
    int B, H_kv, D, ps, max_pages;
    long long num_phys;
    unsigned* status;
};
cudaError_t launch_summarize(const SummarizeArgs& a, cudaStream_t st);

struct AppendArgs {
    uint16_t* K;
    uint16_t* V;
    const int32_t* page_table;
    const int32_t* seq_lens;
    const uint16_t* k_new;  // [B][T][H_kv][D]
    const uint16_t* v_new;
    uint16_t* summ;         // [B][H_kv][max_pages][2][D]
    int B, T, H_kv, D, ps, max_pages;
    long long num_phys;
    unsigned* status;
};
cudaError_t launch_append_refresh(const AppendArgs& a, cudaStream_t st);

// Pages that T consecutive positions of a sequence can span.
inline int append_touched(int T, int ps, int max_pages) {
    const int n = (T - 1 + ps - 1) / ps + 1;
    return n < max_pages ? n : max_pages;
}

struct RopeArgs {
    const uint16_t* q;  // [rows] rows of H_q heads, q_stride elements apart (NULL: H_q = 0)
    const uint16_t* k;  // [rows] rows of H_kv heads, k_stride elements apart (NULL: H_kv = 0)
    long long q_stride, k_stride, rows;
    int H_q, H_kv, D;
    const int32_t* positions;  // [rows]
    const float* table;        // [n_pos][2][rot / 2]
    int n_pos, rot, interleaved;
    const uint16_t* q_weight;  // [D] or NULL: no norm
    const uint16_t* k_weight;
    float eps;
    uint16_t* q_out;  // [rows][H_q][D]
    uint16_t* k_out;  // [rows][H_kv][D]
    unsigned* status;
};
cudaError_t launch_qk_norm_rope(const RopeArgs& a, cudaStream_t st);

struct AppendRopeArgs {
    AppendArgs append;  // k_new and v_new are not used: the rows come from rope.k and v
    RopeArgs rope;      // rows = B * T; positions come from seq_lens
    const uint16_t* v;
    long long v_stride;
    int touched;  // set by the launch
};
cudaError_t launch_append_rope(const AppendRopeArgs& a, cudaStream_t st);
// CTAs of its grid (to be kept below 2^31).
long long append_rope_ctas(const AppendRopeArgs& a);

// The 4-bit cache: [num_phys][H_kv][2][ps * D * 9 / 16] bytes (see include/spd.h).
struct Kv4Args {
    uint8_t* kv4;
    const int32_t* page_table;
    const int32_t* seq_lens;
    const uint16_t* k_new;  // append: [B][T][H_kv][D]
    const uint16_t* v_new;
    uint16_t* summ;         // append: [B][H_kv][max_pages][2][D]
    uint16_t* k_out;        // read: [B][T][H_kv][D]
    uint16_t* v_out;
    int B, T, H_kv, D, ps, max_pages;
    long long num_phys;
    int k_exp, v_exp;
    unsigned* status;
};
cudaError_t launch_kv4_append(const Kv4Args& a, cudaStream_t st);
cudaError_t launch_kv4_read(const Kv4Args& a, cudaStream_t st);

// Split tickets at the start (16 bytes on) of every workspace, the same for every call: no call's
// scores or partials lie before kTicketBytes.  (The 4-bit attention and token_logprobs split no
// more rows than that; where the bf16 attention is told to, its tickets go on behind them.)
constexpr int kTickets = 16384;
constexpr size_t kTicketBytes = (16 + kTickets * sizeof(int) + 255) / 256 * 256;

struct Attn4Args {
    const uint16_t* q;  // [B][T][H_q][D]
    const uint8_t* kv4;
    const int32_t* page_table;
    const int32_t* seq_lens;
    const int32_t* sel;   // sparse only
    const int32_t* nsel;  // sparse only
    int k_max;
    int B, H_q, H_kv, D, ps, max_pages, T;
    long long num_phys;
    int pages_per_split, num_splits;
    float scale_log2;  // softmax scale * log2(e) * 2^k_exp
    float v_scale;     // 2^v_exp
    uint16_t* o;
    float* lse;
    float* part_o;    // [B*H_kv][parts][R][D]: the splits' outputs, then those of groups of splits
    float* part_lse;  // [B*H_kv][parts][R]
    int* counters;    // tickets of the rows, then of their groups, zero on entry and on exit
    int parts;        // num_splits and the groups, if there are any
    int group;        // splits of a group (num_splits: no groups)
    unsigned* status;
    unsigned long long wait_ns;  // limit of every bounded wait
};
// Up to 8 query rows of a KV head (T * G), dense or sparse; 9 to 64, dense.
cudaError_t launch_attn4_decode(const Attn4Args& a, bool sparse, cudaStream_t st);
cudaError_t launch_attn4_verify(const Attn4Args& a, cudaStream_t st);
constexpr int kAttn4DecodeRows = 8;
// Their CTAs on one SM.
int occ_attn4_decode();
int occ_attn4_verify();

struct LogprobArgs {
    const void* logits;  // [rows][n], row_stride elements apart
    bool bf16;
    long long rows, row_stride;
    int n;
    const int32_t* targets;
    float inv_t;
    float* logprob;
    float* entropy;  // may be NULL
    float* lse;      // may be NULL
    int top_k;
    int32_t* top_ids;
    float* top_logprobs;
    void* ws;
    unsigned* status;
};
cudaError_t launch_token_logprobs(const LogprobArgs& a, int num_sms, cudaStream_t st);
size_t token_logprobs_ws(long long rows, int n, int top_k, int num_sms);

// Default limit of every bounded wait in the kernels (spd_set_wait_limit_ns).
constexpr unsigned long long kDefaultWaitNs = 2000000000ull;
// The limit the next launches pass to their kernels.
unsigned long long wait_limit_ns();

struct SpecArgs {
    const float* p;        // [B][k][n] drafter probabilities
    const float* q;        // [B][k+1][n] target probabilities
    const int32_t* draft;  // [B][k]
    const float* u_acc;    // [B][k]
    const float* u_res;    // [B]
    int32_t* n_accepted;   // [B]
    int32_t* tokens;       // [B][k+1]
    int B, k;
    long long n;
    unsigned* status;
    unsigned long long wait_ns;
};
cudaError_t launch_spec_accept(const SpecArgs& a, cudaStream_t st);
size_t spec_smem_bytes(long long n);

// The largest tree of drafted tokens (its masks are 64-bit words).
constexpr int kTreeMax = 64;

struct TreeAttnArgs {
    const uint16_t* q;       // rows [B * T] of H_q * D, q_stride elements apart
    const uint16_t* K;
    const uint16_t* V;
    const int32_t* page_table;
    const int32_t* seq_lens;  // of the cache alone
    const uint16_t* k_tree;  // rows [B * T] of H_kv * D
    const uint16_t* v_tree;
    long long q_stride, k_stride, v_stride;
    const int32_t* parents;  // [B][T]
    int B, H_q, H_kv, D, ps, max_pages, T;
    long long num_phys;
    float scale_log2;
    uint16_t* o;
    float* lse;
    void* ws;
    int num_sms;
    unsigned* status;
    unsigned long long wait_ns;
};
// A page's keys or values of a KV head (k, v); eight slots of it by 64 channels (edge); 64 channels of a group's heads and
// nodes (q), of the nodes (kt, vt).
struct TreeMaps {
    CUtensorMap k, v, k_edge, v_edge, q, kt, vt;
};
cudaError_t launch_tree_attn(const TreeAttnArgs& a, const TreeMaps& m, cudaStream_t st);
size_t tree_attn_ws(int D, int num_sms);  // of a.ws
int tree_nodes_per_tile(int T, int G);    // nodes in q's box

struct TreeAcceptArgs {
    const float* q;          // [B][T][n] target probabilities
    const int32_t* draft;    // [B][T]
    const int32_t* parents;  // [B][T]
    const float* u_acc;      // [B][T]
    const float* u_res;      // [B]
    int32_t* n_path;         // [B]
    int32_t* path;           // [B][T]
    int32_t* tokens;         // [B][T]
    int B, T;
    long long n;
    unsigned* status;
    unsigned long long wait_ns;
};
cudaError_t launch_spec_accept_tree(const TreeAcceptArgs& a, int num_sms, cudaStream_t st);

struct AppendPathArgs {
    AppendArgs append;  // T = nodes; k_new and v_new: node rows, k_stride and v_stride elements apart
    long long k_stride, v_stride;
    const int32_t* path;    // [B][T]
    const int32_t* n_path;  // [B]
    int32_t* new_lens;      // [B]
};
cudaError_t launch_append_path(const AppendPathArgs& a, cudaStream_t st);

struct WeightsArgs {
    const uint16_t* q;  // [B][T][H_q][D]
    const float* lse;   // [B][T][H_q]
    const uint16_t* K;
    const int32_t* page_table;
    const int32_t* seq_lens;
    const int32_t* path;    // [B][T], with n_path [B]; NULL: all T rows in order
    const int32_t* n_path;
    const int32_t* sel;     // [B][H_kv][k_max], with nsel [B][H_kv]; NULL: every page
    const int32_t* nsel;
    int k_max;
    int B, H_q, H_kv, D, ps, max_pages, T;
    long long num_phys;
    float decay, scale_log2;
    const float* w_in;  // [B][H_kv][max_pages * ps] or NULL
    float* w_out;
    unsigned* status;
    unsigned long long wait_ns;
};
// Whether it goes by tiles of 128 tokens (many query rows, or a table for `most` tokens that is wide); map: then boxes of a page of K as
// tree_verify_attn's, else of 16 rows.
bool weights_by_tiles(int T, int G, bool selected, long long most);
cudaError_t launch_weights_update(const WeightsArgs& a, const CUtensorMap& map, int num_sms, cudaStream_t st);

struct EvictArgs {
    uint16_t* K;
    uint16_t* V;
    const int32_t* page_table;
    const int32_t* seq_lens;
    const int32_t* dst_table;
    const float* w;  // [B][H_kv][max_pages * ps]
    float* w_out;
    int32_t* kept;   // [B][H_kv][budget]
    uint16_t* summ;  // [B][H_kv][max_pages][2][D]
    int32_t* new_lens;
    int budget, n_sink, n_recent;
    int B, H_kv, D, ps, max_pages;
    long long num_phys;
    unsigned* status;
};
cudaError_t launch_evict(const EvictArgs& a, int num_sms, cudaStream_t st);

struct ScoreSelectArgs {
    const uint16_t* q;
    const uint16_t* summ;  // [B][H_kv][max_pages][2][D]
    const int32_t* seq_lens;
    spd_budget_policy pol;
    int32_t* sel;
    int32_t* nsel;
    int k_max;
    float* scores;    // [B][H_kv][max_pages]
    int B, H_q, H_kv, D, ps, max_pages;
    long long num_phys;
    unsigned* status;
    // Fused append (pages_append_score_select): the step's token, written into the
    // cache and into its page's summary by the warp that scores that page.
    uint16_t* K;  // NULL: no append
    uint16_t* V;
    const int32_t* page_table;
    const uint16_t* k_new;  // [B][H_kv][D]
    const uint16_t* v_new;
    uint16_t* summ_w;       // == summ
    // Chained step (sparse_decode_step): tiles are handed out in row order from
    // counters, each finished tile is counted per row, and the selection of a row
    // starts when its count is complete (instead of after the whole scoring grid).
    unsigned long long* tile_ctr;  // [2]: chunk and single-tile counters, zero on entry and on exit
    unsigned* warps_done;
    unsigned* sel_claims;          // chained step: the selection CTAs' row claims (zero on entry and on exit)
    unsigned* tiles_done;          // [B*H_kv] progress hints (NULL: not chained), zero on entry and on exit
    unsigned* sel_done;            // [B*H_kv]: set when a row's selection is written
    // [B*H_kv][max_pages] order-preserving score keys (never 0), zero on entry and
    // on exit: a key is its own ready flag, so the scoring warps need no fences
    unsigned* keys;
    // chained step: [B*H_kv][k_max] the physical page of each selected page (read by
    // the attention instead of the page table); NULL otherwise
    int32_t* sel_phys;
    unsigned long long wait_ns;  // limit of every bounded wait
};
// Scores every page (persistent grid sized to num_sms), then selects per row.
cudaError_t launch_score_select(const ScoreSelectArgs& a, int num_sms, cudaStream_t st);

struct AttnArgs {
    const uint16_t* q;  // [B][T][H_q][D] (T = 1 for decode)
    const int32_t* page_table;
    const int32_t* seq_lens;
    const int32_t* sel;   // sparse only
    const int32_t* nsel;  // sparse only
    int k_max;
    int B, H_q, H_kv, D, ps, max_pages, T;
    long long num_phys;
    int items_per_split, num_splits;
    float scale_log2;
    uint16_t* o;
    float* lse;
    float* part_o;    // [B*H_kv][num_splits][R][D]
    float* part_lse;  // [B*H_kv][num_splits][R]
    int* counters;    // [B*H_kv] split tickets, zero on entry and on exit
    int* queue;       // 16 bytes (8-aligned): the unit queue counter, zero on entry and exit
    int num_sms;
    unsigned* status;
    unsigned* sel_done;  // chained step: wait for the row's selection flag instead of the previous grid
    const int32_t* sel_phys;  // chained step: physical pages of sel (NULL: look them up in page_table)
    unsigned long long wait_ns;  // limit of every bounded wait
};
// Rows (T * G) handled per CTA, padded to 16-row MMA tiles.
inline int attn_mtiles(int T, int G) {
    int r = T * G;
    return r <= 16 ? 1 : (r <= 32 ? 2 : 4);
}
cudaError_t launch_sparse_attn(const AttnArgs& a, const CUtensorMap& tmK, const CUtensorMap& tmV,
                               cudaStream_t st);
cudaError_t launch_dense_attn(const AttnArgs& a, const CUtensorMap& tmK, const CUtensorMap& tmV,
                              cudaStream_t st);
// CTAs of the attention kernel that fit on one SM for this shape.
int occ_sparse_attn(int D, int ps);
int occ_dense_attn(int D, int ps, int mtiles);

// Host helpers of the C-ABI layer shared with round.cu.
spd_status device_ready();
spd_status set_error(spd_status s, const char* msg);

cudaError_t launch_lse_merge(int S, int rows, int D, const float* part_o, const float* part_lse,
                             uint16_t* o, float* lse, cudaStream_t st);

}  // namespace spd
