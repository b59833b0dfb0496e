// api_seq.hip -- extern "C" entry points of the operators around the tree: the
// prompt scan, the single-token step, the short convolution, the heads' norms and
// rotation, and the paged cache's attention and writes (declared in
// include/tree_ssd.h). Host-side validation happens here, before anything is enqueued.
#include <math.h>

#include "attn_common.hpp"
#include "seq_launch.hpp"

namespace {

constexpr int kMaxTree = 1024;
constexpr int kMaxDim = 256;
constexpr float kLog2e = 1.44269504088896340736f;  // the scores' exponentials have base 2
// A launch counts its threads in 32 bits, and all of these have work-groups of
// 256: one more work-group than this would run as a grid of what is left over
constexpr long long kMaxBlocks = 0xffffffffLL / 256;

bool dtype_ok(int d) { return d == TSV_F32 || d == TSV_BF16; }

// Rows, sequences and positions end 2^16 below the largest int, so that the kernels'
// sums of one of them and a tile or a step do not pass it
constexpr int kMaxRows = 0x7fff0000;

tsv_status check_seq(const tsv_seq_shape* s) {
    if (!s) return TSV_E_NULL;
    if (!dtype_ok(s->in_dtype)) return TSV_E_DTYPE;
    if (s->n_seqs < 0 || s->n_tokens < 0) return TSV_E_SHAPE;
    if (s->n_heads < 1 || s->head_dim < 1 || s->d_state < 1 || s->n_groups < 1) return TSV_E_SHAPE;
    if (s->n_heads % s->n_groups != 0) return TSV_E_SHAPE;
    if (s->head_dim > kMaxDim || s->d_state > kMaxDim || s->n_heads > 0xffff) return TSV_E_UNSUPPORTED;
    if (s->n_seqs > kMaxRows || s->n_tokens > kMaxRows) return TSV_E_UNSUPPORTED;
    if (tsv::prefill_blocks(s, s->head_dim * s->d_state % 4 == 0) > kMaxBlocks) return TSV_E_UNSUPPORTED;
    return TSV_OK;
}

tsv_status check_attn(const tsv_attn_shape* s, bool tree) {
    if (!s) return TSV_E_NULL;
    if (!dtype_ok(s->in_dtype)) return TSV_E_DTYPE;
    if (!dtype_ok(s->cache_dtype) && s->cache_dtype != TSV_E4M3) return TSV_E_DTYPE;
    if (s->batch < 0 || s->n_nodes < 0 || (tree && s->n_nodes > kMaxTree)) return TSV_E_SHAPE;
    if (s->n_heads < 1 || s->n_kv_heads < 1 || s->n_heads % s->n_kv_heads != 0) return TSV_E_SHAPE;
    if (s->head_dim < 1 || s->n_pages < 0 || s->max_pages < 0) return TSV_E_SHAPE;
    if (s->page_size < 1 || s->page_size > 65536) return TSV_E_SHAPE;
    if ((long long)s->max_pages * s->page_size > kMaxRows) return TSV_E_SHAPE;
    if (!isfinite(s->scale * kLog2e)) return TSV_E_SHAPE;
    if (s->cache_dtype != s->in_dtype && s->cache_dtype != TSV_E4M3) return TSV_E_UNSUPPORTED;
    if (s->head_dim > kMaxDim || s->n_heads > 0xffff) return TSV_E_UNSUPPORTED;
    return TSV_OK;
}

bool scales_ok(const tsv_attn_shape* s, const void* ks, const void* vs) {
    return s->cache_dtype != TSV_E4M3 || (ks && vs);
}

tsv_status result(hipError_t e) { return e == hipSuccess ? TSV_OK : TSV_E_LAUNCH; }

tsv::CacheWriteArgs write_args(const tsv_attn_shape* s, const void* k, const void* v, const int32_t* page_table,
                               const int32_t* cache_len, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                               int32_t* status) {
    tsv::CacheWriteArgs a{};
    a.k = k; a.v = v; a.page_table = page_table; a.cache_len = cache_len;
    a.k_cache = k_cache; a.v_cache = v_cache; a.k_scale = k_scale; a.v_scale = v_scale; a.status = status;
    a.batch = s->batch; a.T = s->n_nodes; a.Hk = s->n_kv_heads; a.D = s->head_dim;
    a.n_pages = s->n_pages; a.page_size = s->page_size; a.max_pages = s->max_pages;
    a.div = tsv::page_div(s->page_size);
    a.heads = tsv::page_div(2 * s->n_kv_heads);
    return a;
}

// ---- the short convolution: what the shapes of prompts and trees share
tsv_status check_conv(int rows, int n, int H, int P, int N, int G, const tsv_conv* c) {
    if (!c) return TSV_E_NULL;
    if (rows < 0 || n < 0) return TSV_E_SHAPE;
    if (H < 1 || P < 1 || N < 1 || G < 1 || H % G != 0) return TSV_E_SHAPE;
    if (c->width < 2 || (c->silu != 0 && c->silu != 1)) return TSV_E_SHAPE;
    if (P > kMaxDim || N > kMaxDim || H > 0xffff || c->width > 4) return TSV_E_UNSUPPORTED;
    if (c->row_stride < (long long)H * P + 2LL * G * N) return TSV_E_SHAPE;
    if (rows > kMaxRows || n > kMaxRows) return TSV_E_UNSUPPORTED;
    return TSV_OK;
}

tsv_status check_conv(const tsv_seq_shape* s, const tsv_conv* c) {
    if (!s) return TSV_E_NULL;
    if (!dtype_ok(s->in_dtype)) return TSV_E_DTYPE;
    const tsv_status st = check_conv(s->n_tokens, s->n_seqs, s->n_heads, s->head_dim, s->d_state, s->n_groups, c);
    if (st != TSV_OK) return st;
    const long long blocks = tsv::conv_blocks(tsv::kConvPrefill, s->n_seqs, s->n_tokens, s->n_heads * s->head_dim, s->n_groups * s->d_state);
    return blocks > kMaxBlocks ? TSV_E_UNSUPPORTED : TSV_OK;
}

tsv_status check_conv(tsv::ConvKind kind, const tsv_shape* s, const tsv_conv* c) {
    if (!s) return TSV_E_NULL;
    if (!dtype_ok(s->in_dtype)) return TSV_E_DTYPE;
    if (s->n_nodes > (kind == tsv::kConvStep ? 1 : kMaxTree)) return TSV_E_SHAPE;
    const tsv_status st = check_conv(s->n_nodes, s->batch, s->n_heads, s->head_dim, s->d_state, s->n_groups, c);
    if (st != TSV_OK || s->batch == 0 || s->n_nodes == 0) return st;
    const long long blocks = tsv::conv_blocks(kind, s->batch, s->n_nodes, s->n_heads * s->head_dim, s->n_groups * s->d_state);
    return blocks > kMaxBlocks ? TSV_E_UNSUPPORTED : TSV_OK;
}

template <class S>
tsv::ConvArgs conv_args(const S* s, const tsv_conv* c, const void* xbc, const float* weight, const float* bias, void* state,
                        void* x, void* B, void* C, int32_t* status) {
    tsv::ConvArgs a{};
    a.xbc = xbc; a.weight = weight; a.bias = bias; a.state = state; a.x = x; a.B = B; a.C = C; a.status = status;
    a.stride = c->row_stride;
    a.HP = s->n_heads * s->head_dim;
    a.GN = s->n_groups * s->d_state;
    a.silu = c->silu;
    return a;
}

// ---- the heads' norms and rotation
tsv_status check_rope(const tsv_attn_shape* s, const tsv_rope* r) {
    if (!r) return TSV_E_NULL;
    if (r->rot_dim < 0 || r->rot_dim % 2 != 0 || r->rot_dim > s->head_dim) return TSV_E_SHAPE;
    if (r->interleaved != 0 && r->interleaved != 1) return TSV_E_SHAPE;
    if (!isfinite(r->eps) || r->eps < 0) return TSV_E_SHAPE;
    return TSV_OK;
}
// elements between rows of H heads: at least one row, and not so many that a byte's number passes 2^63
bool stride_ok(int64_t stride, int H, int D) { return stride >= (int64_t)H * D && stride < (1LL << 28); }

tsv::RopeArgs rope_args(const tsv_attn_shape* s, const tsv_rope* r, const void* q, const void* k, const void* v,
                        const float* inv_freq, const float* qw, const float* kw, void* q_out, void* k_out, int rows) {
    tsv::RopeArgs a{};
    a.q = q; a.k = k; a.v = v; a.inv_freq = inv_freq; a.qw = q ? qw : nullptr; a.kw = k ? kw : nullptr;
    a.q_out = q ? q_out : nullptr; a.k_out = k_out;
    a.qs = q ? r->q_stride : 0; a.ks = k ? r->k_stride : 0; a.vs = v ? r->v_stride : 0;
    a.rows = rows; a.H = s->n_heads; a.Hk = s->n_kv_heads; a.D = s->head_dim;
    a.R = r->rot_dim; a.interleaved = r->interleaved; a.eps = r->eps;
    const int heads = (q ? s->n_heads : 0) + (k ? s->n_kv_heads : 0);
    a.heads = tsv::page_div(heads > 0 ? heads : 1);  // (a call without rows may have neither: nothing is divided then)
    a.key_heads = tsv::page_div(s->n_kv_heads);
    return a;
}

tsv_status check_prefill_attn(const tsv_attn_shape* s, int32_t window, int32_t sinks) {
    tsv_status st = check_attn(s, false);
    if (st != TSV_OK) return st;
    if (window < 0 || sinks < 0 || (window == 0 && sinks > 0)) return TSV_E_SHAPE;
    // rows of one key head are counted in 32 bits
    if ((long long)s->n_nodes * (s->n_heads / s->n_kv_heads) > kMaxRows || s->batch > kMaxRows) return TSV_E_UNSUPPORTED;
    if (tsv::attn_prefill_blocks(s) > kMaxBlocks) return TSV_E_UNSUPPORTED;
    return TSV_OK;
}

}  // namespace

extern "C" {

tsv_status tree_ssd_prefill_workspace(const tsv_seq_shape* s, uint64_t* bytes) {
    tsv_status st = check_seq(s);
    if (st != TSV_OK) return st;
    if (!bytes) return TSV_E_NULL;
    *bytes = tsv::prefill_workspace_bytes(s);
    return TSV_OK;
}

tsv_status tree_ssd_prefill(const tsv_seq_shape* s, const void* x, const void* dt, const float* A, const void* B,
                            const void* C, const float* D, float* h_inout, const int32_t* seq_start, void* y,
                            int32_t* seq_status, void* workspace, uint64_t workspace_bytes, void* stream) {
    uint64_t need = 0;
    tsv_status st = tree_ssd_prefill_workspace(s, &need);
    if (st != TSV_OK) return st;
    if (s->n_seqs == 0) return TSV_OK;
    if (!A || !D || !h_inout || !seq_start) return TSV_E_NULL;
    if (s->n_tokens > 0 && (!x || !dt || !B || !C || !y)) return TSV_E_NULL;
    if (need > 0 && (!workspace || workspace_bytes < need)) return TSV_E_NULL;
    if (need > 0 && (uintptr_t)workspace % 16 != 0) return TSV_E_SHAPE;
    tsv::PrefillArgs a{x, dt, A, B, C, D, h_inout, seq_start, y, s->n_seqs, s->n_tokens, s->n_heads, s->head_dim,
                       s->d_state, s->n_groups};
    if (tsv::prefill_blocks(s, tsv::prefill_states_vec(a, workspace)) > kMaxBlocks) return TSV_E_UNSUPPORTED;
    return result(tsv::launch_prefill(a, s, seq_status, need > 0 ? workspace : nullptr, (hipStream_t)stream));
}

tsv_status tree_ssd_step(const tsv_shape* s, const void* x, const void* dt, const float* A, const void* B, const void* C,
                         const float* D, float* h_inout, void* y, void* stream) {
    if (!s) return TSV_E_NULL;
    if (!dtype_ok(s->in_dtype)) return TSV_E_DTYPE;
    if (s->batch < 0 || s->n_nodes < 0 || s->n_nodes > 1) return TSV_E_SHAPE;
    if (s->n_heads < 1 || s->head_dim < 1 || s->d_state < 1 || s->n_groups < 1) return TSV_E_SHAPE;
    if (s->n_heads % s->n_groups != 0) return TSV_E_SHAPE;
    if (s->head_dim > kMaxDim || s->d_state > kMaxDim || s->n_heads > 0xffff) return TSV_E_UNSUPPORTED;
    if (tsv::step_blocks(s) > kMaxBlocks) return TSV_E_UNSUPPORTED;
    if (s->batch == 0 || s->n_nodes == 0) return TSV_OK;
    if (!x || !dt || !A || !B || !C || !D || !h_inout || !y) return TSV_E_NULL;
    tsv::StepArgs a{x, dt, A, B, C, D, h_inout, y, s->batch, s->n_heads, s->head_dim, s->d_state, s->n_groups};
    return result(tsv::launch_step(a, s->in_dtype == TSV_BF16, (hipStream_t)stream));
}

tsv_status tree_attn_verify_workspace(const tsv_attn_shape* s, uint64_t* bytes) {
    tsv_status st = check_attn(s, true);
    if (st != TSV_OK) return st;
    if (!bytes) return TSV_E_NULL;
    if (s->batch > 0 && s->n_nodes > 0 && tsv::attn_verify_blocks(s) > kMaxBlocks) return TSV_E_UNSUPPORTED;
    *bytes = s->batch > 0 && s->n_nodes > 0 ? tsv::attn_verify_workspace_bytes(s) : 0;
    return TSV_OK;
}

tsv_status tree_attn_verify(const tsv_attn_shape* s, const void* q, const void* k, const void* v, const int32_t* parent,
                            const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                            const int32_t* page_table, const int32_t* cache_len, void* o, int32_t* tree_status,
                            void* workspace, uint64_t workspace_bytes, void* stream) {
    uint64_t need = 0;
    tsv_status st = tree_attn_verify_workspace(s, &need);
    if (st != TSV_OK) return st;
    if (s->batch == 0 || s->n_nodes == 0) return TSV_OK;
    if (!q || !k || !v || !parent || !cache_len || !o) return TSV_E_NULL;
    if (s->max_pages > 0 && !page_table) return TSV_E_NULL;
    if (s->n_pages > 0 && (!k_cache || !v_cache || !scales_ok(s, k_scale, v_scale))) return TSV_E_NULL;
    if (need > 0 && (!workspace || workspace_bytes < need)) return TSV_E_NULL;
    if (need > 0 && (uintptr_t)workspace % 16 != 0) return TSV_E_SHAPE;
    const bool e4m3 = s->cache_dtype == TSV_E4M3;
    tsv::AttnArgs a{q, k, v, parent, k_cache, v_cache, e4m3 ? k_scale : nullptr, e4m3 ? v_scale : nullptr, page_table,
                    cache_len, o, tree_status, s->batch, s->n_nodes, s->n_heads, s->n_kv_heads, s->head_dim, s->n_pages,
                    s->page_size, s->max_pages, s->max_pages * s->page_size, s->scale * kLog2e,
                    tsv::page_div(s->page_size)};
    return result(tsv::launch_attn_verify(a, s, need > 0 ? workspace : nullptr, (hipStream_t)stream));
}

tsv_status tree_attn_commit(const tsv_attn_shape* s, const void* k, const void* v, const int32_t* parent,
                            const int32_t* accepted, const int32_t* accepted_len, int32_t max_path_len,
                            const int32_t* page_table, const int32_t* cache_len, void* k_cache, void* v_cache,
                            float* k_scale, float* v_scale, int32_t* tree_status, void* stream) {
    tsv_status st = check_attn(s, true);
    if (st != TSV_OK) return st;
    if (max_path_len < 0 || max_path_len > kMaxTree) return TSV_E_SHAPE;
    if (tsv::commit_blocks(s->batch, s->n_nodes, max_path_len) > kMaxBlocks) return TSV_E_UNSUPPORTED;
    if (s->batch == 0 || s->n_nodes == 0) return TSV_OK;
    if (!k || !v || !parent || !accepted_len || !cache_len) return TSV_E_NULL;
    if (max_path_len > 0 && !accepted) return TSV_E_NULL;
    if (s->max_pages > 0 && !page_table) return TSV_E_NULL;
    if (s->n_pages > 0 && (!k_cache || !v_cache || !scales_ok(s, k_scale, v_scale))) return TSV_E_NULL;
    tsv::CacheWriteArgs a = write_args(s, k, v, page_table, cache_len, k_cache, v_cache, k_scale, v_scale, tree_status);
    a.parent = parent;
    a.accepted = accepted;
    a.accepted_len = accepted_len;
    a.Lmax = max_path_len;
    return result(tsv::launch_cache_write(a, s->in_dtype == TSV_BF16, s->cache_dtype == TSV_E4M3, (hipStream_t)stream));
}

tsv_status tree_attn_append(const tsv_attn_shape* s, const void* k, const void* v, const int32_t* seq_start,
                            const int32_t* page_table, const int32_t* cache_len, void* k_cache, void* v_cache,
                            float* k_scale, float* v_scale, int32_t* seq_status, void* stream) {
    tsv_status st = check_attn(s, false);
    if (st != TSV_OK) return st;
    if (tsv::append_blocks(s->n_nodes, s->batch) > kMaxBlocks) return TSV_E_UNSUPPORTED;
    if (s->batch == 0) return TSV_OK;
    if (!seq_start || !cache_len) return TSV_E_NULL;
    if (s->n_nodes > 0 && (!k || !v)) return TSV_E_NULL;
    if (s->max_pages > 0 && !page_table) return TSV_E_NULL;
    if (s->n_pages > 0 && (!k_cache || !v_cache || !scales_ok(s, k_scale, v_scale))) return TSV_E_NULL;
    tsv::CacheWriteArgs a = write_args(s, k, v, page_table, cache_len, k_cache, v_cache, k_scale, v_scale, seq_status);
    a.seq_start = seq_start;
    return result(tsv::launch_cache_write(a, s->in_dtype == TSV_BF16, s->cache_dtype == TSV_E4M3, (hipStream_t)stream));
}

tsv_status tree_ssd_conv_prefill(const tsv_seq_shape* s, const tsv_conv* c, const void* xbc, const float* weight,
                                 const float* bias, void* state_inout, const int32_t* seq_start, void* x, void* B, void* C,
                                 int32_t* seq_status, void* stream) {
    tsv_status st = check_conv(s, c);
    if (st != TSV_OK) return st;
    if (s->n_seqs == 0) return TSV_OK;
    if (!weight || !state_inout || !seq_start) return TSV_E_NULL;
    if (s->n_tokens > 0 && (!xbc || !x || !B || !C)) return TSV_E_NULL;
    tsv::ConvArgs a = conv_args(s, c, xbc, weight, bias, state_inout, x, B, C, seq_status);
    a.seq_start = seq_start;
    a.n = s->n_seqs;
    a.rows = s->n_tokens;
    return result(tsv::launch_conv(tsv::kConvPrefill, a, c->width, s->in_dtype == TSV_BF16, (hipStream_t)stream));
}

tsv_status tree_ssd_conv_step(const tsv_shape* s, const tsv_conv* c, const void* xbc, const float* weight, const float* bias,
                              void* state_inout, void* x, void* B, void* C, void* stream) {
    tsv_status st = check_conv(tsv::kConvStep, s, c);
    if (st != TSV_OK) return st;
    if (s->batch == 0 || s->n_nodes == 0) return TSV_OK;
    if (!xbc || !weight || !state_inout || !x || !B || !C) return TSV_E_NULL;
    tsv::ConvArgs a = conv_args(s, c, xbc, weight, bias, state_inout, x, B, C, nullptr);
    a.n = s->batch;
    a.rows = 1;
    return result(tsv::launch_conv(tsv::kConvStep, a, c->width, s->in_dtype == TSV_BF16, (hipStream_t)stream));
}

tsv_status tree_ssd_conv_verify(const tsv_shape* s, const tsv_conv* c, const void* xbc, const float* weight,
                                const float* bias, const void* state, const int32_t* parent, void* x, void* B, void* C,
                                int32_t* tree_status, void* stream) {
    tsv_status st = check_conv(tsv::kConvVerify, s, c);
    if (st != TSV_OK) return st;
    if (s->batch == 0 || s->n_nodes == 0) return TSV_OK;
    if (!xbc || !weight || !state || !parent || !x || !B || !C) return TSV_E_NULL;
    tsv::ConvArgs a = conv_args(s, c, xbc, weight, bias, const_cast<void*>(state), x, B, C, tree_status);
    a.parent = parent;
    a.n = s->batch;
    a.rows = s->n_nodes;
    return result(tsv::launch_conv(tsv::kConvVerify, a, c->width, s->in_dtype == TSV_BF16, (hipStream_t)stream));
}

tsv_status tree_ssd_conv_commit(const tsv_shape* s, const tsv_conv* c, const void* xbc, void* state_inout,
                                const int32_t* parent, const int32_t* accepted, const int32_t* accepted_len,
                                int32_t max_path_len, int32_t* tree_status, void* stream) {
    tsv_status st = check_conv(tsv::kConvCommit, s, c);
    if (st != TSV_OK) return st;
    if (max_path_len < 0 || max_path_len > kMaxTree) return TSV_E_SHAPE;
    if (s->batch == 0 || s->n_nodes == 0) return TSV_OK;
    if (!xbc || !state_inout || !parent || !accepted_len) return TSV_E_NULL;
    if (max_path_len > 0 && !accepted) return TSV_E_NULL;
    tsv::ConvArgs a = conv_args(s, c, xbc, nullptr, nullptr, state_inout, nullptr, nullptr, nullptr, tree_status);
    a.parent = parent;
    a.accepted = accepted;
    a.accepted_len = accepted_len;
    a.Lmax = max_path_len;
    a.n = s->batch;
    a.rows = s->n_nodes;
    return result(tsv::launch_conv(tsv::kConvCommit, a, c->width, s->in_dtype == TSV_BF16, (hipStream_t)stream));
}

tsv_status tree_attn_rope(const tsv_attn_shape* s, const tsv_rope* r, const void* q, const void* k, const int32_t* position,
                          const float* inv_freq, const float* q_weight, const float* k_weight, void* q_out, void* k_out,
                          void* stream) {
    tsv_status st = check_attn(s, false);
    if (st == TSV_OK) st = check_rope(s, r);
    if (st != TSV_OK) return st;
    const long long rows = (long long)s->batch * s->n_nodes;
    if (rows > kMaxRows || tsv::rope_blocks((int)rows, false, 0) > kMaxBlocks) return TSV_E_UNSUPPORTED;
    if (rows == 0) return TSV_OK;
    if ((!q && !k) || (q && !q_out) || (k && !k_out) || !position || (r->rot_dim > 0 && !inv_freq)) return TSV_E_NULL;
    if ((q && !stride_ok(r->q_stride, s->n_heads, s->head_dim)) || (k && !stride_ok(r->k_stride, s->n_kv_heads, s->head_dim)))
        return TSV_E_SHAPE;
    tsv::RopeArgs a = rope_args(s, r, q, k, nullptr, inv_freq, q_weight, k_weight, q_out, k ? k_out : nullptr, (int)rows);
    a.position = position;
    return result(tsv::launch_rope(a, nullptr, s->in_dtype == TSV_BF16, false, (hipStream_t)stream));
}

tsv_status tree_attn_append_rope(const tsv_attn_shape* s, const tsv_rope* r, const void* q, const void* k, const void* v,
                                 const int32_t* seq_start, const float* inv_freq, const float* q_weight,
                                 const float* k_weight, const int32_t* page_table, const int32_t* cache_len, void* q_out,
                                 void* k_cache, void* v_cache, float* k_scale, float* v_scale, int32_t* seq_status,
                                 void* stream) {
    tsv_status st = check_attn(s, false);
    if (st == TSV_OK) st = check_rope(s, r);
    if (st != TSV_OK) return st;
    if (s->n_nodes > kMaxRows || s->batch > kMaxRows || tsv::rope_blocks(s->n_nodes, true, s->batch) > kMaxBlocks) return TSV_E_UNSUPPORTED;
    if (s->batch == 0) return TSV_OK;
    if (!seq_start || !cache_len || (r->rot_dim > 0 && !inv_freq)) return TSV_E_NULL;
    if (s->n_nodes > 0 && (!k || !v || (q && !q_out))) return TSV_E_NULL;
    if (s->max_pages > 0 && !page_table) return TSV_E_NULL;
    if (s->n_pages > 0 && (!k_cache || !v_cache || !scales_ok(s, k_scale, v_scale))) return TSV_E_NULL;
    if ((q && !stride_ok(r->q_stride, s->n_heads, s->head_dim)) || !stride_ok(r->k_stride, s->n_kv_heads, s->head_dim) ||
        !stride_ok(r->v_stride, s->n_kv_heads, s->head_dim))
        return TSV_E_SHAPE;
    tsv::CacheWriteArgs c = write_args(s, k, v, page_table, cache_len, k_cache, v_cache, k_scale, v_scale, seq_status);
    c.seq_start = seq_start;
    tsv::RopeArgs a = rope_args(s, r, q, k, v, inv_freq, q_weight, k_weight, q_out, nullptr, s->n_nodes);
    return result(tsv::launch_rope(a, &c, s->in_dtype == TSV_BF16, s->cache_dtype == TSV_E4M3, (hipStream_t)stream));
}

tsv_status tree_attn_prefill_workspace(const tsv_attn_shape* s, uint64_t* bytes) {
    tsv_status st = check_prefill_attn(s, 0, 0);
    if (st != TSV_OK) return st;
    if (!bytes) return TSV_E_NULL;
    *bytes = s->batch > 0 && s->n_nodes > 0 ? tsv::attn_prefill_workspace_bytes(s) : 0;
    return TSV_OK;
}

tsv_status tree_attn_prefill(const tsv_attn_shape* s, int32_t window, int32_t sinks, const void* q, const int32_t* seq_start,
                             const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                             const int32_t* page_table, const int32_t* cache_len, void* o, int32_t* seq_status,
                             void* workspace, uint64_t workspace_bytes, void* stream) {
    tsv_status st = check_prefill_attn(s, window, sinks);
    uint64_t need = 0;
    if (st == TSV_OK) st = tree_attn_prefill_workspace(s, &need);
    if (st != TSV_OK) return st;
    if (s->batch == 0) return TSV_OK;
    if (!seq_start || !cache_len) return TSV_E_NULL;
    if (s->n_nodes > 0 && (!q || !o)) return TSV_E_NULL;
    if (s->max_pages > 0 && !page_table) return TSV_E_NULL;
    if (s->n_pages > 0 && (!k_cache || !v_cache || !scales_ok(s, k_scale, v_scale))) return TSV_E_NULL;
    if (need > 0 && (!workspace || workspace_bytes < need)) return TSV_E_NULL;
    if (need > 0 && (uintptr_t)workspace % 16 != 0) return TSV_E_SHAPE;
    const bool e4m3 = s->cache_dtype == TSV_E4M3;
    tsv::ChunkArgs a{q, seq_start, k_cache, v_cache, e4m3 ? k_scale : nullptr, e4m3 ? v_scale : nullptr, page_table,
                     cache_len, o, seq_status, s->batch, s->n_nodes, s->n_heads, s->n_kv_heads, s->head_dim, s->n_pages,
                     s->page_size, s->max_pages, s->max_pages * s->page_size, window ? window : 0x7fffffff, sinks,
                     s->scale * kLog2e, tsv::page_div(s->page_size)};
    return result(tsv::launch_attn_prefill(a, s, need > 0 ? workspace : nullptr, (hipStream_t)stream));
}

}  // extern "C"
