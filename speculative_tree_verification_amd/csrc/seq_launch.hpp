// seq_launch.hpp -- the kernels of the calls around the tree, as api_seq.hip
// launches them: the prompt scan, the single-token step and the paged cache.
#pragma once

#include "launch.hpp"

namespace tsv {

struct PageDiv {  // n / page_size by a product (attn_common.hpp)
    uint32_t mul;
    int shift;
};

// ---- sequences around the tree
struct StepArgs {
    const void* x;
    const void* dt;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    float* h;
    void* y;
    int batch, H, P, N, G;
};
long long step_blocks(const tsv_shape* s);  // work-groups
hipError_t launch_step(const StepArgs& a, bool bf16, hipStream_t stream);

struct PrefillArgs {
    const void* x;
    const void* dt;
    const float* A;
    const void* B;
    const void* C;
    const float* D;
    float* h;
    const int32_t* seq_start;
    void* y;
    int n_seqs, n_tokens, H, P, N, G;
};
uint64_t prefill_workspace_bytes(const tsv_seq_shape* s);
// whether the states are taken 4 elements at a time by the combining pass
bool prefill_states_vec(const PrefillArgs& a, const void* workspace);
// most work-groups of any launch of the prompt scan
long long prefill_blocks(const tsv_seq_shape* s, bool states_vec);
hipError_t launch_prefill(const PrefillArgs& a, const tsv_seq_shape* s, int32_t* status, void* workspace, hipStream_t stream);

// ---- the paged cache of attention layers
struct CacheWriteArgs {
    const void* k;
    const void* v;
    const int32_t* parent;        // commit
    const int32_t* accepted;      // commit
    const int32_t* accepted_len;  // commit
    const int32_t* seq_start;     // append; NULL: commit
    const int32_t* page_table;
    const int32_t* cache_len;
    void* k_cache;
    void* v_cache;
    float* k_scale;
    float* v_scale;
    int32_t* status;
    int batch, T, Lmax, Hk, D, n_pages, page_size, max_pages;
    PageDiv div, heads;  // by page_size; by 2 Hk
};
// work-groups: of accepted paths; of n_rows rows and, with a status, its items
long long commit_blocks(int batch, int T, int max_path_len);
long long append_blocks(int n_rows, int items);
hipError_t launch_cache_write(const CacheWriteArgs& a, bool bf16, bool e4m3, hipStream_t stream);

// ---- heads' norms and rotation (attn_rope.hip)
struct RopeArgs {
    const void* q;  // NULL: no queries
    const void* k;  // NULL: no keys (nor values)
    const void* v;
    const int32_t* position;  // rope; append: the cache's
    const float* inv_freq;
    const float* qw;  // NULL: no norm
    const float* kw;
    void* q_out;
    void* k_out;
    long long qs, ks, vs;  // elements between rows
    int rows, H, Hk, D, R, interleaved;
    float eps;
    PageDiv heads, key_heads;  // by a row's heads of q and k, and by those of k
};
long long rope_blocks(int rows, bool append, int items);  // work-groups, with the items' status
// c: into the cache; NULL: to k_out
hipError_t launch_rope(const RopeArgs& a, const CacheWriteArgs* c, bool bf16, bool e4m3, hipStream_t stream);

// ---- the short convolution (conv.hip)
struct ConvArgs {
    const void* xbc;
    const float* weight;  // [C][W]
    const float* bias;    // NULL: 0
    void* state;
    const int32_t* seq_start;     // prefill
    const int32_t* parent;        // verify, commit
    const int32_t* accepted;      // commit
    const int32_t* accepted_len;  // commit
    void* x;
    void* B;
    void* C;
    int32_t* status;
    long long stride;  // elements between rows of xbc
    int n, rows;       // prefill: sequences, packed rows; otherwise items, nodes of each
    int HP, GN, Lmax;
    int silu;
};
enum ConvKind { kConvPrefill, kConvStep, kConvVerify, kConvCommit };
long long conv_blocks(ConvKind kind, int n, int rows, int HP, int GN);  // most work-groups
hipError_t launch_conv(ConvKind kind, const ConvArgs& a, int width, bool bf16, hipStream_t stream);

struct AttnArgs {
    const void* q;
    const void* k;
    const void* v;
    const int32_t* parent;
    const void* k_cache;
    const void* v_cache;
    const float* k_scale;  // NULL: not an 8-bit cache
    const float* v_scale;
    const int32_t* page_table;
    const int32_t* cache_len;
    void* o;
    int32_t* status;
    int batch, T, H, Hk, D, n_pages, page_size, max_pages, room;
    float scale_log2;  // scale * log2(e)
    PageDiv div;
};
uint64_t attn_verify_workspace_bytes(const tsv_attn_shape* s);
// most work-groups of any launch of the attention
long long attn_verify_blocks(const tsv_attn_shape* s);
hipError_t launch_attn_verify(const AttnArgs& a, const tsv_attn_shape* s, void* workspace, hipStream_t stream);

// packed rows over the cache: T rows, item b's from seq_start[b] on
struct ChunkArgs {
    const void* q;
    const int32_t* seq_start;
    const void* k_cache;
    const void* v_cache;
    const float* k_scale;  // NULL: not an 8-bit cache
    const float* v_scale;
    const int32_t* page_table;
    const int32_t* cache_len;
    void* o;
    int32_t* status;
    int batch, T, H, Hk, D, n_pages, page_size, max_pages, room;
    int window, sinks;  // window: 0x7fffffff where there is none
    float scale_log2;
    PageDiv div;
};
uint64_t attn_prefill_workspace_bytes(const tsv_attn_shape* s);
long long attn_prefill_blocks(const tsv_attn_shape* s);  // most work-groups of any launch
hipError_t launch_attn_prefill(const ChunkArgs& a, const tsv_attn_shape* s, void* workspace, hipStream_t stream);

}  // namespace tsv
