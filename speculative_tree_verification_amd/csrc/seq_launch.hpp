// seq_launch.hpp -- the kernels of the calls around the tree, as api_seq.hip
// launches them: the prompt scan, the single-token step and the paged cache.
#pragma once

#include "launch.hpp"

namespace tsv {

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
struct PageDiv {  // n / page_size by a product (attn_common.hpp)
    uint32_t mul;
    int shift;
};
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

}  // namespace tsv
