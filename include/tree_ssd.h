/*
 * tree_ssd.h -- C ABI of libtree_ssd.so: packed-tree verification and commit
 * for one Mamba2/SSD layer on AMD MI355X (gfx950).
 *
 * Method: "STree: Speculative Tree Decoding for Hybrid State Space Models"
 * (atlas.scime.ai summary, sections "Problem" and "Approach"; mlsanity
 * abstract). A draft token tree is packed into one sequence of T nodes, node 0
 * the root and every parent listed before its children. One pass gives every
 * node the exact output the SSM recurrence would give on that node's root path
 * alone. The tree mask L (ancestor-or-self) accumulates the per-token log
 * decays along root paths ("A_tree = L log A", read with log A_j = dt_j * A_h,
 * the log of the discrete transition exp(dt_j * A_h)). Commit ("activation
 * replay for state backtracking") rebuilds only the accepted path's final
 * state from the retained inputs; no per-node state is ever stored.
 *
 * Per batch item b and head h (group g = h / (H / G)), with the state stored
 * as H[p][n] (P x N, n fastest):
 *   H_i = exp(cum_i) h0 + sum_{j on path(i)} exp(cum_i - cum_j) dt_j x_j (outer) B_j
 *   y_i = H_i C_i + D_h x_i,      cum_i = sum_{j on path(i)} dt_j A_h
 * which is the recurrence H <- exp(dt A) H + dt x (outer) B, y = H C + D x run
 * from h0 along the root path of node i.
 *
 * Conventions shared by every entry point
 *   - All tensor pointers are DEVICE pointers owned by the caller, contiguous
 *     row-major. The library allocates nothing, keeps no state between calls,
 *     and is reentrant, with one exception: tree_ssd_commit_layers_static
 *     keeps its layer table in a fixed device array of the library's (one per
 *     GPU), so its calls that overlap on one GPU race. Work is enqueued on
 *     `stream` (a hipStream_t; NULL means
 *     the null stream) without synchronising; results are ready when the
 *     stream reaches that point.
 *   - Host-detectable errors (NULL pointers, bad sizes, bad dtype) return a
 *     tsv_status other than TSV_OK before anything is enqueued.
 *   - Data-dependent errors are reported per batch item in device memory
 *     tree_status[b] (a bit set, see TSV_ST_*). The outputs of an item with any
 *     bit set are left bitwise untouched. tree_status may be NULL (no report;
 *     invalid items are still skipped).
 *   - Nodes are limited to T <= 1024. bf16 inputs with head_dim 64 and
 *     d_state 64 or 128 take MFMA verify kernels at every tree size; other
 *     shapes and fp32 inputs take plain fp32 kernels (same results, lower
 *     throughput).
 *   - The launch runs on the device current to the calling thread.
 */
#ifndef TREE_SSD_H
#define TREE_SSD_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* dtype of x, dt, B, C and y */
typedef enum { TSV_F32 = 0, TSV_BF16 = 1 } tsv_dtype;

/* Return codes */
typedef enum {
    TSV_OK = 0,
    TSV_E_NULL = 1,        /* a required pointer is NULL */
    TSV_E_SHAPE = 2,       /* a size is out of range, H % G != 0, or T > 1024 */
    TSV_E_DTYPE = 3,       /* in_dtype is not a tsv_dtype */
    TSV_E_UNSUPPORTED = 4, /* the size combination has no kernel (this includes
                              head_dim or d_state above 256 and more than
                              65535 heads) */
    TSV_E_LAUNCH = 5       /* the HIP launch failed (see hipGetLastError) */
} tsv_status;

/* Per-item status bits written to tree_status[b] */
#define TSV_ST_BAD_ROOT 1   /* parent[b][0] != -1 */
#define TSV_ST_BAD_PARENT 2 /* some parent[b][i] (i >= 1) is not in [0, i) */
#define TSV_ST_BAD_PATH 4   /* accepted path: len not in [0, max_path_len]
                               or above T, first node not 0, an index not in
                               [0, T), or a node whose parent is not the
                               previous entry */

/* Flags (tsv_shape.flags) */
#define TSV_FLAG_FORCE_GENERIC 1 /* use the plain VALU verify kernel even where
                                    the MFMA kernel applies (testing aid) */
#define TSV_FLAG_FORCE_WIDE 2    /* use the wide-tree MFMA verify kernel for any
                                    tree size it supports (testing / tuning aid) */
#define TSV_FLAG_FORCE_SMALL 4   /* trees of at most 16 nodes: use the 64-node
                                    small-tree MFMA kernel instead of the one-wave
                                    tiny-tree kernel (testing / tuning aid) */

typedef struct {
    int32_t batch;           /* Bt >= 0 (0: nothing to do) */
    int32_t n_nodes;         /* T in [0, 1024] (0: nothing to do) */
    int32_t n_heads;         /* H >= 1 */
    int32_t head_dim;        /* P >= 1 */
    int32_t d_state;         /* N >= 1 */
    int32_t n_groups;        /* G >= 1, H % G == 0; head h uses group h / (H/G) */
    int32_t in_dtype;        /* tsv_dtype of x, dt, B, C, y */
    int32_t flags;           /* TSV_FLAG_* (0 = automatic choice) */
    int32_t heads_per_block; /* launch hint: heads one work-group handles for the
                                MFMA verify kernel; 0 = automatic. Must divide
                                H / G when given. The tiny-tree kernel
                                (T <= 16) takes one head_dim slice per
                                work-group and ignores it. */
} tsv_shape;

/*
 * tree_ssd_verify -- every node's output of one SSD layer over a packed tree
 * (the summary's section "Approach": log decays summed along ancestor paths let
 * one pass over the packed tree give each node the output of its own root path,
 * exactly).
 *
 *   x      [Bt][T][H][P]   in_dtype   token inputs
 *   dt     [Bt][T][H]      in_dtype   step sizes, already positive (after any
 *                                     softplus / bias of the caller)
 *   A      [H]             float      per-head decay rate (normally < 0)
 *   B, C   [Bt][T][G][N]   in_dtype   input / output projections
 *   D      [H]             float      skip weight
 *   h0     [Bt][H][P][N]   float      state before the root (read only)
 *   parent [Bt][T]         int32      parent[b][0] = -1, parent[b][i] in [0, i)
 *   y      [Bt][T][H][P]   in_dtype   output (bf16 results rounded to nearest
 *                                     even from fp32 accumulators)
 *   tree_status [Bt]       int32      optional; set to bits 1|2 of the item's tree
 *
 * Arithmetic: fp32 accumulation throughout. For bf16 inputs with P == 64 and
 * N in {64, 128} the h0 read-out C h0^T runs on bf16 MFMA with h0 split into a
 * bf16 high and low part (about 16 significant bits). For trees of more than
 * 64 nodes the masked decay weights of the intra-tree term are rounded once to
 * bf16 for the bf16 dot-product instruction, except the node's own weight
 * (which carries D) and its parent's, which keep about 16 bits. Other inputs
 * and shapes use fp32 arithmetic on the (exact) input values.
 */
tsv_status tree_ssd_verify(const tsv_shape* s, const void* x, const void* dt, const float* A,
                           const void* B, const void* C, const float* D, const float* h0,
                           const int32_t* parent, void* y, int32_t* tree_status, void* stream);

/*
 * tree_ssd_commit -- overwrite h0 with the state at the end of the accepted
 * root path by replaying the path's tokens (the summary's section "Approach":
 * state is restored from the retained activations rather than from per-node
 * snapshots), using the same inputs the verify call read:
 *   H' = exp(cum_l) h0 + sum_k exp(cum_l - cum_{j_k}) dt_{j_k} x_{j_k} (outer) B_{j_k}
 * for the path j_0 = 0, ..., j_{len-1} = l. len == 0 leaves h0 unchanged.
 *
 *   x, dt, A, B, parent   as for tree_ssd_verify (only path rows are read)
 *   h0_inout [Bt][H][P][N] float   read, then overwritten in place
 *   accepted [Bt][max_path_len] int32  root-path node list of each item
 *   accepted_len [Bt]      int32   number of valid entries of each row
 *   max_path_len           >= 0    row length of `accepted` (1 <= ... <= 1024
 *                                  when Bt > 0; 0 allowed with all len == 0)
 *   tree_status [Bt]       int32   optional; bits 1|2|4 of the item
 *
 * Not idempotent: a second call advances the state again. It must be ordered
 * after every verify that reads the same h0 (same stream, or an event).
 */
tsv_status tree_ssd_commit(const tsv_shape* s, const void* x, const void* dt, const float* A,
                           const void* B, float* h0_inout, const int32_t* parent,
                           const int32_t* accepted, const int32_t* accepted_len,
                           int32_t max_path_len, int32_t* tree_status, void* stream);

/* One layer's operands for tree_ssd_commit_layers: device pointers with the
 * layouts of tree_ssd_commit (x, dt, B in in_dtype; A float; h0 float). */
typedef struct {
    const void* x;   /* [Bt][T][H][P] */
    const void* dt;  /* [Bt][T][H]    */
    const float* A;  /* [H]           */
    const void* B;   /* [Bt][T][G][N] */
    float* h0_inout; /* [Bt][H][P][N] read, then overwritten in place */
} tsv_commit_layer;

/*
 * tree_ssd_commit_layers -- tree_ssd_commit for n_layers layers of one model
 * step in a single launch. All layers share the shape, the draft tree and the
 * accepted path: one decoding step accepts the same tokens in every layer
 * (the summary's section "Approach": every layer's state is rebuilt from its
 * own retained inputs along that path). Once the path is known the layers are
 * independent, so their commits need not run one after another; each layer's
 * result is exactly that of tree_ssd_commit on its operands.
 *
 *   n_layers    >= 0    number of entries of `layers` (0: nothing to do)
 *   layers      device array [n_layers] of tsv_commit_layer, owned by the
 *               caller, read by the kernel (so it must stay valid until the
 *               stream passes this call); no two entries may share h0_inout
 *   parent, accepted, accepted_len, max_path_len
 *               as for tree_ssd_commit, shared by all layers
 *   tree_status [Bt]    optional; written once per item (bits 1|2|4)
 *
 * An item whose tree or path is invalid keeps h0 untouched in every layer.
 * Returns TSV_E_NULL for a NULL `layers` with n_layers > 0 and TSV_E_SHAPE for
 * n_layers < 0; the pointers inside the table are not checked on the host.
 */
tsv_status tree_ssd_commit_layers(const tsv_shape* s, int32_t n_layers,
                                  const tsv_commit_layer* layers, const int32_t* parent,
                                  const int32_t* accepted, const int32_t* accepted_len,
                                  int32_t max_path_len, int32_t* tree_status, void* stream);

/* Most layers tree_ssd_commit_layers_static takes in one call. */
#define TSV_STATIC_MAX_LAYERS 1024

/*
 * tree_ssd_commit_layers_static -- tree_ssd_commit_layers for callers that
 * cannot allocate device memory: code under HIP graph capture, serving loops
 * that must not call hipMalloc, harnesses that forbid it. The layer table is
 * passed in HOST memory; the call stages it into a fixed device array that
 * the library holds for the life of the process (TSV_STATIC_MAX_LAYERS
 * entries of 40 bytes, one copy per GPU, its address looked up on the first
 * call made on that GPU) and then runs the commit kernel of
 * tree_ssd_commit_layers on it, so the results are bitwise those of that
 * call. Nothing is allocated or freed.
 *
 *   layers_host  host array [n_layers] of tsv_commit_layer (device pointers
 *                inside, as for tree_ssd_commit_layers); read during the
 *                call, which passes it to the GPU as kernel arguments (64
 *                entries per staging launch), so it may be freed or reused as
 *                soon as the call returns
 *   every other argument as for tree_ssd_commit_layers.
 *
 * Returns TSV_E_UNSUPPORTED for n_layers > TSV_STATIC_MAX_LAYERS, TSV_E_NULL
 * for a NULL layers_host with n_layers > 0, TSV_E_LAUNCH if the device array
 * cannot be resolved, and otherwise what tree_ssd_commit_layers returns.
 * Every call on one GPU shares that GPU's array and overwrites the entries it
 * uses: two calls whose work overlaps on one GPU (different streams, no
 * ordering between them) race. Calls ordered on one stream do not.
 */
tsv_status tree_ssd_commit_layers_static(const tsv_shape* s, int32_t n_layers,
                                         const tsv_commit_layer* layers_host, const int32_t* parent,
                                         const int32_t* accepted, const int32_t* accepted_len,
                                         int32_t max_path_len, int32_t* tree_status, void* stream);

/*
 * tree_gdn_verify -- every node's output of one gated-delta-rule layer over a
 * packed tree ("TreeWY: Speculative Verification for Gated DeltaNet Hybrids",
 * fugumt page, abstract: one triangular solve over the tree gives every draft
 * node's output, and a small pseudo-value matrix is kept for commit). Per head
 * the state S (dv x dk, stored [p][n]) follows
 *   S <- exp(g) S (I - beta k k^T) + beta v k^T,   o = S q
 * from S0 along each node's root path. With G_i the sum of g over that path,
 * the pseudo-values e solve
 *   e_i + beta_i sum_{j strict ancestor of i} exp(G_i - G_j) (k_i . k_j) e_j
 *       = beta_i (v_i - exp(G_i) S0 k_i)
 * and o_i = exp(G_i) S0 q_i + sum_{j on path(i)} exp(G_i - G_j) (q_i . k_j) e_j.
 *
 * The shape uses tsv_shape with head_dim = dv, d_state = dk, n_groups = 1;
 * in_dtype is the type of q, k, v and o: TSV_F32 or TSV_BF16 (bf16 bit
 * patterns); g, beta, S0 and e are fp32 either way. n_nodes <= 256, dk and
 * dv <= 128 (TSV_E_UNSUPPORTED otherwise). Trees of 65 to 256 nodes take a
 * second kernel, which holds the tree's pair tables in LDS: a tree with more
 * than 4096 ancestor-or-self pairs (the sum over nodes of depth + 1) sets
 * status bit 8 and is left untouched.
 *   q, k   [Bt][T][H][dk]   queries and keys (keys normally of unit length)
 *   v      [Bt][T][H][dv]   values
 *   g      [Bt][T][H]       log gate (<= 0)
 *   beta   [Bt][T][H]       step in [0, 1]
 *   S0     [Bt][H][dv][dk]  state before the root (read only)
 *   parent [Bt][T]          as for tree_ssd_verify
 *   o      [Bt][T][H][dv]   output (in_dtype; bf16 rounded to nearest even)
 *   e      [Bt][T][H][dv]   optional output, fp32: the pseudo-values, input of commit
 *   tree_status [Bt]        optional; bits 1|2, and 8 as above
 * fp32 arithmetic throughout (bf16 inputs are exact in it).
 */
tsv_status tree_gdn_verify(const tsv_shape* s, const void* q, const void* k, const void* v,
                           const float* g, const float* beta, const float* S0,
                           const int32_t* parent, void* o, float* e, int32_t* tree_status,
                           void* stream);

/*
 * tree_gdn_commit -- overwrite S0 with the state at the end of each item's
 * accepted root path from the pseudo-values tree_gdn_verify wrote:
 *   S' = exp(G_l) S0 + sum_{j on the path} exp(G_l - G_j) e_j k_j^T.
 * k (in_dtype), g, parent as for tree_gdn_verify; e (fp32) from it; accepted, accepted_len,
 * max_path_len and tree_status (bits 1|2|4) as for tree_ssd_commit. len == 0
 * leaves S0 unchanged; invalid items leave it untouched. Past 64 nodes,
 * max_path_len must be at most 128 (TSV_E_UNSUPPORTED otherwise): the path's
 * rows are staged whole in LDS.
 */
tsv_status tree_gdn_commit(const tsv_shape* s, const void* k, const float* g, const float* e,
                           float* S0_inout, const int32_t* parent, const int32_t* accepted,
                           const int32_t* accepted_len, int32_t max_path_len, int32_t* tree_status,
                           void* stream);

/*
 * tree_ssd_accept_greedy -- the accepted root path of each verified tree at
 * temperature 0, the input of tree_ssd_commit. The target model's choice
 * after node i is target_tokens[i] (its argmax next token); a child c of an
 * accepted node i is accepted when draft_tokens[c] == target_tokens[i]
 * ("TreeSpark: Adaptive Draft Trees Accelerate Speculative Decoding by
 * 8-14%", section on the lossless guarantee: the target model keeps or rejects
 * draft tokens, and a draft tree offers several candidate paths checked in one
 * pass). The root (node 0, the token the tree grows from) is always accepted.
 * The path is the deepest root path whose every non-root node is accepted; a
 * tree without repeated sibling tokens has at most one, and with repeats the
 * deepest accepted node of smallest index ends the path.
 *
 *   parent        [Bt][T] int32   as for tree_ssd_verify
 *   draft_tokens  [Bt][T] int32   token of each node (node 0: the root token)
 *   target_tokens [Bt][T] int32   target model's greedy next token after each node
 *   max_path_len  in [1, 1024]    row length of `accepted`
 *   accepted      [Bt][max_path_len] int32  output: node indices of the path,
 *                                 root first, cut after max_path_len entries;
 *                                 entries past the length are -1
 *   accepted_len  [Bt] int32      output: entries of the path kept (>= 1)
 *   next_token    [Bt] int32      optional output: target token after the last
 *                                 kept node (the token the next step starts from)
 *   tree_status   [Bt] int32      optional; bits 1|2 of the item's tree
 * Invalid items leave accepted, accepted_len and next_token untouched.
 */
tsv_status tree_ssd_accept_greedy(int32_t batch, int32_t n_nodes, const int32_t* parent,
                                  const int32_t* draft_tokens, const int32_t* target_tokens,
                                  int32_t max_path_len, int32_t* accepted, int32_t* accepted_len,
                                  int32_t* next_token, int32_t* tree_status, void* stream);

#define TSV_ST_BAD_TOKEN 16 /* a non-root draft token is outside [0, vocab) */

/*
 * tree_ssd_accept_stochastic -- the accepted root path of each verified tree
 * at temperature > 0: multi-step speculative sampling over the tree with
 * siblings drawn without replacement ("STree: Speculative Tree Decoding for
 * Hybrid State-Space Models", atlas.scime.ai summary, measured-effects table:
 * multi-step speculative sampling; "TreeSpark: Adaptive Draft Trees
 * Accelerate Speculative Decoding by 8-14%", section on the lossless
 * guarantee: siblings sampled without replacement and rejected tokens
 * resampled from the residual, recursively). The produced tokens follow the
 * target's distribution whatever the draft's.
 *
 * Starting at the root with residual r = p_target[root], the children of the
 * current node u are tested in increasing index. The k-th child's token t was
 * drawn from d = q_draft[u] without the earlier children's tokens, divided by
 * m = 1 - (their draft mass) (d = 0 when m <= 0 or t repeats an earlier
 * sibling's token). It is accepted when u_node[c] * d[t] < r[t]; an accepted
 * child becomes u. A rejection replaces r by max(r - d, 0) divided by its mass
 * (r is kept when that mass is 0). When no child is accepted, next_token is
 * the first token whose running sum of r exceeds u_final times r's total
 * (-1 if r has no mass). The path is cut after max_path_len nodes; a child
 * accepted below the cut gives next_token instead (its token is a draw from
 * the cut node's target). Decisions are taken in fp64; sums over the
 * vocabulary are taken in an order of the kernel's own, so a decision can
 * differ from a left-to-right evaluation only within fp64 rounding of its
 * threshold.
 *
 *   n_nodes       in [1, 1024]; vocab >= 1
 *   parent        [Bt][T] int32   as for tree_ssd_verify
 *   draft_tokens  [Bt][T] int32   token of each node (node 0's is not used)
 *   p_target      [Bt][T][vocab] float32  target distribution of the token
 *                                 after each node (rows sum to 1)
 *   q_draft       [Bt][T][vocab] float32  draft distribution the children of
 *                                 each node drew their tokens from, one after
 *                                 another without replacement, in index order
 *   u_node        [Bt][T] float32 uniforms in [0, 1): each non-root node's test
 *   u_final       [Bt] float32    uniform in [0, 1) of each item's final draw
 *   max_path_len  in [1, 1024]    row length of `accepted`
 *   accepted      [Bt][max_path_len] int32  output: node indices of the path,
 *                                 root first; entries past the length are -1
 *   accepted_len  [Bt] int32      output: entries of the path (>= 1)
 *   next_token    [Bt] int32      optional output: the token after the path
 *   tree_status   [Bt] int32      optional; bits 1|2 of the item's tree, and
 *                                 TSV_ST_BAD_TOKEN
 * Only the rows of visited nodes are read (one pass over p_target and q_draft
 * of a node per rejected child, one more for the final draw). No workspace:
 * the residual is never stored. Invalid items leave accepted, accepted_len and
 * next_token untouched. Returns TSV_E_SHAPE for sizes out of range and
 * TSV_E_NULL for a NULL required pointer.
 */
tsv_status tree_ssd_accept_stochastic(int32_t batch, int32_t n_nodes, int32_t vocab,
                                      const int32_t* parent, const int32_t* draft_tokens,
                                      const float* p_target, const float* q_draft, const float* u_node,
                                      const float* u_final, int32_t max_path_len, int32_t* accepted,
                                      int32_t* accepted_len, int32_t* next_token, int32_t* tree_status,
                                      void* stream);

/*
 * tree_ssd_tree_info -- the tree mask of each item (the summary's L): depth of
 * every node (edges from the root) and its ancestor-or-self set as W 64-bit
 * words, W = max(4, ceil(n_nodes / 64)) (bit j % 64 of word j / 64 set iff
 * node j is on the root path of node i); four words up to 256 nodes.
 *
 *   parent   [batch][n_nodes] int32
 *   depth    [batch][n_nodes] int32     output
 *   anc_bits [batch][n_nodes][W] uint64 output (unused words are zero)
 *   tree_status [batch] int32           optional; bits 1|2
 * Invalid items leave depth and anc_bits untouched.
 */
tsv_status tree_ssd_tree_info(int32_t batch, int32_t n_nodes, const int32_t* parent,
                              int32_t* depth, uint64_t* anc_bits, int32_t* tree_status,
                              void* stream);

/* ------------------------------------------------------------------------
 * The two forms a packed tree replaces, on the same inputs, for measuring it
 * against them ("STree: Speculative Tree Decoding for Hybrid State Space
 * Models", atlas.scime.ai summary: without a packed-tree scan an SSM unrolls
 * the draft tree into repeated sequences with extra states and memory, section
 * "Problem"; the paper's baseline is a fused selective scan over the unrolled
 * tree, section "Experimental setup", times in "Key results". The Bole and
 * TreeWY abstracts, mlsanity and fugumt pages, describe the other form: a full
 * recurrent state materialised for every draft node).
 * ------------------------------------------------------------------------ */

/* Per-item status bit of tree_ssd_unroll_plan: more leaves than max_leaves, or
 * a root path longer than max_len */
#define TSV_ST_OVER_CAPACITY 8

/*
 * tree_ssd_unroll_plan -- the unrolled form of each item's tree: one sequence
 * per leaf (a node that is no node's parent, leaves taken by increasing
 * index), holding the leaf's root path from node 0.
 *
 *   parent     [Bt][T] int32
 *   max_leaves in [1, 1024]   sequence slots per item (Lcap)
 *   max_len    in [1, 1024]   positions per sequence (S)
 *   seq_nodes  [Bt][Lcap][S] int32  output: node at each position, -1 past the end
 *   seq_len    [Bt][Lcap] int32     output: path length, 0 for unused slots
 *   n_leaves   [Bt] int32           output: sequences of the item
 *   tree_status [Bt] int32          optional; bits 1|2, or TSV_ST_OVER_CAPACITY
 * Every output is written for every item: an invalid or over-capacity item
 * gets n_leaves 0 and empty slots.
 */
tsv_status tree_ssd_unroll_plan(int32_t batch, int32_t n_nodes, const int32_t* parent, int32_t max_leaves,
                                int32_t max_len, int32_t* seq_nodes, int32_t* seq_len, int32_t* n_leaves,
                                int32_t* tree_status, void* stream);

/*
 * tree_ssd_unroll_gather -- materialise the unrolled sequences: for sequence
 * q = b * max_leaves + l and position s < seq_len[q], copy node
 * n = seq_nodes[q][s]'s rows, and give every sequence its own copy of h0[b].
 * Layouts follow the packed ones with (item, leaf) as the batch index:
 *   x_u [Bt*Lcap][S][H][P], dt_u [Bt*Lcap][S][H], B_u, C_u [Bt*Lcap][S][G][N]
 *   (in_dtype), h0_u [Bt*Lcap][H][P][N] float.
 * s gives the packed shape (x, dt, B, C, h0 as for tree_ssd_verify). Positions
 * past a sequence's length and sequences of length 0 are not written; a
 * length outside [0, S] or a node index outside [0, T) skips the slot.
 */
tsv_status tree_ssd_unroll_gather(const tsv_shape* s, int32_t max_leaves, int32_t max_len, const void* x,
                                  const void* dt, const void* B, const void* C, const float* h0,
                                  const int32_t* seq_nodes, const int32_t* seq_len, void* x_u, void* dt_u,
                                  void* B_u, void* C_u, float* h0_u, void* stream);

/*
 * tree_ssd_seq_scan -- an ordinary Mamba2 scan over sequences (no tree): for
 * each sequence q and head h, from the state h_inout[q][h],
 *   H <- exp(dt_t A_h) H + dt_t x_t (outer) B_t,   y_t = H C_t + D_h x_t
 * for t < seq_len[q]; the final state is written back to h_inout. The shape's
 * batch is the number of sequences and n_nodes their row count S; layouts as
 * written by tree_ssd_unroll_gather, y_u like x_u. head_dim, d_state <= 256
 * and head_dim * d_state <= 16384 (TSV_E_UNSUPPORTED otherwise). Sequences
 * whose length is outside [1, S] are skipped. fp32 arithmetic.
 */
tsv_status tree_ssd_seq_scan(const tsv_shape* s, const void* x_u, const void* dt_u, const float* A,
                             const void* B_u, const void* C_u, const float* D, float* h_inout,
                             const int32_t* seq_len, void* y_u, void* stream);

/*
 * tree_ssd_snapshot_verify -- every node's state materialised: states[b][h][i]
 * is the state after node i's root path (formed from the parent's stored
 * state), and y_i = states_i C_i + D x_i. Arguments as for tree_ssd_verify,
 * plus
 *   states [Bt][H][T][P][N] float  output (T * P * N * 4 bytes per item and head)
 * head_dim, d_state <= 256, head_dim * d_state <= 16384. An invalid item
 * leaves y and states untouched. fp32 arithmetic.
 */
tsv_status tree_ssd_snapshot_verify(const tsv_shape* s, const void* x, const void* dt, const float* A,
                                    const void* B, const void* C, const float* D, const float* h0,
                                    const int32_t* parent, void* y, float* states, int32_t* tree_status,
                                    void* stream);

/*
 * tree_ssd_snapshot_commit -- the snapshot form's commit: copy the stored state
 * of each item's last accepted node into h0_inout [Bt][H][P][N]. states as
 * written by tree_ssd_snapshot_verify; parent, accepted, accepted_len,
 * max_path_len and tree_status (bits 1|2|4) as for tree_ssd_commit. len == 0
 * leaves h0 unchanged; an invalid item leaves it untouched.
 */
tsv_status tree_ssd_snapshot_commit(const tsv_shape* s, const float* states, float* h0_inout,
                                    const int32_t* parent, const int32_t* accepted,
                                    const int32_t* accepted_len, int32_t max_path_len, int32_t* tree_status,
                                    void* stream);

/* ------------------------------------------------------------------------
 * Sequences around the tree: the prompt scan and the single-token step, which
 * make and advance the state h0 that a tree is verified from. The recurrence
 * is that of tree_ssd_verify; along a sequence every token has the one before
 * it as its parent. These calls and those of the paged cache below return
 * TSV_E_UNSUPPORTED where a launch would have 2^32 threads or more (2^24
 * work-groups: about one for each item or 16 rows, and head).
 * ------------------------------------------------------------------------ */

/* Per-item status bit: seq_start is not 0 <= seq_start[0] <= seq_start[1] <=
 * ... <= n_tokens. The array describes one packing, so the bit is set for
 * every sequence of the call and nothing is written for any of them. */
#define TSV_ST_BAD_SEQ 32

typedef struct {
    int32_t n_seqs;   /* sequences >= 0 (0: nothing to do) */
    int32_t n_tokens; /* rows of the packed arrays >= 0, at most 2^31 - 2^16 (TSV_E_UNSUPPORTED past it) */
    int32_t n_heads;  /* H in [1, 65535] */
    int32_t head_dim; /* P in [1, 256] */
    int32_t d_state;  /* N in [1, 256] */
    int32_t n_groups; /* G >= 1, H % G == 0; head h uses group h / (H / G) */
    int32_t in_dtype; /* tsv_dtype of x, dt, B, C, y */
    int32_t flags;    /* TSV_FLAG_FORCE_GENERIC or 0 */
} tsv_seq_shape;

/*
 * tree_ssd_prefill -- one SSD layer over packed prompts of any lengths: for
 * each sequence q, its tokens t = seq_start[q] .. seq_start[q+1] - 1 in order
 * and each head h, from the state h_inout[q][h],
 *   H <- exp(dt_t A_h) H + dt_t x_t (outer) B_t,   y_t = H C_t + D_h x_t,
 * and the state after the last token is written back to h_inout.
 *
 *   x      [n_tokens][H][P]  in_dtype   dt [n_tokens][H]  in_dtype (positive)
 *   A, D   [H]               float
 *   B, C   [n_tokens][G][N]  in_dtype
 *   h_inout [n_seqs][H][P][N] float     read, then overwritten
 *   seq_start [n_seqs + 1]   int32      rows of each sequence
 *   y      [n_tokens][H][P]  in_dtype   rows of no sequence are left as they were
 *   seq_status [n_seqs]      int32      optional; TSV_ST_BAD_SEQ or 0
 *   workspace  device memory of at least the bytes that
 *              tree_ssd_prefill_workspace gives (16-byte aligned; NULL where
 *              that is 0), in use until the stream passes this call: calls
 *              that may overlap need one each
 * An empty sequence keeps its state. A long sequence is cut into segments that
 * run side by side, each from the state that the ones before it leave. Every
 * work-group reads all of seq_start to find its own: thousands of sequences a
 * call are meant, not millions.
 * A token that is not finite reaches its own and the later outputs of its
 * sequence and its state, and nothing else, as infinities or NaNs (which of the
 * two may differ from kernel to kernel).
 *
 * Arithmetic: bf16 inputs with P == 64 and N in {64, 128} take an MFMA kernel
 * over chunks of 64 tokens: scores and decays in fp32, their masked product
 * rounded once to bf16 as the operand of the product with x; the state held in
 * fp32, read out as a bf16 high and low part (off by at most 2^-18 of an
 * element), and updated with weighted inputs in three such parts (24 bits). Per-token log decays
 * below -128 count as -128 (exp of both is 0 in fp32). Other inputs run the
 * recurrence token by token in fp32.
 * TSV_E_SHAPE for negative sizes, TSV_E_NULL also for a missing workspace.
 */
tsv_status tree_ssd_prefill(const tsv_seq_shape* s, const void* x, const void* dt, const float* A,
                            const void* B, const void* C, const float* D, float* h_inout,
                            const int32_t* seq_start, void* y, int32_t* seq_status, void* workspace,
                            uint64_t workspace_bytes, void* stream);

/* Bytes of workspace that tree_ssd_prefill needs for this shape (host only). */
tsv_status tree_ssd_prefill_workspace(const tsv_seq_shape* s, uint64_t* bytes);

/*
 * tree_ssd_step -- one token of each item, without a tree: the state is
 * advanced in place and read out in one pass over it,
 *   H <- exp(dt A_h) H + dt x (outer) B,   y = H C + D_h x.
 * What tree_ssd_verify and tree_ssd_commit of a one-node tree give, with the
 * state read once. s->n_nodes must be 1 (0: nothing to do; TSV_E_SHAPE
 * otherwise); x, y [Bt][H][P], dt [Bt][H], B, C [Bt][G][N] in in_dtype, A, D
 * [H], h_inout [Bt][H][P][N] float. fp32 arithmetic. Not idempotent.
 */
tsv_status tree_ssd_step(const tsv_shape* s, const void* x, const void* dt, const float* A,
                         const void* B, const void* C, const float* D, float* h_inout, void* y,
                         void* stream);

/* ------------------------------------------------------------------------
 * Attention layers of a hybrid model beside its SSM layers: the nodes of a
 * packed tree (or one new token) attend to a paged key-value cache and to
 * their ancestors, and the accepted path's rows, or prompts' rows, enter the
 * cache.
 *
 * The cache: k_cache, v_cache [n_pages][n_kv_heads][page_size][head_dim] in
 * cache_dtype. Position p of item b is row p % page_size of page
 * page_table[b][p / page_size]; cache_len[b] positions are filled. A cache in
 * TSV_E4M3 (OCP e4m3, 1 sign, 4 exponent and 3 mantissa bits, largest value
 * 448) has a scale for each row and head, k_scale, v_scale
 * [n_pages][n_kv_heads][page_size] float: an element stands for byte * scale.
 * Scales are NULL for other caches. Pages may be shared by items as long as no
 * call writes to a shared position.
 * ------------------------------------------------------------------------ */

/* cache_dtype of a cache in 8 bits, beside the tsv_dtype values */
#define TSV_E4M3 2

/* Per-item status bit: cache_len (with the rows to write) is not in
 * [0, max_pages * page_size], or a page index that the call uses is not in
 * [0, n_pages) */
#define TSV_ST_BAD_CACHE 64

typedef struct {
    int32_t batch;       /* Bt >= 0 (0: nothing to do) */
    int32_t n_nodes;     /* T in [0, 1024]; packed rows: their number (tree_attn_append and those below) */
    int32_t n_heads;     /* query heads H >= 1 */
    int32_t n_kv_heads;  /* Hk >= 1, H % Hk == 0; head h reads key head h / (H / Hk) */
    int32_t head_dim;    /* D in [1, 256] */
    int32_t n_pages;     /* pages of the pool >= 0 */
    int32_t page_size;   /* positions per page, in [1, 65536] */
    int32_t max_pages;   /* row length of page_table >= 0; max_pages * page_size <= 2^31 - 2^16 */
    int32_t in_dtype;    /* tsv_dtype of q, k, v, o */
    int32_t cache_dtype; /* in_dtype or TSV_E4M3 (TSV_E_UNSUPPORTED for other pairs) */
    int32_t flags;       /* TSV_FLAG_FORCE_GENERIC or 0 */
    float scale;         /* factor of the scores, usually head_dim^-1/2 (finite, also times log2(e)) */
} tsv_attn_shape;

/*
 * tree_attn_verify -- attention of every node of a packed tree: node i of item
 * b attends to the cache's positions 0 .. cache_len[b] - 1 and to the nodes on
 * its root path, itself included,
 *   o_i = sum_j softmax_j(scale q_i . k_j) v_j.
 * A tree of one node is plain decoding: the new token's own k and v beside the
 * cache. The cache is not written (tree_attn_commit does that).
 *
 *   q, o   [Bt][T][H][D]    in_dtype
 *   k, v   [Bt][T][Hk][D]   in_dtype   the nodes' own keys and values
 *   parent [Bt][T]          int32      as for tree_ssd_verify
 *   page_table [Bt][max_pages] int32, cache_len [Bt] int32
 *   tree_status [Bt]        optional; bits 1|2 and TSV_ST_BAD_CACHE
 *   workspace  as for tree_ssd_prefill, with tree_attn_verify_workspace
 * Items with a status bit keep their o. The work is split over the cache's
 * length by the lengths found on the device, so short and long items may share
 * a batch; a second launch joins the parts.
 *
 * Arithmetic: fp32 scores, maxima, sums and accumulators. bf16 inputs with D
 * 64 or 128 use bf16 MFMA; the softmax weights (times the scale of an 8-bit
 * value row) enter the product with v as two bf16 parts (16 bits) where at most
 * 16 rows share a key head (T * H / Hk <= 16), and rounded once to bf16
 * otherwise. fp32 inputs use fp32 throughout, with D 64 or 128 on fp32 MFMA;
 * other shapes, and tensors that are not 16-byte aligned, use a plain fp32 kernel.
 * A key or a value that is not finite reaches the nodes that see it and no
 * others. An infinite value gives an infinity there, unless its weight is 0 in
 * fp32 (then the element may be finite, infinite or NaN).
 */
tsv_status tree_attn_verify(const tsv_attn_shape* s, const void* q, const void* k, const void* v,
                            const int32_t* parent, const void* k_cache, const void* v_cache,
                            const float* k_scale, const float* v_scale, const int32_t* page_table,
                            const int32_t* cache_len, void* o, int32_t* tree_status, void* workspace,
                            uint64_t workspace_bytes, void* stream);

/* Bytes of workspace that tree_attn_verify needs for this shape (host only). */
tsv_status tree_attn_verify_workspace(const tsv_attn_shape* s, uint64_t* bytes);

/*
 * tree_attn_commit -- the accepted path's keys and values enter the cache: row
 * accepted[b][i] of k and v goes to position cache_len[b] + i, i <
 * accepted_len[b]. The layers of a model share cache_len, so it is read only;
 * the caller adds accepted_len to it after the last layer.
 *   k, v, parent, page_table, cache_len as for tree_attn_verify; accepted,
 *   accepted_len, max_path_len and tree_status as for tree_ssd_commit, with
 *   TSV_ST_BAD_CACHE. Items with a status bit are not written.
 * Rows are stored as they are, or for TSV_E4M3 with
 *   scale = max(max|row| / 448, 2^-126),  byte = row / scale rounded to even;
 * a row with a NaN or an infinity reads back as NaN.
 */
tsv_status tree_attn_commit(const tsv_attn_shape* s, const void* k, const void* v, const int32_t* parent,
                            const int32_t* accepted, const int32_t* accepted_len, int32_t max_path_len,
                            const int32_t* page_table, const int32_t* cache_len, void* k_cache,
                            void* v_cache, float* k_scale, float* v_scale, int32_t* tree_status,
                            void* stream);

/*
 * tree_attn_append -- packed prompts' keys and values enter the cache: row
 * seq_start[b] + i of k and v [n_nodes][Hk][D] goes to position cache_len[b] +
 * i of item b. seq_start [Bt + 1] and seq_status (TSV_ST_BAD_SEQ and
 * TSV_ST_BAD_CACHE) as for tree_ssd_prefill; storage as for tree_attn_commit;
 * cache_len is read only.
 */
tsv_status tree_attn_append(const tsv_attn_shape* s, const void* k, const void* v, const int32_t* seq_start,
                            const int32_t* page_table, const int32_t* cache_len, void* k_cache,
                            void* v_cache, float* k_scale, float* v_scale, int32_t* seq_status,
                            void* stream);

/* ------------------------------------------------------------------------
 * The short causal convolution in front of an SSM layer: depthwise over the
 * C = H P + 2 G N channels of x, B and C (in this order, as the layer's input
 * projection gives them), with its bias and activation,
 *   y_t = act(bias + sum_{k < W} weight[W-1-k] u_{t-k}),
 * split into the x, B and C that the SSM calls take. The state holds the last
 * W - 1 inputs of an item, oldest first; an item without a past has zeros. The v,
 * k and q of a gated-delta-rule layer are such x, B and C (G its key heads, which
 * tree_gdn_verify takes one for each head): where its projection gives them as q,
 * k, v, the rows of its weight, and weight and bias here, change places.
 *
 *   xbc    rows of C channels, row_stride elements apart   in_dtype
 *   weight [C][W]           float      the tap of the newest input last
 *   bias   [C]              float      may be NULL (0)
 *   state  [n][W-1][C]      in_dtype
 *   x [rows][H][P], B, C [rows][G][N]  in_dtype, contiguous; they may not
 *          overlap xbc or the state
 * Sums are fp32, rounded once; states are the inputs as they are. SiLU is y /
 * (1 + exp(-y)). An input that is not finite reaches the outputs of its channel
 * whose W taps hold it, and nothing else.
 * ------------------------------------------------------------------------ */
typedef struct {
    int32_t width;      /* W in [2, 4] (TSV_E_UNSUPPORTED above) */
    int32_t row_stride; /* elements between rows of xbc, at least C */
    int32_t silu;       /* 1: SiLU, 0: no activation */
} tsv_conv;

/*
 * tree_ssd_conv_prefill -- over packed prompts of any lengths: xbc has
 * s->n_tokens rows, seq_start [n_seqs + 1] and seq_status [n_seqs] (optional;
 * TSV_ST_BAD_SEQ or 0) as for tree_ssd_prefill; state_inout [n_seqs][W-1][C]
 * is the state before, then after, each sequence. Rows of no sequence are left
 * as they were.
 */
tsv_status tree_ssd_conv_prefill(const tsv_seq_shape* s, const tsv_conv* c, const void* xbc, const float* weight,
                                 const float* bias, void* state_inout, const int32_t* seq_start, void* x, void* B,
                                 void* C, int32_t* seq_status, void* stream);

/*
 * tree_ssd_conv_step -- one token of each item: xbc has batch rows; s->n_nodes
 * must be 1 (0: nothing to do). Not idempotent.
 */
tsv_status tree_ssd_conv_step(const tsv_shape* s, const tsv_conv* c, const void* xbc, const float* weight,
                              const float* bias, void* state_inout, void* x, void* B, void* C, void* stream);

/*
 * tree_ssd_conv_verify -- every node of a packed tree: u_{t-k} is the input of
 * its k-th ancestor, past the root the state's rows from the last one on. xbc
 * has batch * n_nodes rows (node i of item b is row b n_nodes + i); parent and
 * tree_status as for tree_ssd_verify. The state is not written.
 */
tsv_status tree_ssd_conv_verify(const tsv_shape* s, const tsv_conv* c, const void* xbc, const float* weight,
                                const float* bias, const void* state, const int32_t* parent, void* x, void* B, void* C,
                                int32_t* tree_status, void* stream);

/*
 * tree_ssd_conv_commit -- the state after the accepted path: its last W - 1
 * inputs, or those behind what is left of the old state. xbc and parent as for
 * tree_ssd_conv_verify; accepted, accepted_len, max_path_len and tree_status as
 * for tree_ssd_commit. c->silu is not used. Not idempotent.
 */
tsv_status tree_ssd_conv_commit(const tsv_shape* s, const tsv_conv* c, const void* xbc, void* state_inout,
                                const int32_t* parent, const int32_t* accepted, const int32_t* accepted_len,
                                int32_t max_path_len, int32_t* tree_status, void* stream);

/* ------------------------------------------------------------------------
 * Queries and keys between a projection and the attention: the heads' norms
 * with the position rotation, in one pass,
 *   z = weight x / sqrt(mean(x^2) + eps)         over a head's D elements
 *   (z_a, z_b) <- (z_a cos t - z_b sin t, z_b cos t + z_a sin t),
 *   t = position * inv_freq[i],  i < rot_dim / 2,
 * for the pairs (a, b) = (i, i + rot_dim / 2), or (2 i, 2 i + 1) where
 * `interleaved`; the elements from rot_dim on are z. A NULL weight leaves the
 * norm out (z = x). fp32 arithmetic, the angle's whole turns taken off in 64
 * bits (so that far positions lose nothing), one rounding at the end. A head
 * with an element that is not finite is not finite where it would be in this
 * arithmetic, other heads are as they would be without it.
 *
 *   q [rows][H][D], k [rows][Hk][D], v [rows][Hk][D]   in_dtype, rows
 *     q_stride, k_stride, v_stride elements apart (slices of one projection's
 *     output do), at least a row's and below 2^28
 *   inv_freq [rot_dim / 2], q_weight [D], k_weight [D]   float
 * ------------------------------------------------------------------------ */
typedef struct {
    int32_t rot_dim;     /* even, in [0, head_dim] */
    int32_t interleaved; /* 0 or 1 */
    float eps;           /* >= 0 */
    int64_t q_stride, k_stride, v_stride; /* those of a NULL tensor are not used */
} tsv_rope;

/*
 * tree_attn_rope -- q and k of s->batch * s->n_nodes rows (a tree's nodes in
 * the order of tree_attn_verify; any rows with batch 1) at position [rows]
 * int32: a node's is cache_len[b] + its depth (tree_ssd_tree_info). Rows with
 * a negative position are left as they were. q_out [rows][H][D], k_out
 * [rows][Hk][D] contiguous in in_dtype, or q and k themselves where those are
 * contiguous; q or k may be NULL (left out). Of s the batch, n_nodes, heads,
 * head_dim and in_dtype are used; the rest is only checked (without a cache
 * n_pages and max_pages 0, page_size 1, cache_dtype as in_dtype).
 */
tsv_status tree_attn_rope(const tsv_attn_shape* s, const tsv_rope* r, const void* q, const void* k,
                          const int32_t* position, const float* inv_freq, const float* q_weight, const float* k_weight,
                          void* q_out, void* k_out, void* stream);

/*
 * tree_attn_append_rope -- tree_attn_append with the norm and the rotation of
 * the keys on the way, at their positions in the cache: k and v of s->n_nodes
 * packed rows enter the cache, and where q is given q_out [n_nodes][H][D] gets
 * the queries of the same rows. An e4m3 row and its scale are formed from the
 * row in fp32, without a rounding in between. seq_start and seq_status as for
 * tree_attn_append; rows of no sequence, and of sequences with a status bit,
 * are left as they were in q_out too.
 */
tsv_status tree_attn_append_rope(const tsv_attn_shape* s, const tsv_rope* r, const void* q, const void* k, const void* v,
                                 const int32_t* seq_start, const float* inv_freq, const float* q_weight,
                                 const float* k_weight, const int32_t* page_table, const int32_t* cache_len, void* q_out,
                                 void* k_cache, void* v_cache, float* k_scale, float* v_scale, int32_t* seq_status,
                                 void* stream);

/*
 * tree_attn_prefill -- attention of packed rows of new tokens over the cache
 * that already holds them (tree_attn_append or tree_attn_append_rope wrote
 * them, behind cache_len, which is still the number of positions before them):
 * row seq_start[b] + i of q and o [n_nodes][H][D] is at position p =
 * cache_len[b] + i of item b and sees the positions j <= p, and with a window
 * (window > 0) of those only the ones with j > p - window or j < sinks:
 *   o = sum_j softmax_j(scale q . k_j) v_j.
 * One row of each item is the single-token step of such a layer. seq_start and
 * seq_status (TSV_ST_BAD_SEQ and TSV_ST_BAD_CACHE) as for tree_attn_append.
 * Rows of no sequence, and of sequences with a status bit, are left as they
 * were. Pages wholly outside the windows of a call's rows and the sinks are not
 * looked at: their entries of the table may hold anything.
 *
 * The work is split over the keys by the lengths found on the device, so that
 * long prompts, chunks over long caches and single tokens may share a call; a
 * second launch joins the parts. What the host chooses by the sizes alone, and
 * what it costs (32 query and 8 key heads of 128, bf16):
 *   - one size of block for all sequences, by their average number of rows, empty
 *     ones among them. A long chunk among hundreds of single tokens, or in a batch
 *     padded with as many empty items, is read in the small blocks of single
 *     tokens, and is faster in a call of its own (512 tokens behind 30000 positions
 *     and 256 behind 1000: 1268 us, in two calls 487).
 *   - with a window nothing is cut once the blocks fill the GPU. A window past
 *     most lengths is then better left out (63 tokens behind 100 positions and one
 *     behind 65000: 682 us in a window of 65536, 114 without).
 * workspace as for tree_attn_verify, with
 * tree_attn_prefill_workspace. Every work-group reads all of seq_start and
 * cache_len: thousands of sequences a call are meant, not millions.
 *
 * Arithmetic: fp32 scores, maxima, sums and accumulators, one rounding of the
 * output. head_dim 64 or 128 with 16-byte aligned q, o and caches of fewer than
 * 2^32 rows of a head runs on matrix instructions: bf16 inputs on bf16 ones,
 * where the weights, relative to a running maximum, are rounded to bf16 once
 * (2^-8 of a weight at most), or, where the sequences have no more than 16
 * (token, query head) rows of a key head on average, taken as two bf16 parts;
 * fp32 inputs on fp32 ones. All other shapes run in plain fp32. A key or value
 * that is not finite reaches the rows that see its position and no others; an
 * infinite value gives an infinity there, unless its weight is 0 in fp32.
 * o may not overlap the other arguments.
 * TSV_E_SHAPE for a negative window or sinks, and for sinks without a window.
 */
tsv_status tree_attn_prefill(const tsv_attn_shape* s, int32_t window, int32_t sinks, const void* q,
                             const int32_t* seq_start, const void* k_cache, const void* v_cache, const float* k_scale,
                             const float* v_scale, const int32_t* page_table, const int32_t* cache_len, void* o,
                             int32_t* seq_status, void* workspace, uint64_t workspace_bytes, void* stream);

/* Bytes of workspace that tree_attn_prefill needs for this shape (host only). */
tsv_status tree_attn_prefill_workspace(const tsv_attn_shape* s, uint64_t* bytes);

/* Static, human-readable name of a tsv_status value. */
const char* tree_ssd_status_string(int32_t status);

/* ABI version of this header (incremented on any incompatible change). */
int32_t tree_ssd_abi_version(void);

#define TREE_SSD_ABI_VERSION 1

#ifdef __cplusplus
}
#endif

#endif /* TREE_SSD_H */
