// tree.h -- internal interface between the C ABI (pa_api.cu) and the kernels of
// a speculative step: trees of drafted tokens.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "kernels.h"

namespace pa {

// ---- plan of drafted trees, commit of the accepted path (tree_step.cu) --------
struct TreePlanParams {
    const int32_t* parents;       // [num_tokens] index in the sequence, < the node's own; -1: follows the cache
    const int32_t* query_start;   // [num_seqs + 1] first row of each sequence
    const int32_t* context_lens;  // cached tokens, the nodes included
    int num_seqs;
    int num_tokens;
    int mask_words;               // 64-bit words of a mask row
    int32_t* positions;           // [num_tokens]
    unsigned long long* tree_mask;  // [num_tokens][mask_words]
    int* err;
};
cudaError_t launch_tree_plan(const TreePlanParams& p, cudaStream_t stream);

struct TreeCommitParams {
    const int32_t* query_start;
    const int32_t* path;           // [num_tokens] nodes of the accepted path, from each sequence's first row on
    const int32_t* accepted_lens;  // [num_seqs]
    const int32_t* context_lens;
    int32_t* context_lens_out;     // may be context_lens
    int num_seqs;
    int num_tokens;
    const int32_t* block_tables;
    int max_blocks;
    int ctx_cap;
    int32_t* free_ring;            // or nullptr: no blocks are given back
    int ring_size;
    const int32_t* free_state;
    int32_t* free_state_out;       // may be free_state
    int64_t num_blocks;
    int num_kv_heads;
    int block_size;
    int chunks;                    // 16-byte chunks of a head's row
    int num_layers;
    int* err;
};
cudaError_t launch_tree_commit(const TreeCommitParams& p, void* const* k_caches, void* const* v_caches,
                               cudaStream_t stream);

// ---- verification (tree_verify.cu) ---------------------------------------------
struct TreeVerifyParams {
    const int32_t* tokens;        // [num_tokens]
    const int32_t* parents;
    const int32_t* query_start;
    int num_seqs;
    int num_tokens;
    const void* target;           // [num_tokens] rows of `vocab` probabilities
    int64_t target_stride;        // elements from row to row
    const void* draft;            // or nullptr
    int64_t draft_stride;
    int vocab;
    const float* accept_uniforms;  // [num_tokens]
    const float* sample_uniforms;  // [num_seqs]
    int32_t* accepted_lens;
    int32_t* path;
    int32_t* next_tokens;
    int* err;
};
constexpr int kMaxVocab = 1 << 20;
cudaError_t launch_tree_verify(const TreeVerifyParams& p, int dtype, int sms, cudaStream_t stream);

// ---- attention of the nodes over the cache (tree_attn*.cu) ----------------------
constexpr int kTreeCtas = 152;    // CTAs of a call at most: what the workspace has room for
constexpr int kTreeMaxLead = 4;   // half tiles that an item begins with, at most
constexpr int kTreePairRows = 256;  // query rows (node, grouped head) of a work item at most: two tiles of 128

struct TreeAttnParams {
    void* out;                    // [num_tokens][num_heads][head_dim], the pools' type
    const int32_t* query_start;
    const uint32_t* tree_mask;    // [num_tokens][mask_words] 32-bit words
    int mask_words;
    const int32_t* block_tables;
    int max_blocks;
    const int32_t* context_lens;
    const void* v_cache;          // (tmap_v)
    int num_seqs;
    int num_tokens;
    int num_heads;
    int num_kv_heads;
    int group;                    // num_heads / num_kv_heads, 1..128
    int tile_tokens;              // nodes of a query tile: 128 / group
    int max_nodes;                // of a sequence: 32 * mask_words
    int max_pairs;                // pairs of query tiles of a sequence, at most
    int block_shift;              // log2(block_size)
    int64_t num_blocks;
    int ctx_cap;
    float scale_log2;             // scale * log2(e), > 0
    int ctas;
    // Workspace: items that several CTAs share.  CTA c leaves the part of an item that
    // begins before it in slot 2 c, of one that goes on behind it in slot 2 c + 1.
    int4* splits;                 // [ctas] of the item that begins in CTA c: first row, nodes, KV head, parts
                                  // (0: it does not go on behind the CTA)
    int* aborted;                 // [ctas] 1: a wait of the CTA ran out, its parts are not there
    int row_cap;                  // rows of a slot
    float2* part_ml;              // [2 ctas][row_cap] maximum, sum
    float* part_o;                // [2 ctas][row_cap][head_dim] sums of weighted values
    int* err;
    unsigned long long wait_limit_ns;
    int debug_flags;              // kDebugDropFirstFill
};

struct TreeWorkspaceLayout {
    size_t splits, aborted, part_ml, part_o, total;
};
// Rows of a slot, for sequences of at most max_nodes nodes.
inline int tree_row_cap(int max_nodes, int group) {
    const int tile_tokens = 128 / group;
    if (max_nodes <= tile_tokens) return (max_nodes * group + 7) / 8 * 8;
    return kTreePairRows;
}
inline TreeWorkspaceLayout tree_workspace_layout(int row_cap, int head_dim) {
    TreeWorkspaceLayout w{};
    size_t off = (size_t)kTreeCtas * sizeof(int4);
    w.aborted = off;
    off += (size_t)kTreeCtas * sizeof(int);
    w.part_ml = off = (off + 255) / 256 * 256;
    off += 2 * (size_t)kTreeCtas * row_cap * sizeof(float2);
    w.part_o = off = (off + 255) / 256 * 256;
    off += 2 * (size_t)kTreeCtas * row_cap * head_dim * sizeof(float);
    w.total = (off + 255) / 256 * 256;
    return w;
}

// tmap_q: the query rows as a 3-D tensor {head_dim, heads, tokens}, box {64, group,
// tile_tokens}; tmap_k, tmap_v: the pools as 4-D tensors {64, 8 rows, slabs, groups of
// 8 rows}, one box per (block, head) tile; 128-byte swizzle.  dtype PA_F16 or PA_BF16.
cudaError_t launch_tree_attention(const TreeAttnParams& p, int dtype, int head_dim, const CUtensorMap* tmap_q,
                                  const CUtensorMap* tmap_k, const CUtensorMap* tmap_v, cudaStream_t stream);

}  // namespace pa
