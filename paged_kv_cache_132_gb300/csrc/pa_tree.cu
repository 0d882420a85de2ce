// pa_tree.cu -- the C ABI of a step of drafted trees (include/pa.h): argument checks
// and launches.  As in pa_api.cu, every argument error is caught here, before anything
// reaches the GPU.
#include <nvtx3/nvToolsExt.h>

#include <algorithm>
#include <cmath>

#include "host.h"
#include "tree.h"

namespace {

using namespace pa::host;

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

// Does an output of `bytes` bytes share memory with an input of `input_bytes`?
bool overlap(const void* out, int64_t bytes, const void* in, int64_t input_bytes) {
    const auto a = reinterpret_cast<uintptr_t>(out), b = reinterpret_cast<uintptr_t>(in);
    return in && bytes > 0 && input_bytes > 0 && a < b + (uint64_t)input_bytes && b < a + (uint64_t)bytes;
}

// Do any two of the layers' pools, of `bytes` bytes each, share memory?
bool pools_overlap(void* const* k_caches, void* const* v_caches, int num_layers, uint64_t bytes) {
    uintptr_t at[2 * pa::kMaxCopyLayers];
    for (int l = 0; l < num_layers; ++l) {
        at[2 * l] = reinterpret_cast<uintptr_t>(k_caches[l]);
        at[2 * l + 1] = reinterpret_cast<uintptr_t>(v_caches[l]);
    }
    std::sort(at, at + 2 * num_layers);
    for (int i = 1; i < 2 * num_layers; ++i)
        if (at[i] - at[i - 1] < bytes) return true;
    return false;
}

}  // namespace

extern "C" {

int pa_plan_tree(const int32_t* parents, const int32_t* query_start_loc, const int32_t* context_lens, int32_t num_seqs,
                 int32_t num_tokens, int32_t* positions, uint64_t* tree_mask, int32_t mask_words, void* stream) {
    NvtxRange range("pa_plan_tree");
    if (num_seqs < 0 || num_tokens < 0 || mask_words <= 0) return PA_ERR_INVALID_ARG;
    if (num_tokens > 0 && (!aligned(parents, 4) || !aligned(positions, 4) || !aligned(tree_mask, 8)))
        return PA_ERR_INVALID_ARG;
    if (!aligned(query_start_loc, 4) || (num_seqs > 0 && !aligned(context_lens, 4))) return PA_ERR_INVALID_ARG;
    if (mask_words > PA_MAX_TREE_NODES / 64) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    const int64_t rows = 4LL * num_tokens, mask_bytes = 8LL * num_tokens * mask_words;
    for (const void* in : {parents, query_start_loc, context_lens}) {
        const int64_t bytes = in == parents ? rows : 4LL * (num_seqs + (in == query_start_loc));
        if (overlap(positions, rows, in, bytes) || overlap(tree_mask, mask_bytes, in, bytes)) return PA_ERR_INVALID_ARG;
    }
    const int dev = current_device();
    if (dev < 0) return PA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return PA_ERR_CUDA;
    pa::TreePlanParams p{};
    p.parents = parents;
    p.query_start = query_start_loc;
    p.context_lens = context_lens;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.mask_words = mask_words;
    p.positions = positions;
    p.tree_mask = reinterpret_cast<unsigned long long*>(tree_mask);
    p.err = err;
    return status_of(pa::launch_tree_plan(p, static_cast<cudaStream_t>(stream)));
}

size_t pa_tree_attention_workspace_size(int32_t num_tokens, int32_t mask_words, int32_t num_heads,
                                        int32_t num_kv_heads, int32_t head_dim) {
    if (num_tokens < 0 || mask_words <= 0 || mask_words > PA_MAX_TREE_NODES / 64 || num_heads <= 0 ||
        num_kv_heads <= 0 || num_heads % num_kv_heads != 0 || num_heads / num_kv_heads > 128 || head_dim <= 0)
        return 0;
    const int nodes = num_tokens < 64 * mask_words ? num_tokens : 64 * mask_words;
    return pa::tree_workspace_layout(pa::tree_row_cap(nodes, num_heads / num_kv_heads), head_dim).total;
}

int pa_tree_attention(void* out, const void* query, int64_t query_stride, const int32_t* query_start_loc,
                      int32_t num_tokens, const uint64_t* tree_mask, int32_t mask_words, const void* k_cache,
                      const void* v_cache, const pa_cache_desc* cache, const int32_t* block_tables,
                      int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t num_seqs, int32_t num_heads,
                      int32_t num_kv_heads, float scale, void* workspace, size_t workspace_bytes, void* stream) {
    NvtxRange range("pa_tree_attention");
    pa::PoolShape shape;
    int rc = check_cache(cache, &shape);
    if (rc != PA_OK) return rc;
    if (num_seqs < 0 || num_tokens < 0 || mask_words <= 0 || num_heads <= 0 || num_kv_heads != cache->num_kv_heads ||
        num_heads % num_kv_heads != 0 || max_blocks_per_seq <= 0 || !(scale > 0.f) ||
        !std::isfinite(scale * 1.4426950408889634f))
        return PA_ERR_INVALID_ARG;
    if (query_stride < (int64_t)num_heads * shape.head_dim || (query_stride * shape.elem_bytes) % 16 != 0)
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!aligned(out, 32) || !aligned(query, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start_loc, 4) ||
        !aligned(tree_mask, 8))
        return PA_ERR_INVALID_ARG;
    const int group = num_heads / num_kv_heads;
    if (cache->dtype == PA_F32 || group > 128 || mask_words > PA_MAX_TREE_NODES / 64) return PA_ERR_UNSUPPORTED;
    if (!(shape.head_dim == 64 || shape.head_dim == 128)) return PA_ERR_UNSUPPORTED;
    if (!(shape.block_size == 8 || shape.block_size == 16 || shape.block_size == 32)) return PA_ERR_UNSUPPORTED;
    constexpr int64_t kMaxStride = (1LL << 39) - 1;  // a tensor copy's strides are below 2^40 bytes
    if (query_stride > kMaxStride || (double)query_stride * num_tokens > 1e17) return PA_ERR_UNSUPPORTED;

    pa::TreeAttnParams p{};
    p.out = out;
    p.query_start = query_start_loc;
    p.tree_mask = reinterpret_cast<const uint32_t*>(tree_mask);
    p.mask_words = 2 * mask_words;
    p.block_tables = block_tables;
    p.max_blocks = max_blocks_per_seq;
    p.context_lens = context_lens;
    p.v_cache = v_cache;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.group = group;
    p.tile_tokens = 128 / group;
    p.max_nodes = 64 * mask_words;
    const int nodes = num_tokens < p.max_nodes ? num_tokens : p.max_nodes;
    p.max_pairs = (nodes + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
    p.block_shift = shape.block_size == 8 ? 3 : shape.block_size == 16 ? 4 : 5;
    p.num_blocks = shape.num_blocks;
    const int64_t cap = (int64_t)max_blocks_per_seq * shape.block_size;
    p.ctx_cap = (int)(cap < 0x7fffff80LL ? cap : 0x7fffff80LL);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.row_cap = pa::tree_row_cap(nodes, group);
    p.wait_limit_ns = wait_limit_ns();
    p.debug_flags = option(PA_OPT_DROP_FIRST_FILL) ? pa::kDebugDropFirstFill : 0;
    // The longest list of K/V tiles these tables allow; its half tiles, with those that each
    // item begins with, stay 32-bit numbers.
    const double items = (double)num_seqs * p.max_pairs * num_kv_heads;
    const double tiles = items * (double)((p.ctx_cap + 127LL) / 128);
    if (2. * tiles + pa::kTreeMaxLead * items > 2147483647.) return PA_ERR_UNSUPPORTED;
    const pa::TreeWorkspaceLayout lay = pa::tree_workspace_layout(p.row_cap, shape.head_dim);
    if (!aligned(workspace, 256) || workspace_bytes < lay.total) return PA_ERR_WORKSPACE;
    const int64_t row = (int64_t)num_heads * shape.head_dim;
    if (overlap(out, num_tokens * row * shape.elem_bytes, query,
                ((num_tokens - 1) * query_stride + row) * shape.elem_bytes))
        return PA_ERR_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    p.splits = reinterpret_cast<int4*>(ws);
    p.aborted = reinterpret_cast<int*>(ws + lay.aborted);
    p.part_ml = reinterpret_cast<float2*>(ws + lay.part_ml);
    p.part_o = reinterpret_cast<float*>(ws + lay.part_o);

    const int dev = current_device();
    if (dev < 0) return PA_ERR_CUDA;
    p.err = error_word(dev);
    const int sms = sm_count(dev);
    if (!p.err || sms <= 0) return PA_ERR_CUDA;
    p.ctas = sms < pa::kTreeCtas ? sms : pa::kTreeCtas;
    if (tiles < p.ctas) p.ctas = tiles < 1. ? 1 : (int)tiles;

    CUtensorMap tmap_q, tmap_k, tmap_v;  // copies: later lookups may reuse a cache slot
    const CUtensorMap* m =
        rows_map(query, cache->dtype, num_tokens, num_heads, shape.head_dim, query_stride, group, p.tile_tokens);
    if (!m) return PA_ERR_UNSUPPORTED;
    tmap_q = *m;
    if (!(m = group_map(k_cache, cache->dtype, shape))) return PA_ERR_UNSUPPORTED;
    tmap_k = *m;
    if (!(m = group_map(v_cache, cache->dtype, shape))) return PA_ERR_UNSUPPORTED;
    tmap_v = *m;
    return status_of(pa::launch_tree_attention(p, cache->dtype, shape.head_dim, &tmap_q, &tmap_k, &tmap_v,
                                               static_cast<cudaStream_t>(stream)));
}

int pa_verify_tree(const int32_t* tokens, const int32_t* parents, const int32_t* query_start_loc, int32_t num_seqs,
                   int32_t num_tokens, const void* target_probs, int64_t target_stride, const void* draft_probs,
                   int64_t draft_stride, int32_t vocab_size, int32_t dtype, const float* accept_uniforms,
                   const float* sample_uniforms, int32_t* accepted_lens, int32_t* path, int32_t* next_tokens,
                   void* stream) {
    NvtxRange range("pa_verify_tree");
    const int eb = elem_bytes(dtype);
    if (eb == 0 || num_seqs < 0 || num_tokens < 0 || vocab_size <= 0 || target_stride < vocab_size ||
        (draft_probs && draft_stride < vocab_size))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!aligned(query_start_loc, 4) || !aligned(sample_uniforms, 4) || !aligned(accepted_lens, 4) ||
        !aligned(next_tokens, 4))
        return PA_ERR_INVALID_ARG;
    if (num_tokens > 0 && (!aligned(tokens, 4) || !aligned(parents, 4) || !aligned(target_probs, eb) ||
                           (draft_probs && !aligned(draft_probs, eb)) || !aligned(accept_uniforms, 4) ||
                           !aligned(path, 4)))
        return PA_ERR_INVALID_ARG;
    if (vocab_size > pa::kMaxVocab || num_seqs > (1 << 24)) return PA_ERR_UNSUPPORTED;
    // A sequence's results are written while others, and its own path, are still read.
    const int64_t rows = 4LL * num_tokens, seqs = 4LL * num_seqs;
    for (const void* in : {tokens, parents})
        if (overlap(path, rows, in, rows) || overlap(accepted_lens, seqs, in, rows) || overlap(next_tokens, seqs, in, rows))
            return PA_ERR_INVALID_ARG;
    if (overlap(path, rows, query_start_loc, seqs + 4) || overlap(accepted_lens, seqs, query_start_loc, seqs + 4) ||
        overlap(next_tokens, seqs, query_start_loc, seqs + 4))
        return PA_ERR_INVALID_ARG;
    const int dev = current_device();
    if (dev < 0) return PA_ERR_CUDA;
    int* err = error_word(dev);
    const int sms = sm_count(dev);
    if (!err || sms <= 0) return PA_ERR_CUDA;
    pa::TreeVerifyParams p{};
    p.tokens = tokens;
    p.parents = parents;
    p.query_start = query_start_loc;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.target = target_probs;
    p.target_stride = target_stride;
    p.draft = draft_probs;
    p.draft_stride = draft_stride;
    p.vocab = vocab_size;
    p.accept_uniforms = accept_uniforms;
    p.sample_uniforms = sample_uniforms;
    p.accepted_lens = accepted_lens;
    p.path = path;
    p.next_tokens = next_tokens;
    p.err = err;
    return status_of(pa::launch_tree_verify(p, dtype, sms, static_cast<cudaStream_t>(stream)));
}

int pa_commit_tree(void* const* k_caches, void* const* v_caches, int32_t num_layers, const pa_cache_desc* cache,
                   const int32_t* query_start_loc, int32_t num_seqs, int32_t num_tokens, const int32_t* path,
                   const int32_t* accepted_lens, const int32_t* context_lens, int32_t* context_lens_out,
                   const int32_t* block_tables, int32_t max_blocks_per_seq, int32_t* free_ring, int32_t ring_size,
                   const int32_t* free_state, int32_t* free_state_out, void* stream) {
    NvtxRange range("pa_commit_tree");
    pa::PoolShape shape;
    int rc = check_cache(cache, &shape);
    if (rc != PA_OK) return rc;
    if (num_layers < 1 || num_layers > pa::kMaxCopyLayers || num_seqs < 0 || num_tokens < 0 ||
        max_blocks_per_seq <= 0 || !k_caches || !v_caches || (free_ring && ring_size <= 0))
        return PA_ERR_INVALID_ARG;
    if (free_ring && (!aligned(free_ring, 4) || !aligned(free_state, 4) || !aligned(free_state_out, 4)))
        return PA_ERR_INVALID_ARG;
    if (!aligned(query_start_loc, 4)) return PA_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!aligned(accepted_lens, 4) || !aligned(context_lens, 4) || !aligned(context_lens_out, 4) ||
                         !aligned(block_tables, 4) || (num_tokens > 0 && !aligned(path, 4))))
        return PA_ERR_INVALID_ARG;
    for (int l = 0; l < num_layers; ++l)
        if (!aligned(k_caches[l], 16) || !aligned(v_caches[l], 16)) return PA_ERR_INVALID_ARG;
    if (num_seqs > pa::kMaxStepSeqs || (free_ring && ring_size >= pa::kMaxStepCount)) return PA_ERR_UNSUPPORTED;
    // A path's rows move in every pool at once: in one that is given twice they would move twice.
    const uint64_t pool_bytes = (uint64_t)shape.num_blocks * shape.num_kv_heads * shape.block_size * shape.head_dim *
                                shape.elem_bytes;
    if (pools_overlap(k_caches, v_caches, num_layers, pool_bytes)) return PA_ERR_INVALID_ARG;
    // The moves read what the lengths are made of; context_lens itself is overwritten behind them.
    const int64_t seqs = 4LL * num_seqs;
    if (overlap(context_lens_out, seqs, accepted_lens, seqs) || overlap(context_lens_out, seqs, path, 4LL * num_tokens) ||
        overlap(context_lens_out, seqs, query_start_loc, seqs + 4) ||
        (context_lens_out != context_lens && overlap(context_lens_out, seqs, context_lens, seqs)))
        return PA_ERR_INVALID_ARG;
    const int dev = current_device();
    if (dev < 0) return PA_ERR_CUDA;
    int* err = error_word(dev);
    if (!err) return PA_ERR_CUDA;
    pa::TreeCommitParams p{};
    p.query_start = query_start_loc;
    p.path = path;
    p.accepted_lens = accepted_lens;
    p.context_lens = context_lens;
    p.context_lens_out = context_lens_out;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.block_tables = block_tables;
    p.max_blocks = max_blocks_per_seq;
    const int64_t cap = (int64_t)max_blocks_per_seq * shape.block_size;
    p.ctx_cap = (int)(cap < 0x7fffffffLL ? cap : 0x7fffffffLL);
    p.free_ring = free_ring;
    p.ring_size = ring_size;
    p.free_state = free_state;
    p.free_state_out = free_state_out;
    p.num_blocks = shape.num_blocks;
    p.num_kv_heads = shape.num_kv_heads;
    p.block_size = shape.block_size;
    p.chunks = shape.head_dim * shape.elem_bytes / 16;
    p.num_layers = num_layers;
    p.err = err;
    return status_of(pa::launch_tree_commit(p, k_caches, v_caches, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
