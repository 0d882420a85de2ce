// tree_step.cu -- what a step of drafted trees does to the bookkeeping around the
// cache: positions and ancestor masks of the nodes from their parents, and, once
// the trees are verified, the commit of the accepted paths.
//
// Plan.  Node i attends to itself and its ancestors: a thread follows the parents up
// from its node (in shared memory, one step some 30 cycles) and sets a bit for each.
// Parents stand before their nodes, so the words of the mask row are finished from
// the last to the first.  Its position is the tree's first one plus its depth (a
// chain's is plan_step's).  Bound: latency: 2.7 us for 64 trees of 16 nodes (graph
// replay, launch included), 4.4 us for 2048 trees of up to 61.
//
// Commit.  Node path[i] of the accepted path becomes the i-th token behind the cached
// ones: its rows move to that place in every layer's pools.  As path[i] >= i and
// increases, a place that is written is not read by a later i, so a thread that goes
// through the path in order, several loads before their stores, moves its 16 bytes of
// every row without any synchronisation.  The moves are computed once per CTA (a
// sequence and some of the layers).  The lengths are cut, and the blocks that only
// held refused nodes go back behind the ring's last free entry, sequence after
// sequence (a prefix sum), by one CTA: of the same launch, unless it overwrites the
// lengths that the others read.  Bound: HBM for batches, latency below: 2.9 us for one
// sequence and four layers; 7.7 us for 96 sequences and 32 layers (graph replay; 26 MB
// read and written in pieces of 256 bytes, 3.4 TB/s).
#include "common.cuh"
#include "tree.h"

namespace pa {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
constexpr int kTreeStaged = PA_MAX_TREE_NODES;  // parents in shared memory

__global__ void __launch_bounds__(128) tree_plan_kernel(const TreePlanParams p) {
    __shared__ int staged[kTreeStaged];
    pdl_wait_prerequisites();
    const int s = blockIdx.x, words = p.mask_words;
    const int row0 = p.query_start[s], end = p.query_start[s + 1], ctx = p.context_lens[s];
    const int first = p.query_start[0], behind = p.query_start[p.num_seqs];
    // Rows outside every sequence (a captured step's padding).
    for (int row = blockIdx.x * blockDim.x + threadIdx.x; row < p.num_tokens; row += gridDim.x * blockDim.x)
        if (row < first || row >= behind) {
            p.positions[row] = -1;
            for (int w = 0; w < words; ++w) p.tree_mask[(int64_t)row * words + w] = 0;
        }
    const int n = end - row0;
    if (row0 < 0 || n < 0 || end > p.num_tokens || n > 64 * words || ctx < n) {
        if (threadIdx.x == 0) set_error(p.err, PA_DEVERR_CONTEXT_LEN);
        const int stop = min(end, p.num_tokens);
        for (int row = max(row0, 0) + threadIdx.x; row < stop; row += blockDim.x) {
            p.positions[row] = -1;
            for (int w = 0; w < words; ++w) p.tree_mask[(int64_t)row * words + w] = 0;
        }
        return;
    }
    bool bad = false;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        int up = p.parents[row0 + i];
        if (up < -1 || up >= i) {
            bad = true;
            up = -1;
        }
        staged[i] = up;
    }
    if (bad) set_error(p.err, PA_DEVERR_TREE);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        unsigned long long* const mask = p.tree_mask + (int64_t)(row0 + i) * words;
        unsigned long long bits = 0;
        int word = words - 1, depth = 0;
        for (int at = i;;) {
            for (; word > at >> 6; --word) {
                mask[word] = bits;
                bits = 0;
            }
            bits |= 1ull << (at & 63);
            const int up = staged[at];
            if (up < 0) break;
            ++depth;
            at = up;
        }
        for (; word >= 0; --word) {
            mask[word] = bits;
            bits = 0;
        }
        p.positions[row0 + i] = ctx - n + depth;
    }
}

// ---------------------------------------------------------------------------
// commit
// ---------------------------------------------------------------------------
struct TreePools {
    uint4* k[kMaxCopyLayers];
    uint4* v[kMaxCopyLayers];
};

constexpr int kMoveThreads = 256;
constexpr int kMovesInFlight = 8;
constexpr int kLengthThreads = 1024;
// Sequences up to which the lengths are one CTA of the moves' launch.
constexpr int kFusedLengthSeqs = 2048;

// A sequence's nodes and the part of them that stays.
struct Kept {
    int row0, n, ctx, keep;  // n = 0 and keep = 0 when the lengths break the rules
    bool good;
};
__device__ inline Kept tree_kept(const TreeCommitParams& p, int s) {
    const int a = p.query_start[s], b = p.query_start[s + 1];
    Kept q{a, b - a, p.context_lens[s], p.accepted_lens[s], true};
    q.good = a >= 0 && b >= a && b <= p.num_tokens && q.ctx >= q.n && q.ctx <= p.ctx_cap && q.keep >= 0 && q.keep <= q.n;
    if (!q.good) q.n = q.keep = 0;
    return q;
}
// Does entry i break the path's rules: 0 <= path[0] < path[1] < ... < n ?
__device__ inline bool path_breaks(const TreeCommitParams& p, const Kept& q, int i) {
    const int at = p.path[q.row0 + i], before = i > 0 ? p.path[q.row0 + i - 1] : -1;
    return at <= before || at >= q.n;
}

// New length of a sequence and the blocks it gives back (columns [first, first + count)
// of its table row).
struct Cut {
    int ctx, first, count;
};
__device__ inline Cut tree_cut(const TreeCommitParams& p, int s, bool report) {
    if (s >= p.num_seqs) return {0, 0, 0};
    const Kept q = tree_kept(p, s);
    bool wrong = false;
#pragma unroll 4
    for (int i = 0; i < q.keep; ++i) wrong |= path_breaks(p, q, i);
    if (report && !q.good) set_error(p.err, PA_DEVERR_CONTEXT_LEN);
    if (report && wrong) set_error(p.err, PA_DEVERR_TREE);
    if (!q.good || wrong) return {q.ctx, 0, 0};  // stays as it is
    const int after = q.ctx - q.n + q.keep;
    const int held = (int)(((unsigned)q.ctx + (unsigned)p.block_size - 1u) / (unsigned)p.block_size);
    const int need = (int)(((unsigned)after + (unsigned)p.block_size - 1u) / (unsigned)p.block_size);
    return {after, need, held - need};
}

template <int THREADS>
__device__ void tree_lengths(const TreeCommitParams& p) {
    __shared__ long long sums[THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // Sum of x over the CTA, and the sum over the threads before this one.
    auto scan = [&](long long x, long long& total) {
        long long incl = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const long long up = __shfl_up_sync(kAll, incl, d);
            if (lane >= d) incl += up;
        }
        __syncthreads();
        if (lane == 31) sums[warp] = incl;
        __syncthreads();
        long long before = incl - x;
        total = 0;
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += sums[w];
            total += sums[w];
        }
        return before;
    };
    const bool ring = p.free_ring != nullptr;
    int head = 0, count = 0;
    if (ring) {
        head = p.free_state[0];
        count = p.free_state[1];
    }
    Cut mine = tree_cut(p, tid, true);
    const bool single = p.num_seqs <= THREADS;
    long long given = 0;
    if (!single || ring) {
        long long here = mine.count;
        for (int s = tid + THREADS; s - tid < p.num_seqs; s += THREADS) here += tree_cut(p, s, true).count;
        scan(here, given);
    }
    const bool fits = head >= 0 && head < p.ring_size && count >= 0 && count + given <= p.ring_size;
    if (ring && !fits && tid == 0) set_error(p.err, PA_DEVERR_STEP);
    long long done = 0;
    bool wrong = false;
    for (int s0 = 0; s0 < p.num_seqs; s0 += THREADS) {
        const int s = s0 + tid;
        if (s0 > 0) mine = tree_cut(p, s, false);
        if (ring && fits) {
            long long total;
            long long at = head + count + done + scan(mine.count, total);
            done += total;
            for (int k = 0; k < mine.count; ++k, ++at) {
                const int id = p.block_tables[(int64_t)s * p.max_blocks + mine.first + k];
                wrong |= id < 0 || id >= p.num_blocks;
                p.free_ring[at % p.ring_size] = id;
            }
        }
        if (s < p.num_seqs) p.context_lens_out[s] = mine.ctx;
    }
    if (wrong) set_error(p.err, PA_DEVERR_BLOCK_ID);
    __syncthreads();  // free_state_out may be free_state, which every thread has read
    if (ring && tid == 0) {
        p.free_state_out[0] = head;
        p.free_state_out[1] = fits ? (int)(count + given) : count;
    }
}

__global__ void __launch_bounds__(kLengthThreads) tree_lengths_kernel(const __grid_constant__ TreeCommitParams p) {
    pdl_wait_prerequisites();  // the moves read the lengths
    tree_lengths<kLengthThreads>(p);
}

// CTA (x, y): sequence x, layers y, y + gridDim.y, ...; with `lengths`, CTA (0, 0)
// does the lengths and the sequences begin at x = 1.
__global__ void __launch_bounds__(kMoveThreads)
    tree_move_kernel(const __grid_constant__ TreeCommitParams p, const __grid_constant__ TreePools pools, int lengths) {
    __shared__ int64_t from[32], to[32];  // first chunk of the row of head 0
    __shared__ int moves;
    pdl_wait_prerequisites();
    if (lengths && blockIdx.x == 0) {
        if (blockIdx.y == 0) tree_lengths<kMoveThreads>(p);
        return;
    }
    const int s = (int)blockIdx.x - lengths, tid = threadIdx.x, lane = tid & 31;
    const Kept q = tree_kept(p, s);
    bool wrong = false;
    for (int i = tid; i < q.keep; i += kMoveThreads) wrong |= path_breaks(p, q, i);
    if (__syncthreads_or(wrong)) return;  // reported with the lengths
    const int64_t head_chunks = (int64_t)p.block_size * p.chunks;
    const int units = 2 * p.num_kv_heads * p.chunks;
    for (int i0 = 0; i0 < q.keep; i0 += 32) {
        if (tid < 32) {
            // The moves of 32 entries, in order.
            const int i = i0 + lane;
            const int at = i < q.keep ? p.path[q.row0 + i] : i;
            int64_t row[2] = {0, 0};
            bool move = at != i;
            if (move) {
                const int32_t* const table = p.block_tables + (int64_t)s * p.max_blocks;
                const unsigned pos[2] = {(unsigned)(q.ctx - q.n + at), (unsigned)(q.ctx - q.n + i)};
                int id[2], block[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    block[e] = (int)(pos[e] / (unsigned)p.block_size);
                    id[e] = table[block[e]];
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (id[e] < 0 || id[e] >= p.num_blocks) {
                        set_error(p.err, PA_DEVERR_BLOCK_ID);
                        move = false;
                    }
                    row[e] = (int64_t)id[e] * p.num_kv_heads * head_chunks +
                             (int64_t)(pos[e] - (unsigned)block[e] * (unsigned)p.block_size) * p.chunks;
                }
            }
            const unsigned all = __ballot_sync(kAll, move);
            if (move) {
                const int k = __popc(all & ((1u << lane) - 1u));
                from[k] = row[0];
                to[k] = row[1];
            }
            if (lane == 0) moves = __popc(all);
        }
        __syncthreads();
        const int n = moves;
        for (int layer = blockIdx.y; n > 0 && layer < p.num_layers; layer += gridDim.y)
            for (int u = tid; u < units; u += kMoveThreads) {
                const int hc = u < units / 2 ? u : u - units / 2;
                const int h = hc / p.chunks;
                uint4* const pool = (u < units / 2 ? pools.k[layer] : pools.v[layer]) + h * head_chunks + (hc - h * p.chunks);
                for (int k0 = 0; k0 < n; k0 += kMovesInFlight) {
                    uint4 data[kMovesInFlight];
#pragma unroll
                    for (int k = 0; k < kMovesInFlight; ++k)
                        if (k0 + k < n) data[k] = pool[from[k0 + k]];
#pragma unroll
                    for (int k = 0; k < kMovesInFlight; ++k)
                        if (k0 + k < n) pool[to[k0 + k]] = data[k];
                }
            }
        __syncthreads();
    }
}

cudaLaunchConfig_t launch_config(dim3 grid, int threads, cudaStream_t stream, cudaLaunchAttribute* attr) {
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

}  // namespace

cudaError_t launch_tree_plan(const TreePlanParams& p, cudaStream_t stream) {
    if (p.num_seqs == 0) {  // padding alone
        const cudaError_t e = cudaMemsetAsync(p.positions, 0xff, (size_t)p.num_tokens * 4, stream);
        if (e != cudaSuccess) return e;
        return cudaMemsetAsync(p.tree_mask, 0, (size_t)p.num_tokens * p.mask_words * 8, stream);
    }
    cudaLaunchAttribute attr;
    const int64_t most = 64LL * p.mask_words < p.num_tokens ? 64LL * p.mask_words : p.num_tokens;
    const int threads = most >= 128 ? 128 : (int)((most + 31) / 32) * 32;
    const cudaLaunchConfig_t cfg = launch_config(dim3((unsigned)p.num_seqs), threads, stream, &attr);
    return cudaLaunchKernelEx(&cfg, tree_plan_kernel, p);
}

cudaError_t launch_tree_commit(const TreeCommitParams& p, void* const* k_caches, void* const* v_caches,
                               cudaStream_t stream) {
    if (p.num_seqs == 0) {
        if (!p.free_ring || p.free_state_out == p.free_state) return cudaSuccess;
        return cudaMemcpyAsync(p.free_state_out, p.free_state, 8, cudaMemcpyDeviceToDevice, stream);
    }
    TreePools pools{};
    for (int l = 0; l < p.num_layers; ++l) {
        pools.k[l] = static_cast<uint4*>(k_caches[l]);
        pools.v[l] = static_cast<uint4*>(v_caches[l]);
    }
    cudaLaunchAttribute attr;
    const bool apart = p.context_lens_out + p.num_seqs <= p.context_lens || p.context_lens + p.num_seqs <= p.context_lens_out;
    const int fused = apart && p.num_seqs <= kFusedLengthSeqs ? 1 : 0;
    // Some six CTAs per SM: fewer layers to a CTA for few sequences.
    int slices = (6 * 152 + p.num_seqs - 1) / p.num_seqs;
    if (slices > p.num_layers) slices = p.num_layers;
    cudaLaunchConfig_t cfg = launch_config(dim3((unsigned)(p.num_seqs + fused), (unsigned)slices), kMoveThreads, stream, &attr);
    cudaError_t e = cudaLaunchKernelEx(&cfg, tree_move_kernel, p, pools, fused);
    if (e != cudaSuccess || fused) return e;
    cfg = launch_config(dim3(1), kLengthThreads, stream, &attr);
    return cudaLaunchKernelEx(&cfg, tree_lengths_kernel, p);
}

}  // namespace pa
