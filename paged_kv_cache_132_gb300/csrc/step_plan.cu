// step_plan.cu -- the plan of a serving step on the GPU: block tables, slots
// and positions from request lengths, without a round trip to the host.
//
// The block manager's bookkeeping ("paged-attention은 도대체 뭘 최적화 하는
// 것일까", §6 blocks are taken from the free pool only when the last block is
// full, §17 ensure_capacity, §18 step 8 blocks return to the pool) for every
// sequence of a step at once, in the order a host that visits the sequences
// one after the other would do it: the free list is a ring, finished sequences
// append their blocks to its end, then growing ones take from its head.
//
// Three prefix sums over the sequences (new tokens, blocks given back, blocks
// taken) place everything; the entries they place are found by binary search
// in the sums, one thread per block or token, so a step of one long prompt and
// one of thousands of single tokens cost alike.
//
// Bound: latency.  A step's data are a few bytes per sequence and 12 per token
// (a megabyte at most), but its loads depend on one another.  So the step is one
// launch: one CTA, or for large steps one cluster of kStepCluster CTAs, each of
// which makes the sums for itself in shared memory.  Nothing that a thread
// writes is read by another one -- a block that is given back and taken again in
// the same step is looked up in the table that gives it -- and the outputs that
// may be inputs (lengths, free state) are written after a barrier of them all.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace pa {
namespace {

constexpr int kStepThreads = 1024;
constexpr int kStepCluster = 8;  // the largest cluster every GPU of the family schedules
// Steps of more token rows or sequences than these run on the cluster.
constexpr int kStepSmallTokens = 2048;
constexpr int kStepSmallSeqs = 1024;
constexpr int kStepUnroll = 4;   // entries of a thread whose loads are in flight together

// For each x: the last index i in [0, n) with start[i] <= x (start[0] = 0 <= x,
// non-decreasing), n <= 2^steps.  The searches go step by step together, so
// that their loads overlap.
template <int N>
__device__ inline void find_sequences(const int* start, int n, int steps, const int (&x)[N], int (&found)[N]) {
#pragma unroll
    for (int u = 0; u < N; ++u) found[u] = 0;
    for (int bit = steps > 0 ? 1 << (steps - 1) : 0; bit; bit >>= 1)
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const int mid = found[u] + bit;
            if (mid < n && start[mid] <= x[u]) found[u] = mid;
        }
}

__device__ inline int blocks_of(int tokens, int block_size) {
    return (int)(((unsigned)tokens + (unsigned)block_size - 1u) / (unsigned)block_size);
}

// Counts saturate at kMaxStepCount: what reaches it fits no step.
struct Sums {
    int tokens, given, taken;
};

__device__ inline Sums add(const Sums& a, const Sums& b) {
    return {min(a.tokens + b.tokens, kMaxStepCount), min(a.given + b.given, kMaxStepCount),
            min(a.taken + b.taken, kMaxStepCount)};
}
__device__ inline Sums inclusive_in_warp(Sums a, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sums up{__shfl_up_sync(0xffffffffu, a.tokens, d), __shfl_up_sync(0xffffffffu, a.given, d),
                      __shfl_up_sync(0xffffffffu, a.taken, d)};
        if (lane >= d) a = add(a, up);
    }
    return a;
}

// One sequence's step; invalid lengths leave it as it is.
struct Change {
    int ctx, grow;
    bool done, bad;
};
__device__ inline Change change_of(const StepPlanParams& p, int s) {
    const int n = p.new_lens[s];
    Change c{p.context_lens[s], n > 0 ? n : 0, n == -1, false};
    c.bad = c.ctx < 0 || c.ctx > p.ctx_cap || n < -1 || c.grow > p.ctx_cap - c.ctx;
    if (c.bad) {
        c.grow = 0;
        c.done = false;
    }
    return c;
}
__device__ inline Sums sums_of(const StepPlanParams& p, const Change& c) {
    Sums a{min(c.grow, kMaxStepCount), 0, 0};
    if (c.done) a.given = min(blocks_of(c.ctx, p.block_size), kMaxStepCount);
    if (c.grow) a.taken = min(blocks_of(c.ctx + c.grow, p.block_size) - blocks_of(c.ctx, p.block_size), kMaxStepCount);
    return a;
}

template <bool CLUSTER>
__global__ void __launch_bounds__(kStepThreads) step_plan_kernel(const StepPlanParams p) {
    extern __shared__ int starts[];  // three prefix sums of num_seqs entries
    __shared__ Sums warp_sums[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = CLUSTER ? (int)blockIdx.x : 0;
    const int first = rank * kStepThreads + tid;             // this thread's entries of each kind
    const int stride = (CLUSTER ? kStepCluster : 1) * kStepThreads;
    int* token_start = starts;
    int* given_start = starts + p.num_seqs;
    int* taken_start = starts + 2 * p.num_seqs;
    pdl_launch_dependents();
    pdl_wait_prerequisites();

    // A thread's consecutive sequences.
    const int each = (p.num_seqs + kStepThreads - 1) / kStepThreads;
    const int s0 = min(tid * each, p.num_seqs), s1 = min(s0 + each, p.num_seqs);
    const int head = p.free_state[0], free_count = p.free_state[1];
    Sums mine{0, 0, 0};
    bool bad = false;
#pragma unroll 4
    for (int s = s0; s < s1; ++s) {
        const Change c = change_of(p, s);
        bad |= c.bad;
        mine = add(mine, sums_of(p, c));
    }
    if (bad && rank == 0) set_error(p.err, PA_DEVERR_CONTEXT_LEN);
    const Sums incl = inclusive_in_warp(mine, lane);
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    if (warp == 0) warp_sums[lane] = inclusive_in_warp(warp_sums[lane], lane);
    __syncthreads();
    const Sums total = warp_sums[31];
    const bool fits = head >= 0 && head < p.ring_size && free_count >= 0 &&
                      (long long)free_count + total.given <= p.ring_size &&
                      total.taken <= (long long)free_count + total.given && total.tokens <= p.max_tokens &&
                      total.tokens < kMaxStepCount && total.given < kMaxStepCount && total.taken < kMaxStepCount;
    if (!fits && first == 0) set_error(p.err, PA_DEVERR_STEP);
    const int tokens = fits ? total.tokens : 0, given = fits ? total.given : 0, taken = fits ? total.taken : 0;

    // The sums before each sequence.
    Sums run = {incl.tokens - mine.tokens, incl.given - mine.given, incl.taken - mine.taken};
    if (warp) run = add(run, warp_sums[warp - 1]);
    for (int s = s0; s < s1; ++s) {
        token_start[s] = run.tokens;
        given_start[s] = run.given;
        taken_start[s] = run.taken;
        if (rank == 0) p.query_start_loc[s] = fits ? run.tokens : 0;
        if (s + 1 < s1) run = add(run, sums_of(p, change_of(p, s)));
    }
    if (first == 0) p.query_start_loc[p.num_seqs] = tokens;
    __syncthreads();

    const int steps = p.num_seqs > 1 ? 32 - __clz(p.num_seqs - 1) : 0;
    auto ring_at = [&](int k) {  // entry k from the head on; head + k < 2 * ring_size
        const unsigned i = (unsigned)head + (unsigned)k;
        return (int)(i >= (unsigned)p.ring_size ? i - (unsigned)p.ring_size : i);
    };
    auto table_at = [&](int s, int block) { return (int64_t)s * p.max_blocks + block; };
    // Where block k of those given back stands, and where block k of those taken
    // comes from: the ring, or the table of the sequence that gives it back.
    auto given_at = [&](const int (&k)[kStepUnroll], const int32_t* (&from)[kStepUnroll]) {
        int seq[kStepUnroll];
        find_sequences(given_start, p.num_seqs, steps, k, seq);
#pragma unroll
        for (int u = 0; u < kStepUnroll; ++u)
            from[u] = p.block_tables + table_at(seq[u], k[u] - given_start[seq[u]]);
    };
    auto taken_from = [&](const int (&k)[kStepUnroll], const int32_t* (&from)[kStepUnroll]) {
        bool beyond = false;
#pragma unroll
        for (int u = 0; u < kStepUnroll; ++u) beyond |= k[u] >= free_count;
        if (beyond) {
            int back[kStepUnroll];
#pragma unroll
            for (int u = 0; u < kStepUnroll; ++u) back[u] = max(k[u] - free_count, 0);
            given_at(back, from);
        }
#pragma unroll
        for (int u = 0; u < kStepUnroll; ++u)
            if (k[u] < free_count) from[u] = p.free_ring + ring_at(k[u]);
    };
    bool wrong = false;  // a block id out of range
    auto good_id = [&](int32_t id) {
        const bool good = id >= 0 && id < p.num_blocks;
        wrong |= !good;
        return good;
    };

    // Blocks of finished sequences, behind the ring's last free entry.
    for (int k0 = first; k0 < given; k0 += kStepUnroll * stride) {
        int k[kStepUnroll];
        const int32_t* from[kStepUnroll];
        int32_t id[kStepUnroll];
#pragma unroll
        for (int u = 0; u < kStepUnroll; ++u) k[u] = min(k0 + u * stride, given - 1);
        given_at(k, from);
#pragma unroll
        for (int u = 0; u < kStepUnroll; ++u) id[u] = *from[u];
#pragma unroll
        for (int u = 0; u < kStepUnroll; ++u) {  // the last entry again where there is none
            good_id(id[u]);
            p.free_ring[ring_at(free_count + k[u])] = id[u];
        }
    }
    // Blocks of growing sequences, from its head.
    for (int k0 = first; k0 < taken; k0 += kStepUnroll * stride) {
        int k[kStepUnroll], seq[kStepUnroll], held[kStepUnroll];
        const int32_t* from[kStepUnroll];
        int32_t id[kStepUnroll];
#pragma unroll
        for (int u = 0; u < kStepUnroll; ++u) k[u] = min(k0 + u * stride, taken - 1);
        find_sequences(taken_start, p.num_seqs, steps, k, seq);
        taken_from(k, from);
#pragma unroll
        for (int u = 0; u < kStepUnroll; ++u) {
            id[u] = *from[u];
            held[u] = blocks_of(p.context_lens[seq[u]], p.block_size);
        }
#pragma unroll
        for (int u = 0; u < kStepUnroll; ++u) {
            good_id(id[u]);
            p.block_tables[table_at(seq[u], held[u] + k[u] - taken_start[seq[u]])] = id[u];
        }
    }
    // Positions and slots.
    for (int t0 = first; t0 < p.max_tokens; t0 += kStepUnroll * stride) {
        int32_t id[kStepUnroll];
        int position[kStepUnroll];
        if (t0 < tokens) {
            int t[kStepUnroll], seq[kStepUnroll], ctx[kStepUnroll], k[kStepUnroll];
            const int32_t* from[kStepUnroll];
#pragma unroll
            for (int u = 0; u < kStepUnroll; ++u) t[u] = min(t0 + u * stride, tokens - 1);
            find_sequences(token_start, p.num_seqs, steps, t, seq);
#pragma unroll
            for (int u = 0; u < kStepUnroll; ++u) ctx[u] = p.context_lens[seq[u]];
#pragma unroll
            for (int u = 0; u < kStepUnroll; ++u) {
                position[u] = ctx[u] + (t[u] - token_start[seq[u]]);
                const int block = (int)((unsigned)position[u] / (unsigned)p.block_size);
                const int held = blocks_of(ctx[u], p.block_size);
                k[u] = block < held ? -1 : taken_start[seq[u]] + block - held;
            }
            taken_from(k, from);
#pragma unroll
            for (int u = 0; u < kStepUnroll; ++u)  // the last block held, not yet full
                if (k[u] < 0)
                    from[u] = p.block_tables +
                              table_at(seq[u], (int)((unsigned)position[u] / (unsigned)p.block_size));
#pragma unroll
            for (int u = 0; u < kStepUnroll; ++u) id[u] = *from[u];
        }
#pragma unroll
        for (int u = 0; u < kStepUnroll; ++u) {
            const int t = t0 + u * stride;
            if (t >= p.max_tokens) continue;
            int64_t slot = -1;
            int place = -1;
            if (t < tokens) {
                place = position[u];
                if (good_id(id[u]))
                    slot = (int64_t)id[u] * p.block_size + (int)((unsigned)place % (unsigned)p.block_size);
            }
            p.positions[t] = place;
            p.slot_mapping[t] = slot;
        }
    }
    if (wrong) set_error(p.err, PA_DEVERR_BLOCK_ID);

    // Every input was read: the outputs may be the same memory.
    if (CLUSTER)
        cooperative_groups::this_cluster().sync();
    else
        __syncthreads();
    for (int s = first; s < p.num_seqs; s += stride) {
        const Change c = change_of(p, s);
        p.context_lens_out[s] = !fits ? c.ctx : c.done ? 0 : c.ctx + c.grow;
    }
    if (first == 0) {
        p.free_state_out[0] = fits ? ring_at(taken) : head;
        p.free_state_out[1] = fits ? free_count + given - taken : free_count;
    }
}

}  // namespace

cudaError_t launch_step_plan(const StepPlanParams& p, cudaStream_t stream) {
    const bool large = p.max_tokens > kStepSmallTokens || p.num_seqs > kStepSmallSeqs;
    const auto kernel = large ? step_plan_kernel<true> : step_plan_kernel<false>;
    const size_t smem = 3 * (size_t)p.num_seqs * sizeof(int);
    if (smem > 40 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   3 * kMaxStepSeqs * (int)sizeof(int));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(large ? kStepCluster : 1);
    cfg.blockDim = dim3(kStepThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kStepCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = large ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace pa
