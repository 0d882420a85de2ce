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
// Bound: latency.  A step's data are a few bytes per sequence and 12 per token row
// (1 MB for the large step below), but its loads depend on one another.  So a step is one
// CTA, or for large steps one cluster of kStepCluster CTAs, each of which makes
// the sums for itself in shared memory, and then a second kernel that places the
// tokens on the whole GPU.  Nothing that a thread writes is read by another one
// of the same kernel -- a block that is given back and taken again in the same
// step is looked up in the table that gives it -- and the outputs that may be
// inputs (lengths, free state) are written after a barrier of them all.
//
// Measured (graph replays, launch included; an empty step takes 2.3 us): 4.4 us
// for 256 sequences of one new token; 13.3 us for 4096 sequences with 74 000 new
// tokens, 3 700 blocks given back and 4 600 taken (1 MB).  In one CTA the sums
// alone take 1 us per 1024 sequences (three prefix sums by shuffles).
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"

namespace pa {
namespace {

constexpr int kStepThreads = 1024;
constexpr int kSlotThreads = 256;
constexpr int kStepCluster = 8;  // the largest cluster every GPU of the family schedules
// Steps of more token rows or sequences than these run on the cluster and the
// slots kernel.  Measured, one CTA against those: 4.4 and 5.8 us for a prompt of
// 4096 tokens, 6.9 and 6.7 us for 8 of 1024; 5.8 and 7.5 us for 1024 sequences of
// one token, 7.9 and 7.9 us for 2048.  The rows are those that there is room for
// (the host knows no others): 256 sequences of one token take 4.5 us with room for
// 256 rows, 5.6 with 8192, 7.2 with 8193 to 65536.
constexpr int kStepSmallTokens = 8192;
constexpr int kStepSmallSeqs = 2048;
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

// Block of a position and blocks of a number of tokens; block sizes are powers
// of two as a rule (block_shift >= 0), and a division costs some 20 instructions.
__device__ inline int block_of(const StepPlanParams& p, unsigned position) {
    return (int)(p.block_shift >= 0 ? position >> p.block_shift : position / (unsigned)p.block_size);
}
__device__ inline int blocks_of(const StepPlanParams& p, int tokens) {
    return block_of(p, (unsigned)tokens + (unsigned)p.block_size - 1u);
}

__device__ inline int64_t slot_of(const StepPlanParams& p, int32_t id, int position) {
    return (int64_t)id * p.block_size + (position - block_of(p, (unsigned)position) * p.block_size);
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
    if (c.done) a.given = min(blocks_of(p, c.ctx), kMaxStepCount);
    if (c.grow) a.taken = min(blocks_of(p, c.ctx + c.grow) - blocks_of(p, c.ctx), kMaxStepCount);
    return a;
}

// LARGE: a cluster, and the tokens are left to step_slots_kernel.
template <bool LARGE>
__global__ void __launch_bounds__(kStepThreads) step_plan_kernel(const StepPlanParams p) {
    extern __shared__ int starts[];  // three prefix sums of num_seqs entries
    __shared__ Sums warp_sums[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = LARGE ? (int)blockIdx.x : 0;
    const int first = rank * kStepThreads + tid;             // this thread's entries of each kind
    const int stride = (LARGE ? kStepCluster : 1) * kStepThreads;
    int* token_start = starts;
    int* given_start = starts + p.num_seqs;
    int* taken_start = starts + 2 * p.num_seqs;
    // Only for the slots kernel of the same call: any other kernel starts when the
    // lengths and tables are written.
    if (LARGE && p.max_tokens > 0) pdl_launch_dependents();
    pdl_wait_prerequisites();

    // The sums, EACH sequences of a thread at a time; the next ones load meanwhile.
    constexpr int EACH = LARGE ? 4 : 1;
    const int head = p.free_state[0], free_count = p.free_state[1];
    Sums total{0, 0, 0};
    bool bad = false;
    Change next[EACH];
    auto load = [&](int s) {
#pragma unroll
        for (int e = 0; e < EACH; ++e)
            next[e] = s + e < p.num_seqs ? change_of(p, s + e) : Change{0, 0, false, false};
    };
    load(tid * EACH);
    for (int base = 0; base < p.num_seqs; base += kStepThreads * EACH) {
        const int s = base + tid * EACH;
        Sums each[EACH], mine{0, 0, 0};
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
            bad |= next[e].bad;
            each[e] = sums_of(p, next[e]);
            mine = add(mine, each[e]);
        }
        load(s + kStepThreads * EACH);
        const Sums incl = inclusive_in_warp(mine, lane);
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();
        if (warp == 0) warp_sums[lane] = inclusive_in_warp(warp_sums[lane], lane);
        __syncthreads();
        Sums before = {incl.tokens - mine.tokens, incl.given - mine.given, incl.taken - mine.taken};
        if (warp) before = add(before, warp_sums[warp - 1]);
        before = add(before, total);
#pragma unroll
        for (int e = 0; e < EACH; ++e)
            if (s + e < p.num_seqs) {
                token_start[s + e] = before.tokens;
                given_start[s + e] = before.given;
                taken_start[s + e] = before.taken;
                before = add(before, each[e]);
            }
        total = add(total, warp_sums[31]);
        __syncthreads();
    }
    if (bad && rank == 0) set_error(p.err, PA_DEVERR_CONTEXT_LEN);
    const bool fits = head >= 0 && head < p.ring_size && free_count >= 0 &&
                      (long long)free_count + total.given <= p.ring_size &&
                      total.taken <= (long long)free_count + total.given && total.tokens <= p.max_tokens &&
                      total.tokens < kMaxStepCount && total.given < kMaxStepCount && total.taken < kMaxStepCount;
    if (!fits && first == 0) set_error(p.err, PA_DEVERR_STEP);
    const int tokens = fits ? total.tokens : 0, given = fits ? total.given : 0, taken = fits ? total.taken : 0;
    for (int s = first; s < p.num_seqs; s += stride) p.query_start_loc[s] = fits ? token_start[s] : 0;
    if (first == 0) p.query_start_loc[p.num_seqs] = tokens;

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
            held[u] = blocks_of(p, p.context_lens[seq[u]]);
        }
#pragma unroll
        for (int u = 0; u < kStepUnroll; ++u) {
            good_id(id[u]);
            p.block_tables[table_at(seq[u], held[u] + k[u] - taken_start[seq[u]])] = id[u];
        }
    }
    // Positions and slots.
    for (int t0 = first; !LARGE && t0 < p.max_tokens; t0 += kStepUnroll * stride) {
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
                const int block = block_of(p, (unsigned)position[u]);
                const int held = blocks_of(p, ctx[u]);
                k[u] = block < held ? -1 : taken_start[seq[u]] + block - held;
            }
            taken_from(k, from);
#pragma unroll
            for (int u = 0; u < kStepUnroll; ++u)  // the last block held, not yet full
                if (k[u] < 0)
                    from[u] = p.block_tables + table_at(seq[u], block_of(p, (unsigned)position[u]));
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
                    slot = slot_of(p, id[u], place);
            }
            p.positions[t] = place;
            p.slot_mapping[t] = slot;
        }
    }
    if (wrong) set_error(p.err, PA_DEVERR_BLOCK_ID);

    // Every input was read: the outputs may be the same memory.
    if (LARGE)
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

// Positions and slots of a large step, from the plan's start rows, lengths and
// tables.  The start rows are searched in shared memory.
__global__ void __launch_bounds__(kSlotThreads) step_slots_kernel(const StepPlanParams p) {
    extern __shared__ int starts[];
    pdl_wait_prerequisites();
    const int64_t base = (int64_t)blockIdx.x * (kSlotThreads * kStepUnroll) + threadIdx.x;
    const int tokens = p.query_start_loc[p.num_seqs];
    const int steps = p.num_seqs > 1 ? 32 - __clz(p.num_seqs - 1) : 0;
    if ((int64_t)blockIdx.x * (kSlotThreads * kStepUnroll) < tokens) {
        for (int s = threadIdx.x; s < p.num_seqs; s += kSlotThreads) starts[s] = p.query_start_loc[s];
        __syncthreads();
    }
    int t[kStepUnroll], seq[kStepUnroll], position[kStepUnroll];
    int32_t id[kStepUnroll];
    if (base < tokens) {
#pragma unroll
        for (int u = 0; u < kStepUnroll; ++u) t[u] = (int)min(base + u * kSlotThreads, (int64_t)tokens - 1);
        find_sequences(starts, p.num_seqs, steps, t, seq);
#pragma unroll
        for (int u = 0; u < kStepUnroll; ++u) {
            const int end = seq[u] + 1 < p.num_seqs ? starts[seq[u] + 1] : tokens;
            position[u] = p.context_lens_out[seq[u]] - (end - t[u]);
        }
#pragma unroll
        for (int u = 0; u < kStepUnroll; ++u)
            id[u] = p.block_tables[(int64_t)seq[u] * p.max_blocks + block_of(p, (unsigned)position[u])];
    }
    bool wrong = false;
#pragma unroll
    for (int u = 0; u < kStepUnroll; ++u) {
        const int64_t at = base + u * kSlotThreads;
        if (at >= p.max_tokens) continue;
        int64_t slot = -1;
        int place = -1;
        if (at < tokens) {
            place = position[u];
            const bool good = id[u] >= 0 && id[u] < p.num_blocks;
            wrong |= !good;
            if (good) slot = slot_of(p, id[u], place);
        }
        p.positions[at] = place;
        p.slot_mapping[at] = slot;
    }
    if (wrong) set_error(p.err, PA_DEVERR_BLOCK_ID);
}

cudaError_t launch(void (*kernel)(const StepPlanParams), unsigned ctas, unsigned cluster, int threads, size_t smem,
                   const StepPlanParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_step_plan(StepPlanParams p, cudaStream_t stream) {
    p.block_shift = -1;
    if ((p.block_size & (p.block_size - 1)) == 0)
        for (p.block_shift = 0; (1 << p.block_shift) < p.block_size;) ++p.block_shift;
    const bool large = p.max_tokens > kStepSmallTokens || p.num_seqs > kStepSmallSeqs;
    const size_t smem = 3 * (size_t)p.num_seqs * sizeof(int);
    if (!large) return launch(step_plan_kernel<false>, 1, 1, kStepThreads, smem, p, stream);
    constexpr int kMaxDevices = 64;
    static int configured[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(step_plan_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 3 * kMaxStepSeqs * (int)sizeof(int));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(step_slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kMaxStepSeqs * (int)sizeof(int));
        if (e != cudaSuccess) return e;
        __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
    }
    e = launch(step_plan_kernel<true>, kStepCluster, kStepCluster, kStepThreads, smem, p, stream);
    if (e != cudaSuccess || p.max_tokens == 0) return e;
    const unsigned ctas = (unsigned)(((int64_t)p.max_tokens + kSlotThreads * kStepUnroll - 1) / (kSlotThreads * kStepUnroll));
    return launch(step_slots_kernel, ctas, 1, kSlotThreads, smem / 3, p, stream);
}

}  // namespace pa
