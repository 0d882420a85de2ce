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
// (a megabyte at most), but its loads depend on one another.  One CTA does the
// sums and the tables, with the sums in shared memory; slots and positions
// follow in the same CTA up to kTokensInPlan tokens, and in a second kernel
// over the whole GPU above that.
#include "common.cuh"
#include "kernels.h"

namespace pa {
namespace {

constexpr int kStepThreads = 1024;
constexpr int kSlotThreads = 256;
constexpr int kSlotTokens = 4;  // consecutive tokens of a thread

// Last index i in [0, n) with start[i] <= x; start[0] <= x, non-decreasing.
__device__ inline int find_sequence(const int* start, int n, int x) {
    int lo = 0, hi = n;  // start[lo] <= x < start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ inline int blocks_of(int tokens, int block_size) {
    return (int)(((unsigned)tokens + (unsigned)block_size - 1u) / (unsigned)block_size);
}

// Position and slot of one token; -1 where its block id is out of range.
__device__ inline void place_token(const StepPlanParams& p, int t, int seq, int position) {
    const int32_t id = p.block_tables[(int64_t)seq * p.max_blocks + (unsigned)position / (unsigned)p.block_size];
    const bool good = id >= 0 && id < p.num_blocks;
    if (!good) set_error(p.err, PA_DEVERR_BLOCK_ID);
    p.positions[t] = position;
    p.slot_mapping[t] =
        good ? (int64_t)id * p.block_size + (int)((unsigned)position % (unsigned)p.block_size) : -1;
}

struct Sums {
    long long tokens, given, taken;
};

__device__ inline Sums add(const Sums& a, const Sums& b) {
    return {a.tokens + b.tokens, a.given + b.given, a.taken + b.taken};
}
__device__ inline Sums shuffle_up(const Sums& a, int d) {
    return {__shfl_up_sync(0xffffffffu, a.tokens, d), __shfl_up_sync(0xffffffffu, a.given, d),
            __shfl_up_sync(0xffffffffu, a.taken, d)};
}
__device__ inline Sums inclusive_in_warp(Sums a, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sums up = shuffle_up(a, d);
        if (lane >= d) a = add(a, up);
    }
    return a;
}

// One CTA.  Every input is read before the outputs that may alias it
// (context_lens, free_state) are written.
__global__ void __launch_bounds__(kStepThreads) step_plan_kernel(const StepPlanParams p) {
    extern __shared__ int starts[];  // [num_seqs + 1] first token, [num_seqs + 1] first block given or taken
    __shared__ Sums warp_sums[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int* token_start = starts;
    int* block_start = starts + p.num_seqs + 1;
    pdl_launch_dependents();
    pdl_wait_prerequisites();

    // A thread's consecutive sequences.
    const int each = (p.num_seqs + kStepThreads - 1) / kStepThreads;
    const int s0 = min(tid * each, p.num_seqs), s1 = min(s0 + each, p.num_seqs);
    auto counts = [&](int s, int& ctx, int& grow, bool& done) {
        ctx = p.context_lens[s];
        const int n = p.new_lens[s];
        done = n == -1;
        grow = n > 0 ? n : 0;
        if (ctx < 0 || ctx > p.ctx_cap || n < -1 || grow > p.ctx_cap - ctx) {
            set_error(p.err, PA_DEVERR_CONTEXT_LEN);
            grow = 0;  // the sequence stays as it is
            done = false;
            return false;
        }
        return true;
    };
    auto count = [&](int s) {
        int ctx, grow;
        bool done;
        Sums a{0, 0, 0};
        if (!counts(s, ctx, grow, done)) return a;
        const int held = blocks_of(ctx, p.block_size);
        a.tokens = grow;
        a.given = done ? held : 0;
        a.taken = grow ? blocks_of(ctx + grow, p.block_size) - held : 0;
        return a;
    };
    Sums mine{0, 0, 0};
    for (int s = s0; s < s1; ++s) mine = add(mine, count(s));
    const Sums incl = inclusive_in_warp(mine, lane);
    if (lane == 31) warp_sums[warp] = incl;
    const int head = p.free_state[0], free_count = p.free_state[1];
    __syncthreads();
    if (warp == 0) warp_sums[lane] = inclusive_in_warp(warp_sums[lane], lane);
    __syncthreads();
    const Sums total = warp_sums[31];
    Sums at = warp ? add(warp_sums[warp - 1], incl) : incl;  // the sums before this thread's sequences
    at.tokens -= mine.tokens;
    at.given -= mine.given;
    at.taken -= mine.taken;

    const bool fits = head >= 0 && head < p.ring_size && free_count >= 0 &&
                      free_count + total.given <= p.ring_size && total.taken <= free_count + total.given &&
                      total.tokens <= p.max_tokens;
    if (!fits && tid == 0) set_error(p.err, PA_DEVERR_STEP);
    const int tokens = fits ? (int)total.tokens : 0;

    {
        Sums run = at;
        for (int s = s0; s < s1; ++s) {
            const int first = fits ? (int)run.tokens : 0;
            token_start[s] = first;
            block_start[s] = fits ? (int)run.given : 0;
            p.query_start_loc[s] = first;
            run = add(run, count(s));
        }
        if (tid == 0) {
            token_start[p.num_seqs] = tokens;
            p.query_start_loc[p.num_seqs] = tokens;
        }
    }
    // Position of entry k of the ring.
    auto ring_at = [&](long long k) {
        const long long i = head + k;  // < 2 * ring_size
        return (int)(i >= p.ring_size ? i - p.ring_size : i);
    };
    if (fits && total.given > 0) {
        __syncthreads();
        for (int k = tid; k < (int)total.given; k += kStepThreads) {
            const int s = find_sequence(block_start, p.num_seqs, k);
            const int32_t id = p.block_tables[(int64_t)s * p.max_blocks + (k - block_start[s])];
            if (id < 0 || id >= p.num_blocks) set_error(p.err, PA_DEVERR_BLOCK_ID);
            p.free_ring[ring_at((long long)free_count + k)] = id;
        }
    }
    if (fits && total.taken > 0) {
        __syncthreads();
        Sums run = at;
        for (int s = s0; s < s1; ++s) {
            block_start[s] = (int)run.taken;
            run = add(run, count(s));
        }
        __syncthreads();
        for (int k = tid; k < (int)total.taken; k += kStepThreads) {
            const int s = find_sequence(block_start, p.num_seqs, k);
            const int32_t id = p.free_ring[ring_at(k)];
            if (id < 0 || id >= p.num_blocks) set_error(p.err, PA_DEVERR_BLOCK_ID);
            const int held = blocks_of(p.context_lens[s], p.block_size);
            p.block_tables[(int64_t)s * p.max_blocks + held + (k - block_start[s])] = id;
        }
    }
    __syncthreads();
    if (p.place_tokens)
        for (int t = tid; t < p.max_tokens; t += kStepThreads) {
            if (t < tokens) {
                const int s = find_sequence(token_start, p.num_seqs, t);
                place_token(p, t, s, p.context_lens[s] + (t - token_start[s]));
            } else {
                p.positions[t] = -1;
                p.slot_mapping[t] = -1;
            }
        }
    __syncthreads();  // the inputs were read: the outputs may be the same memory
    for (int s = s0; s < s1; ++s) {
        int ctx, grow;
        bool done;
        counts(s, ctx, grow, done);
        p.context_lens_out[s] = !fits ? ctx : done ? 0 : ctx + grow;
    }
    if (tid == 0) {
        p.free_state_out[0] = fits ? ring_at(total.taken) : head;
        p.free_state_out[1] = fits ? (int)(free_count + total.given - total.taken) : free_count;
    }
}

// Slots and positions of many tokens, from the plan's start rows and lengths.
__global__ void __launch_bounds__(kSlotThreads) step_slots_kernel(const StepPlanParams p) {
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    const int tokens = p.query_start_loc[p.num_seqs];
    const int64_t first = ((int64_t)blockIdx.x * kSlotThreads + threadIdx.x) * kSlotTokens;
    int s = -1, end = 0, ctx = 0;
    for (int i = 0; i < kSlotTokens; ++i) {
        if (first + i >= p.max_tokens) return;
        const int t = (int)(first + i);
        if (t >= tokens) {
            p.positions[t] = -1;
            p.slot_mapping[t] = -1;
            continue;
        }
        if (s < 0 || t >= end) {
            s = find_sequence(p.query_start_loc, p.num_seqs, t);
            end = p.query_start_loc[s + 1];
            ctx = p.context_lens_out[s];
        }
        place_token(p, t, s, ctx - (end - t));
    }
}

cudaError_t launch_dependent(void (*kernel)(const StepPlanParams), unsigned grid, unsigned threads, size_t smem,
                             const StepPlanParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Up to here the planning CTA places the tokens itself; above it a second
// kernel does.
constexpr int kTokensInPlan = 4096;

}  // namespace

cudaError_t launch_step_plan(StepPlanParams p, cudaStream_t stream) {
    const size_t smem = 2 * ((size_t)p.num_seqs + 1) * sizeof(int);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(step_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   2 * (kMaxStepSeqs + 1) * (int)sizeof(int));
        if (e != cudaSuccess) return e;
    }
    p.place_tokens = p.max_tokens <= kTokensInPlan;
    cudaError_t e = launch_dependent(step_plan_kernel, 1, kStepThreads, smem, p, stream);
    if (e != cudaSuccess || p.place_tokens) return e;
    const unsigned ctas = (unsigned)(((int64_t)p.max_tokens + kSlotThreads * kSlotTokens - 1) / (kSlotThreads * kSlotTokens));
    return launch_dependent(step_slots_kernel, ctas, kSlotThreads, 0, p, stream);
}

}  // namespace pa
