// prompt.cu -- work list of the prompt attention, and its launch by dtype.
#include "common.cuh"
#include "kernels.h"

namespace pa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanBuckets = 128;

// Sequences by their number of units: 0..15 exactly, above that four buckets
// per factor of two.
__device__ inline int plan_bucket(int units) {
    if (units < 16) return units;
    const int e = 31 - __clz(units);
    return 16 + (e - 4) * 4 + ((units >> (e - 2)) & 3);  // < 128 for every positive int
}

// The units of every sequence, the longest sequences first and of each the
// last query tiles (the longest key ranges) first: the attention's CTAs take
// them in this order from a counter, so what is left for the end is short.
// One CTA, two passes over the start rows (a histogram of the units by bucket;
// the units at their bucket's place, in any order inside a bucket).
__global__ void __launch_bounds__(kPlanThreads) prompt_plan_kernel(const PromptParams p) {
    __shared__ int place[kPlanBuckets];
    __shared__ unsigned long long rows;  // of all sequences
    __shared__ int4 placed[kPlanThreads];  // first row, length, units, place of the first unit
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < kPlanBuckets) place[threadIdx.x] = 0;
    if (threadIdx.x == 0) rows = 0;
    pdl_launch_dependents();
    pdl_wait_prerequisites();
    __syncthreads();
    const int span = 2 * p.tile_tokens;
    auto sequence = [&](int s, int& row0, int& len) {
        row0 = len = 0;
        if (s >= p.num_seqs) return;
        const int a = __ldcg(p.query_start + s), b = __ldcg(p.query_start + s + 1);
        if (a < 0 || b < a || b > p.num_tokens) {
            set_error(p.err, PA_DEVERR_CONTEXT_LEN);
            return;
        }
        row0 = a;
        len = b - a;
    };
    unsigned long long warp_rows = 0;
    for (int s0 = threadIdx.x - lane; s0 < p.num_seqs; s0 += kPlanThreads) {
        int row0, len;
        sequence(s0 + lane, row0, len);
        const int units = (len + span - 1) / span;
        if (units) atomicAdd(&place[plan_bucket(units)], units);
        // a warp's sum needs 36 bits: two of 21
        warp_rows += __reduce_add_sync(0xffffffffu, (unsigned)len & 0xffffu) +
                     ((unsigned long long)__reduce_add_sync(0xffffffffu, (unsigned)len >> 16) << 16);
    }
    if (lane == 0 && warp_rows) atomicAdd(&rows, warp_rows);
    __syncthreads();
    if (rows > (unsigned long long)p.num_tokens) {
        // Sequences that overlap: the list need not have room for them.
        if (threadIdx.x == 0) {
            set_error(p.err, PA_DEVERR_CONTEXT_LEN);
            *p.num_units = 0;
            *p.next_item = 0;
        }
        return;
    }
    if (threadIdx.x < 32) {
        // Places of the buckets, the largest first: lane l has buckets 127 - 4 l ... 124 - 4 l.
        int before[4], run = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            before[k] = run;
            run += place[kPlanBuckets - 1 - 4 * lane - k];
        }
        int incl = run;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += up;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) place[kPlanBuckets - 1 - 4 * lane - k] = incl - run + before[k];
        if (lane == 31) {
            *p.num_units = incl;  // <= max_units: the sequences' rows do not exceed num_tokens
            *p.next_item = 0;
        }
    }
    __syncthreads();
    // A place for each sequence by a thread, and up to 4 units; more units by a warp.
    for (int base = 0; base < p.num_seqs; base += kPlanThreads) {
        int row0, len;
        sequence(base + threadIdx.x, row0, len);
        const int units = (len + span - 1) / span;
        const int at = units ? atomicAdd(&place[plan_bucket(units)], units) : 0;
        const bool wide = units > 4;
        placed[threadIdx.x] = make_int4(row0, len, wide ? units : 0, at);
        if (!wide)
            for (int k = 0; k < units; ++k) p.items[at + k] = make_int4(row0, len, units - 1 - k, 0);
        if (!__syncthreads_or(wide)) continue;
        for (int s = threadIdx.x >> 5; s < kPlanThreads && base + s < p.num_seqs; s += kPlanThreads / 32) {
            const int4 q = placed[s];
            for (int k = lane; k < q.z; k += 32) p.items[q.w + k] = make_int4(q.x, q.y, q.z - 1 - k, 0);
        }
        __syncthreads();
    }
}

cudaError_t launch_prompt_plan(const PromptParams& p, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prompt_plan_kernel, p);
}

}  // namespace

cudaError_t launch_prompt_f16(const PromptParams& p, int head_dim, int sms, const CUtensorMap* tq,
                              const CUtensorMap* tk, const CUtensorMap* tv, cudaStream_t stream);
cudaError_t launch_prompt_bf16(const PromptParams& p, int head_dim, int sms, const CUtensorMap* tq,
                               const CUtensorMap* tk, const CUtensorMap* tv, cudaStream_t stream);

cudaError_t launch_prompt(const PromptParams& p, int dtype, int head_dim, int sms, const CUtensorMap* tmap_q,
                          const CUtensorMap* tmap_k, const CUtensorMap* tmap_v, cudaStream_t stream) {
    if (p.items) {
        const cudaError_t e = launch_prompt_plan(p, stream);
        if (e != cudaSuccess) return e;
    }
    if (dtype == PA_F16) return launch_prompt_f16(p, head_dim, sms, tmap_q, tmap_k, tmap_v, stream);
    if (dtype == PA_BF16) return launch_prompt_bf16(p, head_dim, sms, tmap_q, tmap_k, tmap_v, stream);
    return cudaErrorNotSupported;
}

}  // namespace pa
