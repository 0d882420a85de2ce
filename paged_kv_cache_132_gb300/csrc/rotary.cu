// rotary.cu -- rotary position embedding of a step's new query and key rows,
// fused with the cache write ("Efficient Memory Management for Large Language
// Model Serving with PagedAttention Review", §3-2 "fused reshape and block
// write"): the rows leave the projections once, and the keys and values enter
// their slots in the same pass.
//
// For the pair (a, b) number i of the first rotary_dim elements of a head,
//     a' = a cos_i - b sin_i,  b' = b cos_i + a sin_i
// with cos_i, sin_i from the caller's table (row = position), in binary32 and
// rounded once.
//
// Bound: HBM.  One CTA per token; a lane owns two 16-byte chunks of a head row
// that rotate together (halves: chunk c and its partner rotary_dim / 2 on;
// interleaved: two neighbours, each holding whole pairs), and the lanes of a
// row copy or rotate the same chunks of every head they visit, so a token's
// cosines and sines are loaded once per lane and stay in registers.  The first
// rows are loaded before the position is known.
//
// Measured: 85.0 us for 20 588 bf16 tokens of 32 + 2 * 8 heads of 128 with the
// keys kept (559 MB: 6.6 TB/s, 0.98 of the copy bandwidth) with 64 threads a
// token, 108.5 us with 256; 2.6 us for 256 tokens (6.4 MB) with 256 threads,
// 3.3 us with 64.
#include "attn_common.cuh"
#include "common.cuh"
#include "kernels.h"

namespace pa {
namespace {

constexpr int kRotaryThreads = 256;       // of a token's CTA in small steps, where latency counts
constexpr int kRotaryThreadsMany = 64;    // ... with many tokens: more CTAs, each with more loads in flight
// The few threads pay their passes over a token's rows one after the other, the many
// fill the GPU with fewer tokens: so the tokens are held against the lanes of a
// token's rows.  From kRotaryManyTokens tokens a lane on, 64 threads.  Measured
// (graph replays), 256 threads and 64:
//   384 lanes (48 16-bit rows of 128): 512 tokens 3.2 and 3.6 us, 768 4.4 and 3.9,
//     2048 8.2 and 6.7, 8192 40 and 33;
//   768 lanes (48 32-bit rows of 128): 1024 tokens 7.0 and 7.4 us, 1536 9.9 and 11.6,
//     2560 19.0 and 16.2;
//   960 lanes (120 16-bit rows of 128): 1024 tokens 8.7 and 10.8 us, 1536 12.7 and
//     14.5, 2048 18.6 and 17.7, 2560 26.5 and 28.9, 4096 43.0 and 41.9;
//   48 lanes (6 16-bit rows of 128): 64 tokens 2.0 and 1.9 us, 1024 3.7 and 2.3.
constexpr int kRotaryManyTokens = 2;
constexpr int kRotaryRows = 2;            // rows of a lane in flight

template <typename T>
__device__ inline uint4 pack_chunk(const float* x) {
    uint4 w;
    if constexpr (sizeof(T) == 4) {
        w = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    } else {
        w.x = pack_rn<T>(x[0], x[1]);
        w.y = pack_rn<T>(x[2], x[3]);
        w.z = pack_rn<T>(x[4], x[5]);
        w.w = pack_rn<T>(x[6], x[7]);
    }
    return w;
}

template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryParams p) {
    constexpr int V = 16 / sizeof(T);  // elements of a chunk, and pairs of a lane
    pdl_wait_prerequisites();
    // The attention's planning kernel, as after the plain cache write.  Not before
    // the wait: the plan of the step may be what comes before.
    pdl_launch_dependents();
    const int64_t token = blockIdx.x;
    const int rows_per_pass = blockDim.x / p.lanes;
    const int row0 = threadIdx.x / p.lanes;
    if (row0 >= rows_per_pass) return;
    const int c = threadIdx.x - row0 * p.lanes;
    const bool rotates = c < p.rot_lanes;
    // The lane's chunks of a row.
    const int chunk0 = INTERLEAVED || !rotates ? 2 * c : c;
    const int chunk1 = INTERLEAVED || !rotates ? 2 * c + 1 : c + p.rot_lanes;
    const bool has1 = chunk1 < p.chunks;  // false: the last lane of an odd number of chunks
    const int rows = p.num_heads + 2 * p.num_kv_heads;
    const uint4* q = static_cast<const uint4*>(p.query) + token * p.query_stride;
    const uint4* k = static_cast<const uint4*>(p.key) + token * p.key_stride;
    const uint4* v = static_cast<const uint4*>(p.value) + token * p.value_stride;

    uint4 x[kRotaryRows][2];
    auto load = [&](int r0) {
#pragma unroll
        for (int u = 0; u < kRotaryRows; ++u) {
            const int r = r0 + u * rows_per_pass;
            if (r >= rows) continue;
            const uint4* src = r < p.num_heads ? q + (int64_t)r * p.chunks
                               : r < p.num_heads + p.num_kv_heads
                                   ? k + (int64_t)(r - p.num_heads) * p.chunks
                                   : v + (int64_t)(r - p.num_heads - p.num_kv_heads) * p.chunks;
            x[u][0] = __ldcs(src + chunk0);
            if (has1) x[u][1] = __ldcs(src + chunk1);
        }
    };
    // Not through the read-only path: the kernel before may have written them
    // after this grid was launched.
    const int pos = __ldcg(p.positions + token);
    const int64_t slot = __ldcg(p.slot_mapping + token);
    load(row0);
    if (pos < 0) return;  // a padding row
    if (pos >= p.num_positions) {
        if (threadIdx.x == 0) set_error(p.err, PA_DEVERR_POSITION);
        return;
    }
    const bool cached = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots && threadIdx.x == 0) set_error(p.err, PA_DEVERR_SLOT);
    const int64_t block = cached ? slot / p.block_size : 0;
    const int64_t offset = slot - block * p.block_size;

    float cs[V], sn[V];
    if (rotates) {
        const float4* row = reinterpret_cast<const float4*>(p.cos_sin + (int64_t)pos * p.rotary_dim + c * V);
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 a = row[i], b = row[p.rotary_dim / 8 + i];
            cs[4 * i] = a.x, cs[4 * i + 1] = a.y, cs[4 * i + 2] = a.z, cs[4 * i + 3] = a.w;
            sn[4 * i] = b.x, sn[4 * i + 1] = b.y, sn[4 * i + 2] = b.z, sn[4 * i + 3] = b.w;
        }
    }

    for (int r0 = row0; r0 < rows; r0 += kRotaryRows * rows_per_pass) {
        if (r0 != row0) load(r0);
#pragma unroll
        for (int u = 0; u < kRotaryRows; ++u) {
            const int r = r0 + u * rows_per_pass;
            if (r >= rows) continue;
            const bool is_value = r >= p.num_heads + p.num_kv_heads;
            uint4 y0 = x[u][0], y1 = x[u][1];
            if (rotates && !is_value) {
                float a[V], b[V];
                unpack16(y0, a, T());
                unpack16(y1, b, T());
                if (INTERLEAVED) {
                    // pairs 0 .. V/2-1 of the lane in chunk 0, the others in chunk 1
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
                        a[2 * i] = a0 * cs[i] - a1 * sn[i];
                        a[2 * i + 1] = a1 * cs[i] + a0 * sn[i];
                        b[2 * i] = b0 * cs[V / 2 + i] - b1 * sn[V / 2 + i];
                        b[2 * i + 1] = b1 * cs[V / 2 + i] + b0 * sn[V / 2 + i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float a0 = a[i], b0 = b[i];
                        a[i] = a0 * cs[i] - b0 * sn[i];
                        b[i] = b0 * cs[i] + a0 * sn[i];
                    }
                }
                y0 = pack_chunk<T>(a);
                y1 = pack_chunk<T>(b);
            }
            if (r < p.num_heads) {
                uint4* dst = static_cast<uint4*>(p.query_out) + token * p.query_out_stride + (int64_t)r * p.chunks;
                dst[chunk0] = y0;
                if (has1) dst[chunk1] = y1;
                continue;
            }
            const int h = r - p.num_heads - (is_value ? p.num_kv_heads : 0);
            if (!is_value && p.key_out) {
                uint4* dst = static_cast<uint4*>(p.key_out) + token * p.key_out_stride + (int64_t)h * p.chunks;
                dst[chunk0] = y0;
                if (has1) dst[chunk1] = y1;
            }
            if (cached) {
                uint4* dst = static_cast<uint4*>(is_value ? p.v_cache : p.k_cache) +
                             ((block * p.num_kv_heads + h) * p.block_size + offset) * p.chunks;
                dst[chunk0] = y0;
                if (has1) dst[chunk1] = y1;
            }
        }
    }
}

template <typename T>
cudaError_t launch(const RotaryParams& p, bool interleaved, int64_t num_tokens, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)num_tokens);
    const int64_t token_lanes = ((int64_t)p.num_heads + 2 * (int64_t)p.num_kv_heads) * p.lanes;
    const bool many = num_tokens >= kRotaryManyTokens * token_lanes && p.lanes <= kRotaryThreadsMany;
    cfg.blockDim = dim3((unsigned)(many ? kRotaryThreadsMany : kRotaryThreads));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return interleaved ? cudaLaunchKernelEx(&cfg, rotary_kernel<T, true>, p)
                       : cudaLaunchKernelEx(&cfg, rotary_kernel<T, false>, p);
}

}  // namespace

bool rotary_supported(int head_dim, int rotary_dim, int elem_bytes) {
    // whole lanes of pairs, and a row's lanes in one CTA
    return rotary_dim * elem_bytes % 32 == 0 && (head_dim * elem_bytes / 16 + 1) / 2 <= kRotaryThreads;
}

cudaError_t launch_rotary(RotaryParams p, int dtype, int head_dim, int elem_bytes, bool interleaved,
                          int64_t num_tokens, cudaStream_t stream) {
    if (num_tokens == 0) return cudaSuccess;
    if (num_tokens > 0x7fffffffLL) return cudaErrorNotSupported;
    p.chunks = head_dim * elem_bytes / 16;
    p.lanes = (p.chunks + 1) / 2;
    p.rot_lanes = p.rotary_dim * elem_bytes / 32;
    const int per_chunk = 16 / elem_bytes;
    p.query_stride /= per_chunk;
    p.key_stride /= per_chunk;
    p.value_stride /= per_chunk;
    p.query_out_stride /= per_chunk;
    p.key_out_stride /= per_chunk;
    switch (dtype) {
        case PA_F32: return launch<float>(p, interleaved, num_tokens, stream);
        case PA_F16: return launch<__half>(p, interleaved, num_tokens, stream);
        case PA_BF16: return launch<__nv_bfloat16>(p, interleaved, num_tokens, stream);
        default: return cudaErrorNotSupported;
    }
}

}  // namespace pa
