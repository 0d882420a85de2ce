// Host part of the library with its launches and the CUDA runtime's calls replaced, to
// count how often tensor maps are encoded.  No GPU is used; no pointer is followed.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdio>
#include <map>

static std::map<const void*, int> g_encoded;

static CUresult fake_encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void* base, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                            CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill) {
    ++g_encoded[base];
    return CUDA_SUCCESS;
}
static cudaError_t fake_device(int* dev) { return *dev = 0, cudaSuccess; }
static cudaError_t fake_attribute(int* value, cudaDeviceAttr, int) { return *value = 152, cudaSuccess; }
static cudaError_t fake_entry_point(const char*, void** fn, unsigned, unsigned long long,
                                    cudaDriverEntryPointQueryResult* q) {
    *fn = reinterpret_cast<void*>(&fake_encode);
    *q = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
template <class T>
static cudaError_t fake_symbol(void** p, const T&) { return *p = reinterpret_cast<void*>(0x1000), cudaSuccess; }

#define cudaGetDevice fake_device
#define cudaDeviceGetAttribute fake_attribute
#define cudaGetDriverEntryPointByVersion fake_entry_point
#define cudaGetSymbolAddress fake_symbol
#include "../paged_kv_cache_132_gb300/csrc/pa_api.cu"

namespace pa {
cudaError_t launch_reshape_and_cache(const void*, const void*, void*, void*, const int64_t*, int64_t, const PoolShape&,
                                     int*, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_copy_blocks(void* const*, void* const*, int, const int64_t*, int64_t, const PoolShape&, int*,
                               cudaStream_t) { return cudaSuccess; }
cudaError_t launch_swap_blocks(void* const*, void* const*, int64_t, void* const*, void* const*, int64_t, int,
                               const int64_t*, int64_t, const PoolShape&, int*, cudaStream_t) { return cudaSuccess; }
bool rotary_supported(int, int, int) { return true; }
cudaError_t launch_rotary(RotaryParams, int, int, int, bool, int64_t, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_step_plan(StepPlanParams, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_check_unique_slots(const int64_t*, int64_t, int*, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_check_pairs(const int64_t*, int64_t, bool, int*, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_check_decode_inputs(const int32_t*, const int32_t*, int, int, int, int, int64_t, int*,
                                       cudaStream_t) { return cudaSuccess; }
DecodeWorkspaceLayout decode_workspace_layout(int, int, int, int) { return DecodeWorkspaceLayout{}; }
cudaError_t launch_decode(const DecodeParams&, int, int, int, int, int, DecodeVariant, const CUtensorMap*,
                          const CUtensorMap*, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_prefill(const PrefillParams&, int, int, const CUtensorMap*, const CUtensorMap*, const CUtensorMap*,
                           cudaStream_t) { return cudaSuccess; }
cudaError_t launch_prompt(const PromptParams&, int, int, int, const CUtensorMap*, const CUtensorMap*,
                          const CUtensorMap*, cudaStream_t) { return cudaSuccess; }
}  // namespace pa

static char* at(int64_t mib) { return reinterpret_cast<char*>(mib << 20); }

int main(int argc, char** argv) {
    const int layers = std::atoi(argv[1]), steps = std::atoi(argv[2]);
    const bool prefill = argc > 3;
    const pa_cache_desc cache{64, 2, 16, 128, PA_BF16};
    int64_t fresh = 100000;  // activations: new memory every time
    for (int step = 0; step < steps; ++step)
        for (int l = 0; l < layers; ++l) {
            char *k = at(1 + 2 * l), *v = at(2 + 2 * l);
            const int32_t* ints = reinterpret_cast<int32_t*>(at(90000));
            char* rows = at(fresh);
            fresh += 4;
            int rc = pa_prompt_attention(at(80000), rows, 1024, rows + 4096, 256, rows + 8192, 256, ints, 2, 40, 8, 2,
                                         128, PA_BF16, 0.1f, at(70000), 1 << 20, nullptr);
            if (rc == PA_OK)
                rc = pa_decode(at(80000), PA_F32, rows, k, v, &cache, ints, 4, ints, 2, 64, 8, 2, 0.1f, 0, at(70000),
                               1 << 20, nullptr);
            if (rc == PA_OK && prefill)
                rc = pa_prefill(at(80000), PA_F32, rows + 16384, ints, 8, 8, k, v, &cache, ints, 4, ints, 2, 8, 2, 0.1f,
                                nullptr);
            if (rc != PA_OK) return std::printf("call failed: %s\n", pa_status_string(rc)), 1;
        }
    int pools = 0, rows = 0;
    for (const auto& e : g_encoded) (e.first < at(60000) ? pools : rows) += e.second;
    std::printf("%d %d\n", pools, rows);
    return 0;
}
