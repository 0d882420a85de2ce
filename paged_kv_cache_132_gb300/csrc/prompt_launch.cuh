// prompt_launch.cuh -- launch of one prompt attention kernel instance: one CTA
// per SM (fewer when there are fewer items), 512 threads, launched as a
// programmatic dependent of the kernel before it.
#pragma once

#include "prompt.cuh"

namespace pa {

template <typename T, int D>
cudaError_t launch_prompt_t(const PromptParams& p, int sms, const CUtensorMap* tq, const CUtensorMap* tk,
                            const CUtensorMap* tv, cudaStream_t stream) {
    using Shape = PromptShape<D>;
    constexpr int kMaxDevices = 64;
    static int configured[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(prompt_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Shape::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
    }
    const int64_t items = prompt_max_units(p.num_tokens, p.num_seqs, p.tile_tokens) * p.num_kv_heads;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(items < sms ? items : sms));
    cfg.blockDim = dim3(Shape::THREADS);
    cfg.dynamicSmemBytes = Shape::SMEM_BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prompt_kernel<T, D>, p, *tq, *tk, *tv);
}

}  // namespace pa
