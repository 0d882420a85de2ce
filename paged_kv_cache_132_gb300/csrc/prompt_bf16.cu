// Prompt attention kernels for bf16 rows (head_dim 64 and 128).
#include "prompt_launch.cuh"

namespace pa {
cudaError_t launch_prompt_bf16(const PromptParams& p, int head_dim, int sms, const CUtensorMap* tq,
                              const CUtensorMap* tk, const CUtensorMap* tv, cudaStream_t stream) {
    if (head_dim == 64) return launch_prompt_t<__nv_bfloat16, 64>(p, sms, tq, tk, tv, stream);
    if (head_dim == 128) return launch_prompt_t<__nv_bfloat16, 128>(p, sms, tq, tk, tv, stream);
    return cudaErrorNotSupported;
}
}  // namespace pa
