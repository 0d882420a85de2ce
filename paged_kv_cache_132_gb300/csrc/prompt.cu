// prompt.cu -- dispatch of the prompt attention launch by dtype.
#include "kernels.h"
#include "../../include/pa.h"

namespace pa {

cudaError_t launch_prompt_f16(const PromptParams& p, int head_dim, int sms, const CUtensorMap* tq,
                              const CUtensorMap* tk, const CUtensorMap* tv, cudaStream_t stream);
cudaError_t launch_prompt_bf16(const PromptParams& p, int head_dim, int sms, const CUtensorMap* tq,
                               const CUtensorMap* tk, const CUtensorMap* tv, cudaStream_t stream);

cudaError_t launch_prompt(const PromptParams& p, int dtype, int head_dim, int sms, const CUtensorMap* tmap_q,
                          const CUtensorMap* tmap_k, const CUtensorMap* tmap_v, cudaStream_t stream) {
    if (dtype == PA_F16) return launch_prompt_f16(p, head_dim, sms, tmap_q, tmap_k, tmap_v, stream);
    if (dtype == PA_BF16) return launch_prompt_bf16(p, head_dim, sms, tmap_q, tmap_k, tmap_v, stream);
    return cudaErrorNotSupported;
}

}  // namespace pa
