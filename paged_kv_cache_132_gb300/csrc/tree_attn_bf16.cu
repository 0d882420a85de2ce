// Tree attention kernels for bf16 pools (head_dim 64 and 128), and the reduce kernels.
#include "tree_attn.cuh"

namespace pa {
cudaError_t launch_tree_attention_bf16(const TreeAttnParams& p, int head_dim, const CUtensorMap* tq,
                                     const CUtensorMap* tk, const CUtensorMap* tv, cudaStream_t stream) {
    if (head_dim == 64) return launch_tree_attention_t<__nv_bfloat16, 64>(p, tq, tk, tv, stream);
    if (head_dim == 128) return launch_tree_attention_t<__nv_bfloat16, 128>(p, tq, tk, tv, stream);
    return cudaErrorNotSupported;
}
}  // namespace pa
