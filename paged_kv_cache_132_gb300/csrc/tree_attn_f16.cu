// Tree attention kernels for f16 pools (head_dim 64 and 128), and the reduce kernels.
#include "tree_attn.cuh"

namespace pa {
cudaError_t launch_tree_attention_f16(const TreeAttnParams& p, int head_dim, const CUtensorMap* tq,
                                     const CUtensorMap* tk, const CUtensorMap* tv, cudaStream_t stream) {
    if (head_dim == 64) return launch_tree_attention_t<__half, 64>(p, tq, tk, tv, stream);
    if (head_dim == 128) return launch_tree_attention_t<__half, 128>(p, tq, tk, tv, stream);
    return cudaErrorNotSupported;
}
}  // namespace pa
