// Which kernel a call of the attention over pages takes.
#include "kv.cuh"

namespace csa2 {

size_t kv_mma_workspace_bytes(int head_dim);
cudaError_t launch_kv_mma(const KvAttn& a, int head_dim, int dtype, int kv_dtype, cudaStream_t st);

size_t kv_attn_workspace_bytes(int max_new, int H, int kv_heads, int head_dim) {
    (void)max_new, (void)H, (void)kv_heads;
    return kv_mma_workspace_bytes(head_dim);
}

cudaError_t launch_kv_attn(const KvAttn& a, int head_dim, int dtype, int kv_dtype, cudaStream_t st) {
    return launch_kv_mma(a, head_dim, dtype, kv_dtype, st);
}

}  // namespace csa2
