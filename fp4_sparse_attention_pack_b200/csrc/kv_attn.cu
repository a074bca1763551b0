// Which kernel a call of the attention over pages takes.
#include "kv_attn.cuh"

namespace csa2 {

size_t kv_mma_workspace_bytes(int head_dim);
cudaError_t launch_kv_mma(const KvAttn& a, int head_dim, int dtype, int kv_dtype, cudaStream_t st);
size_t kv_rows_workspace_bytes(int head_dim);
cudaError_t launch_kv_rows(const KvAttn& a, int head_dim, int dtype, int kv_dtype, cudaStream_t st);

size_t kv_attn_workspace_bytes(int max_new, int H, int kv_heads, int head_dim) {
    return kv_few_rows(max_new, H / kv_heads) ? kv_rows_workspace_bytes(head_dim) : kv_mma_workspace_bytes(head_dim);
}

cudaError_t launch_kv_attn(const KvAttn& a, int head_dim, int dtype, int kv_dtype, cudaStream_t st) {
    return kv_few_rows(a.max_new, a.H / a.c.kv_heads) ? launch_kv_rows(a, head_dim, dtype, kv_dtype, st)
                                                      : launch_kv_mma(a, head_dim, dtype, kv_dtype, st);
}

}  // namespace csa2
