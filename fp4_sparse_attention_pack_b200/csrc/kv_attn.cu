// Which kernel a call of the attention over pages takes.
#include "kv_attn.cuh"

namespace csa2 {

size_t kv_mma_workspace_bytes(int head_dim);
cudaError_t launch_kv_mma(const KvAttn& a, int head_dim, int dtype, int kv_dtype, cudaStream_t st);
size_t kv_rows_workspace_bytes(int head_dim);
cudaError_t launch_kv_rows(const KvAttn& a, int head_dim, int dtype, cudaStream_t st);

size_t kv_codes_workspace_bytes(bool few, int head_dim);
cudaError_t launch_kv_codes(const KvAttn& a, bool few, int head_dim, int dtype, cudaStream_t st);

size_t kv_attn_workspace_bytes(int max_new, int H, const csa2_kv_cache& c) {
    const int g = H / c.kv_heads;
    if (kv_codes(max_new, g, c.dtype)) return kv_codes_workspace_bytes(kv_few_rows(max_new, g), c.head_dim);
    return kv_few_rows(max_new, g) ? kv_rows_workspace_bytes(c.head_dim) : kv_mma_workspace_bytes(c.head_dim);
}

cudaError_t launch_kv_attn(const KvAttn& a, int head_dim, int dtype, int kv_dtype, cudaStream_t st) {
    const int g = a.H / a.c.kv_heads;
    if (kv_codes(a.max_new, g, kv_dtype)) return launch_kv_codes(a, kv_few_rows(a.max_new, g), head_dim, dtype, st);
    return kv_few_rows(a.max_new, g) ? launch_kv_rows(a, head_dim, dtype, st)
                                     : launch_kv_mma(a, head_dim, dtype, kv_dtype, st);
}

}  // namespace csa2
