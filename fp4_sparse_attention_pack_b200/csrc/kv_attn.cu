// Attention of new tokens over the pages, one warp for each (token, head): the
// plain online softmax over the visible keys, every lane holding dim / 32
// channels of the query and of the output.
#include <type_traits>

#include "kv.cuh"

namespace csa2 {

namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float kv_to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float kv_to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float kv_to_float(__nv_fp8_e4m3 v) { return (float)v; }
__device__ __forceinline__ void kv_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void kv_store(__half* p, float v) { *p = __float2half_rn(v); }

template <typename T, typename C, int kDim>
__global__ void __launch_bounds__(32 * kWarps) k_kv_attn_plain(const __grid_constant__ KvAttn a) {
    const int lane = threadIdx.x & 31;
    const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (w >= (int64_t)a.total * a.H) return;
    const int t = (int)(w / a.H), h = (int)(w % a.H);
    int lo = 0, hi = a.c.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    const NewTokens nt = new_tokens(a.cu, lo, a.total, a.max_new);
    if (nt.m < 0) {
        if (lane == 0) atomicOr(a.c.status, CSA2_DEVERR_COUNT);
        return;
    }
    if (t < nt.row0 || t >= nt.row0 + nt.m) return;
    const int n = kv_held(a.c, lo);
    const int p = n - nt.m + (t - nt.row0);
    const int first = a.window > 0 ? max(0, p - a.window + 1) : 0;
    constexpr int kPer = kDim / 32;
    float q[kPer], o[kPer], m = -INFINITY, l = 0.0f;
    const T* qp = reinterpret_cast<const T*>(a.q.p) + t * a.q.ts + h * a.q.hs;
#pragma unroll
    for (int i = 0; i < kPer; ++i) q[i] = kv_to_float(qp[lane + 32 * i]), o[i] = 0.0f;
    const int hk = h / (a.H / a.c.kv_heads);
    for (int j = first; j <= p; ++j) {
        const int page = kv_page(a.c, lo, j / PAGE);
        if (page < 0) continue;
        const int64_t at = (((int64_t)page * a.c.kv_heads + hk) * PAGE + j % PAGE) * kDim;
        const C* kp = reinterpret_cast<const C*>(a.c.k) + at;
        const C* vp = reinterpret_cast<const C*>(a.c.v) + at;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) s += q[i] * kv_to_float(kp[lane + 32 * i]);
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale;
        const float mn = fmaxf(m, s), f = mn == -INFINITY ? 1.0f : expf(m - mn), e = mn == -INFINITY ? 0.0f : expf(s - mn);
        l = l * f + e;
#pragma unroll
        for (int i = 0; i < kPer; ++i) o[i] = o[i] * f + e * kv_to_float(vp[lane + 32 * i]);
        m = mn;
    }
    T* op = reinterpret_cast<T*>(a.out.p) + t * a.out.ts + h * a.out.hs;
    const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
#pragma unroll
    for (int i = 0; i < kPer; ++i) kv_store(op + lane + 32 * i, o[i] * inv);
    if (a.lse && lane == 0) a.lse[(int64_t)t * a.H + h] = l == 0.0f ? -INFINITY : m + logf(l);
}

template <typename T, typename C>
cudaError_t attn_as(const KvAttn& a, int dim, cudaStream_t st) {
    const int64_t rows = (int64_t)a.total * a.H;
    const unsigned grid = (unsigned)((rows + kWarps - 1) / kWarps);
    if (dim == 64) k_kv_attn_plain<T, C, 64><<<grid, 32 * kWarps, 0, st>>>(a);
    else k_kv_attn_plain<T, C, 128><<<grid, 32 * kWarps, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t kv_attn_workspace_bytes(int max_new, int H, int kv_heads, int head_dim) {
    (void)max_new, (void)H, (void)kv_heads, (void)head_dim;
    return 0;
}

cudaError_t launch_kv_attn(const KvAttn& a, int head_dim, int dtype, int kv_dtype, cudaStream_t st) {
    const bool e4m3 = kv_dtype == CSA2_KV_E4M3;
    if (dtype == CSA2_DTYPE_BF16)
        return e4m3 ? attn_as<__nv_bfloat16, __nv_fp8_e4m3>(a, head_dim, st)
                    : attn_as<__nv_bfloat16, __nv_bfloat16>(a, head_dim, st);
    return e4m3 ? attn_as<__half, __nv_fp8_e4m3>(a, head_dim, st) : attn_as<__half, __half>(a, head_dim, st);
}

}  // namespace csa2
