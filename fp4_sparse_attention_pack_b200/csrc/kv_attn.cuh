// What the two attention kernels over pages share: modes, conversions, the tensor
// maps of the pools, and the join of partial results.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <cfloat>

#include "kv_plan.cuh"

namespace csa2 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGap = 8.0f;  // log2 units by which a block may exceed the maximum in use

// Types of (cache, queries): 16-bit ones of one type, or an E4M3 cache.
enum Mode { kBf16, kF16, kE4m3Bf16, kE4m3F16 };
constexpr bool is_e4m3(int mode) { return mode >= kE4m3Bf16; }

struct KvMaps {
    CUtensorMap k, v;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool bf) {
    uint32_t r;
    if (bf)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// x 2^e in two factors that are floats; never 0 for a positive x, so that a masked
// score times it is -infinity.
__device__ __forceinline__ float times_pow2(float x, int e) {
    const int e1 = e / 2;
    return fmaxf(x * pow2i(e1) * pow2i(e - e1), FLT_MIN);
}

// A 16-byte chunk of a row of bf16 queries, held by kChunks neighbouring lanes,
// to fp16 times 2^e, which takes the row's largest magnitude into [2^14, 2^15).
// Returns e.
template <int kChunks>
__device__ __forceinline__ int scale_row(uint4& v) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
#pragma unroll
    for (int d = kChunks / 2; d; d >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    const int e = top == 0 ? 0 : 14 - ((int)max(top >> 7, 1u) - 127);
    const int e1 = e / 2;
    const float f1 = pow2i(e1), f2 = pow2i(e - e1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = pack16(__uint_as_float(w[i] << 16) * f1 * f2, __uint_as_float(w[i] & 0xFFFF0000u) * f1 * f2, false);
    v = make_uint4(w[0], w[1], w[2], w[3]);
    return e;
}

// The items that a range's end divides: blockIdx.x the CTA that begins it,
// blockIdx.y 32 of its rows (a warp's lanes); the warps share the channels.
template <int kDim, bool kBf>
__global__ void __launch_bounds__(128) k_kv_join(const __grid_constant__ KvAttn a, const __grid_constant__ KvParts parts,
                                                 int g, int tile_rows) {
    cudaGridDependencySynchronize();
    const int cta = blockIdx.x;
    const int4 cut = parts.cut[cta];
    if (cut.w < 0) return;
    const KvSeq s = kv_seq(a, cut.x);
    const int row = 32 * blockIdx.y + (threadIdx.x & 31);
    const int64_t r = (int64_t)cut.z * tile_rows + row;
    if (r >= (int64_t)s.m * g) return;
    float M = -INFINITY, L = 0.0f;
    for (int k = cta; k <= cut.w; ++k) {
        const float2 ml = parts.ml[(2 * (int64_t)k + (k == cta)) * tile_rows + row];
        M = fmaxf(M, ml.x);
    }
    const float Ms = M == -INFINITY ? 0.0f : M;
    float4 acc[kDim / 16];
#pragma unroll
    for (int i = 0; i < kDim / 16; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = cta; k <= cut.w; ++k) {
        const int64_t slot = 2 * (int64_t)k + (k == cta);
        const float2 ml = parts.ml[slot * tile_rows + row];
        const float w = exp2f(ml.x - Ms);
        L += ml.y * w;
#pragma unroll
        for (int i = 0; i < kDim / 16; ++i) {
            const float4 o = parts.o[(slot * (kDim / 4) + (threadIdx.x >> 5) + 4 * i) * tile_rows + row];
            acc[i].x += w * o.x, acc[i].y += w * o.y, acc[i].z += w * o.z, acc[i].w += w * o.w;
        }
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    const int64_t token = s.row0 + r / g;
    const int head = cut.y * g + (int)(r % g);
    uint16_t* out = reinterpret_cast<uint16_t*>(a.out.p) + token * a.out.ts + (int64_t)head * a.out.hs;
#pragma unroll
    for (int i = 0; i < kDim / 16; ++i) {
        uint2 w = make_uint2(pack16(acc[i].x * inv, acc[i].y * inv, kBf), pack16(acc[i].z * inv, acc[i].w * inv, kBf));
        if (L == 0.0f) w = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(out + 4 * ((threadIdx.x >> 5) + 4 * i)) = w;
    }
    if (a.lse && threadIdx.x < 32) a.lse[token * a.H + head] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
}

inline PFN_cuTensorMapEncodeTiled_v12000 kv_encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void* p = nullptr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
    }();
    return fn;
}

// A pool as rows of head_dim channels; boxes of 64 rows x 128 bytes (64 bytes
// when a row is no longer), swizzled by their width.
inline bool make_pool_map(CUtensorMap* m, const void* base, int64_t rows, int dim, int mode) {
    auto fn = kv_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)dim, (cuuint64_t)rows};
    const int elem = is_e4m3(mode) ? 1 : 2, width = dim * elem < 128 ? dim * elem : 128;
    cuuint64_t strides[1] = {(cuuint64_t)dim * elem};
    cuuint32_t box[2] = {(cuuint32_t)(width / elem), PAGE};
    cuuint32_t estr[2] = {1, 1};
    const CUtensorMapDataType type = is_e4m3(mode)  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : mode == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launch `kernel` so that its start overlaps the end of the launch before it.
template <typename... Args>
cudaError_t launch_behind(void (*kernel)(Args...), dim3 grid, int threads, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

// Rows to an item of the few-rows kernel for calls of at most max_new tokens a
// sequence: 16 or 32, or 0 when they are more (the chunk kernel's calls).
inline int kv_rows_tile(int max_new, int g) {
    const int64_t rows = (int64_t)max_new * g;
    return rows <= 16 ? 16 : 0;
}

}  // namespace csa2
