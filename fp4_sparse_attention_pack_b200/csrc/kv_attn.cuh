// What the three attention kernels over pages share: modes, conversions, the tensor
// maps of the pools, values that are not finite, and the join of partial results.
//
// Scores, exponentials, sums and outputs are fp32 until the output's one rounding, but
// for the probabilities: the tensor cores multiply them with the values, so they are
// rounded to the values' type (fp16 for E4M3; kv_codes.cu splits that in three).  The row
// sum adds them unrounded, as lse needs it; the roundings of many keys average out.
// Against 64 bits an output is off by 0.0023 of its size where its own rounding leaves
// 0.0017 (bf16), 0.00028 and 0.00021 (fp16), 0.0017 both ways (E4M3).  A second bf16 term
// for the rest of each probability took one token of 16 sequences to 32,768 from 205 to
// 210 us and one over 1,000 from 14.8 to 15.6 us; in the chunk kernel it would be a
// second product with V.
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

// By how much (log2 units) the reference of a row's exponentials is below the maximum when
// it is taken, where probabilities are rounded to fp16 (kv_mma.cu, kv_rows.cu).  The
// largest then lies in [2^7, 2^15], so half a step of fp16's subnormals, which smaller
// ones fall into, is 2^-32 of it: an attention sink may hide the keys behind it only by
// that much.  bf16 has fp32's range.
constexpr float below(int mode) { return mode == kBf16 ? 0.0f : 7.0f; }

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

// Queries in bf16 become fp16 times a power of two that takes the row's largest
// magnitude into [2^14, 2^15): its exponent from the largest magnitude's bits, and
// eight channels times it.
__device__ __forceinline__ uint32_t top_bits(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    return top;
}
__device__ __forceinline__ int row_exp(uint32_t top) { return top == 0 ? 0 : 14 - ((int)max(top >> 7, 1u) - 127); }
__device__ __forceinline__ uint4 scaled(const uint4& v, int e) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    const int e1 = e / 2;
    const float f1 = pow2i(e1), f2 = pow2i(e - e1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = pack16(__uint_as_float(w[i] << 16) * f1 * f2, __uint_as_float(w[i] & 0xFFFF0000u) * f1 * f2, false);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Values that are not finite.  A key that some rows of an item see and others do not has
// probability 0 for the others, but 0 x NaN and 0 x infinity are NaN.  So such elements
// are taken out of V before the product (drop_unfinite), and when the CTA's results are
// written the rows that see the key take them back (give_back).  Keys that all rows see
// need none of it.  (Taking them back at each item's end cost the E4M3 chunk kernel 5 to
// 14% in registers.)
template <int kMode>
__device__ __forceinline__ bool drop_unfinite(uint4& v) {
    constexpr uint32_t kTop = is_e4m3(kMode) ? 0x7F7F7F7Fu : kMode == kBf16 ? 0x7F807F80u : 0x7C007C00u;
    uint32_t w[4] = {v.x, v.y, v.z, v.w}, any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t hit = is_e4m3(kMode) ? __vcmpeq4(w[i] & kTop, kTop) : __vcmpeq2(w[i] & kTop, kTop);
        w[i] &= ~hit;
        any |= hit;
    }
    v = make_uint4(w[0], w[1], w[2], w[3]);
    return any != 0;
}
// Element c of a row of V where it is not finite, else 0.
template <int kMode>
__device__ __forceinline__ float unfinite_at(const uint8_t* row, int c) {
    if constexpr (is_e4m3(kMode)) return (row[c] & 0x7F) == 0x7F ? NAN : 0.0f;
    constexpr uint32_t kTop = kMode == kBf16 ? 0x7F80u : 0x7C00u;
    const uint32_t h = reinterpret_cast<const uint16_t*>(row)[c];
    if ((h & kTop) != kTop) return 0.0f;
    return kMode == kBf16 ? __uint_as_float(h << 16) : __half2float(__ushort_as_half((unsigned short)h));
}
// An output element plus such a value.
template <bool kBf>
__device__ __forceinline__ void add16(uint16_t* at, float x) {
    const float y = kBf ? __uint_as_float((uint32_t)*at << 16) : __half2float(__ushort_as_half(*at));
    *at = (uint16_t)(pack16(y + x, 0.0f, kBf) & 0xFFFF);
}

// The keys that every row of an item sees; others are seen by some rows or by none.
struct KvCommon {
    int lo, hi;
    __device__ __forceinline__ KvCommon(const KvFrag& f, int window) : lo(first_key(f.v.hi, window)), hi(f.s.n - f.s.m + f.v.t0) {}
    __device__ __forceinline__ bool has(int key) const { return key >= lo && key <= hi; }
    // a block with keys that it does not hold
    __device__ __forceinline__ bool leaves(int key0, int keys) const { return key0 < lo || key0 + keys - 1 > hi; }
};

// Whether any of the chunks that it has seen holds such an element.
template <int kMode>
struct Unfinite {
    uint32_t bits[4] = {0, 0, 0, 0};  // sums of 0 x the elements, or bit 7 of each code that is NaN
    __device__ __forceinline__ void see(const uint4& v) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (is_e4m3(kMode)) bits[i] |= (w[i] & 0x7F7F7F7Fu) + 0x01010101u;
            else if constexpr (kMode == kBf16) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(bits[i]) : "r"(w[i]), "r"(0u));
            else asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(bits[i]) : "r"(w[i]), "r"(0u));
        }
    }
    __device__ __forceinline__ bool any() const {
        return ((bits[0] | bits[1] | bits[2] | bits[3]) & (is_e4m3(kMode) ? 0x80808080u : 0x7FFF7FFFu)) != 0;
    }
};

// A warp's pass over a block of V in shared memory (kSlabs slabs of kBlk rows of kRowBytes)
// that not all rows of the item see: rows that none sees become 0, and the others lose what
// is not finite.  True if a value was taken out.
template <int kMode, int kBlk, int kRowBytes, int kSlabs, class Unseen>
__device__ __forceinline__ bool clear_rows(uint8_t* block, const KvCommon& common, int key0, const Unseen& unseen) {
    constexpr int kSteps = kSlabs * kBlk * kRowBytes / 512;  // of 512 bytes
    const int lane = threadIdx.x & 31;
    uint4* const at = reinterpret_cast<uint4*>(block) + lane;
    const auto row = [&](int k) { return (k * 512 + lane * 16) / kRowBytes % kBlk; };
#pragma unroll 4
    for (int k = 0; k < kSteps; ++k)
        if (unseen(row(k))) at[32 * k] = make_uint4(0, 0, 0, 0);
    Unfinite<kMode> found;  // (a lane reads what it has written)
#pragma unroll 4
    for (int k = 0; k < kSteps; ++k)
        if (!common.has(key0 + row(k))) found.see(at[32 * k]);
    if (!__any_sync(0xffffffffu, found.any())) return false;
#pragma unroll 1
    for (int k = 0; k < kSteps; ++k) {
        if (common.has(key0 + row(k))) continue;
        uint4 v = at[32 * k];
        if (drop_unfinite<kMode>(v)) at[32 * k] = v;
    }
    return true;
}

// The CTA's results are written; `threads` of its threads add what was taken out to the
// rows that see it.  Thread = channel of every few rows.
template <int kMode, int kDim, int kRows, int kBlk, bool kRowsFast, class Cursor>
__device__ __forceinline__ void give_back(const KvAttn& a, const KvParts& parts, int g, Cursor cur, int threads) {
    const int c = threadIdx.x % kDim;
    KvFrag f;
    while (cur.next(a, g, f)) {
        const KvCommon common(f, a.window);
        const int end = min(f.f1 * kBlk - 1, f.v.hi);
#pragma unroll 1
        for (int key = max(f.f0 * kBlk, f.v.lo); key <= end; ++key) {
            if (common.has(key)) {
                key = common.hi;
                continue;
            }
            const int page = a.c.page_table[(int64_t)f.b * a.c.max_pages + key / PAGE];
            if (page < 0 || page >= a.c.num_pages) continue;
            const int64_t row = ((int64_t)page * a.c.kv_heads + f.h) * PAGE + key % PAGE;
            const float x = unfinite_at<kMode>(a.c.v + row * kDim * (is_e4m3(kMode) ? 1 : 2), c);
            if (x == 0.0f) continue;
#pragma unroll 1
            for (int r = threadIdx.x / kDim; r < f.rows; r += threads / kDim) {
                const int q = f.tile * kRows + r, token = q / g, pos = f.s.n - f.s.m + token;
                if (key > pos || key < first_key(pos, a.window)) continue;
                if (f.first && f.last) {
                    add16<kMode == kBf16 || kMode == kE4m3Bf16>(
                        reinterpret_cast<uint16_t*>(a.out.p) + (int64_t)(f.s.row0 + token) * a.out.ts +
                            (int64_t)(f.h * g + q - token * g) * a.out.hs + c, x);
                } else {
                    float* part = reinterpret_cast<float*>(parts.o) + (2 * (int64_t)blockIdx.x + (f.first ? 1 : 0)) * kRows * kDim;
                    part[kRowsFast ? (c / 4 * kRows + r) * 4 + c % 4 : r * kDim + c] += x;
                }
            }
        }
    }
}

// The items that cuts divide.  A thread joins four channels of a row, four loads in
// flight; when the items have many partial results each (few long sequences), 4 or
// 16 threads take every 4th or 16th of them and meet in shared memory, in a fixed
// order.  A task is `width` such columns of one item; the tasks of all items are spread over the blocks, which are as many
// as run at once (a grid for each CTA that might be cut cost 4 us in waves of
// blocks that have nothing to do).  kRowsFast: a partial result lies
// [channels / 4][rows], else [rows][channels / 4].
constexpr int kJoinThreads = 256, kJoinBlocksPerSm = 4;
template <int kDim, bool kBf, bool kRowsFast>
__global__ void __launch_bounds__(kJoinThreads, kJoinBlocksPerSm)
    k_kv_join(const __grid_constant__ KvAttn a, const __grid_constant__ KvParts parts, int g, int tile_rows, int ctas) {
    __shared__ float4 s_o[kJoinThreads];
    __shared__ float2 s_ml[kJoinThreads];
    __shared__ int s_cut[kJoinThreads], s_count[kJoinThreads / 32];
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cols = tile_rows * (kDim / 4);
    for (int c0 = 0; c0 < ctas; c0 += kJoinThreads) {  // 256 CTAs' cuts at a time
        const int c = c0 + threadIdx.x;
        const bool is_cut = c < ctas && parts.cut[c].last >= 0;
        const unsigned who = __ballot_sync(0xffffffffu, is_cut);
        __syncthreads();
        if (lane == 0) s_count[warp] = __popc(who);
        __syncthreads();
        int before = 0, cuts = 0;
        for (int w = 0; w < kJoinThreads / 32; ++w) {
            before += w < warp ? s_count[w] : 0;
            cuts += s_count[w];
        }
        if (is_cut) s_cut[before + __popc(who & ((1u << lane) - 1))] = c;
        __syncthreads();
        const int n = min(kJoinThreads, ctas - c0), groups = 16 * cuts < n ? 16 : 4 * cuts < n ? 4 : 1, width = kJoinThreads / groups;
        const int tasks = cols / width, grp = threadIdx.x / width;
        for (int task = blockIdx.x; task < cuts * tasks; task += gridDim.x) {
            const int cta = s_cut[task / tasks], col = task % tasks * width + threadIdx.x % width;
            const KvCut cut = parts.cut[cta];
            const int row = kRowsFast ? col % tile_rows : col / (kDim / 4), chunk = kRowsFast ? col / tile_rows : col % (kDim / 4);
            const int all = cut.last - cta + 1;
            const bool mine = row < cut.rows;
            float M = -INFINITY, L = 0.0f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            constexpr int kMany = 4;
            for (int k0 = grp; mine && k0 < all; k0 += kMany * groups) {
                float2 ml[kMany];
                float4 o[kMany];
#pragma unroll
                for (int i = 0; i < kMany; ++i) {
                    const int k = k0 + i * groups;
                    ml[i] = make_float2(-INFINITY, 0.0f);
                    o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (k < all) {
                        const int64_t slot = 2 * (int64_t)(cta + k) + (k == 0);
                        ml[i] = parts.ml[slot * tile_rows + row];
                        o[i] = parts.o[slot * cols + col];
                    }
                }
                float m = M;
#pragma unroll
                for (int i = 0; i < kMany; ++i) m = fmaxf(m, ml[i].x);
                const float ms = m == -INFINITY ? 0.0f : m, w0 = exp2f(M - ms);
                M = m;
                L *= w0;
                acc.x *= w0, acc.y *= w0, acc.z *= w0, acc.w *= w0;
#pragma unroll
                for (int i = 0; i < kMany; ++i) {
                    const float w = exp2f(ml[i].x - ms);
                    L += w * ml[i].y;
                    acc.x += w * o[i].x, acc.y += w * o[i].y, acc.z += w * o[i].z, acc.w += w * o[i].w;
                }
            }
            if (groups > 1) {
                __syncthreads();  // the task before has been read
                s_o[threadIdx.x] = acc;
                s_ml[threadIdx.x] = make_float2(M, L);
                __syncthreads();
                if (grp > 0) continue;
                for (int k = 1; k < min(groups, all); ++k) {
                    const float2 ml = s_ml[k * width + threadIdx.x];
                    const float4 o = s_o[k * width + threadIdx.x];
                    const float m = fmaxf(M, ml.x), ms = m == -INFINITY ? 0.0f : m;
                    const float w0 = exp2f(M - ms), w1 = exp2f(ml.x - ms);
                    M = m;
                    L = L * w0 + ml.y * w1;
                    acc = make_float4(acc.x * w0 + o.x * w1, acc.y * w0 + o.y * w1, acc.z * w0 + o.z * w1, acc.w * w0 + o.w * w1);
                }
            }
            if (!mine) continue;
            const float inv = L == 0.0f ? 0.0f : 1.0f / L;
            const int r = cut.row0 + row;
            const int64_t token = cut.token0 + r / g;
            const int head = cut.head0 + r % g;
            uint2 w = make_uint2(pack16(acc.x * inv, acc.y * inv, kBf), pack16(acc.z * inv, acc.w * inv, kBf));
            if (L == 0.0f) w = make_uint2(0, 0);
            *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out.p) + token * a.out.ts + (int64_t)head * a.out.hs + 4 * chunk) = w;
            if (a.lse && chunk == 0) a.lse[token * a.H + head] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
        }
        __syncthreads();  // s_cut has been read
    }
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

// A pool as rows of head_dim channels; boxes of 64 rows x `width` bytes.
inline bool make_pool_map(CUtensorMap* m, const void* base, int64_t rows, int dim, int mode, int width, CUtensorMapSwizzle swizzle) {
    auto fn = kv_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)dim, (cuuint64_t)rows};
    const int elem = is_e4m3(mode) ? 1 : 2;
    cuuint64_t strides[1] = {(cuuint64_t)dim * elem};
    cuuint32_t box[2] = {(cuuint32_t)(width / elem), PAGE};
    cuuint32_t estr[2] = {1, 1};
    const CUtensorMapDataType type = is_e4m3(mode)  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                     : mode == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launch `kernel` so that its start overlaps the end of the launch before it
// (it waits for that with cudaGridDependencySynchronize).
template <typename... Args>
cudaError_t launch_behind(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

// Calls of at most 16 rows to an item go to the few-rows kernel.  (8 sequences over
// 32,768, 64 / 8 heads of 128: one token 169 us there, 178 us in the chunk kernel; two
// 171 and 183 us; one token with heads of 64 97 and 126 us.  Two tiles of 16 rows in
// it, 4 tokens each: 348 us against 181 us in the chunk kernel.)
inline bool kv_few_rows(int max_new, int g) { return (int64_t)max_new * g <= 16; }

// Calls over E4M3 pages with at most 32 rows to an item: the tensor cores read the
// codes.  (8 sequences over 65,536, 64 / 8 heads of 128: one token 174 us against 386 us
// in the chunk kernel, which widens codes in shared memory, 4 tokens 235 against 392 us;
// heads of 64: 126 against 331 and 197 against 333 us.  More rows in this form would
// need more than 3 x 32 columns of each product in TMEM.)
inline bool kv_codes(int max_new, int g, int kv_dtype) {
    return kv_dtype == CSA2_KV_E4M3 && (int64_t)max_new * g <= 32;
}

}  // namespace csa2
