// Attention over the pages for few query rows (a decode step, drafted tokens): at
// most 16 rows (token, head of the group) to a sequence and kv head.
//
// Every key and value is read once and used for all the rows, some 2 x rows
// flops a byte, so the cache's bytes bound it.  A page of 64 keys is a stage of
// a TMA ring (64 to 92 KB of pages in each of two CTAs an SM); warp w of four
// takes its keys 16 w .. 16 w + 15 with an online softmax of its own, so the
// warps meet only at an item's end:
//
//   S = Q K^T   mma m16n8k16 (rows x 16 keys, K = head_dim)
//   P = 2^(c S - m), kept in registers: the accumulators of S are P's operand
//   O += P V    mma m16n8k16 (K = 16 keys)
//
// (mma.sync, not tcgen05: 16 rows of its 128 would be used, and the operands come
// out of registers without a hand-over.)  Caches of 16 bits; kv_codes.cu takes E4M3.
// The work is cut evenly over the CTAs (kv_plan.cuh), which splits long
// sequences when there are few.
//
// One token of 16 sequences to 32,768, 64 / 8 heads of 128, bf16: 205 to 211 us by the
// machine (6.2 to 6.4 TB/s, 97% of the copy rate and more); heads of 64: 85%.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cstring>

#include "kv_attn.cuh"
#include "kv_plan.cuh"
#include "sm100.cuh"

namespace csa2 {

namespace {

using namespace sm100;

constexpr int kRows = 16;      // of an item
constexpr int kWarps = 4;
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kOver = 3;       // an item's start and end, in pages
constexpr int kMinPer = 6;     // least cost of a CTA's range
constexpr int kSnap = 1;
constexpr int kCtasPerSm = 2;

template <int kDim, int kMode>
struct __align__(1024) Smem {
    static constexpr int kSlabs = kDim / 64;  // of 128-byte rows
    static constexpr int kPageBytes = PAGE * kDim * 2;
    static constexpr int kQStride = kDim * 2 + 16;
    static constexpr int kRedBytes = 2 * kRows * kDim * 4;  // two warps' sums
    static constexpr int kRoom = 112 * 1024 - kRedBytes - kRows * kQStride - 2048;
    static constexpr int kStages = kRoom / (2 * kPageBytes) < 12 ? kRoom / (2 * kPageBytes) : 12;
    uint8_t kv[kStages][2][kPageBytes];
    uint8_t q[kRows][kQStride];
    float red[2][kRows][kDim];
    float ml[kWarps][kRows][2];
    uint8_t bad[kStages];
    int unfinite;  // values were taken out
    KvCursor<kRows, PAGE, kOver> cur;  // the CTA's, for them
    uint64_t full[kStages], empty[kStages];
    int abort;
};

template <class S>
__device__ __forceinline__ bool wait_bar_warp(S& sm, uint64_t* bar, uint32_t parity) {
    bool ok = mbar_try(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) {
        const uint64_t t0 = global_ns();
        while (!ok) {
            if (*reinterpret_cast<volatile int*>(&sm.abort)) break;
            ok = mbar_try_sleep(bar, parity, 20000u);
            if (!ok && global_ns() - t0 > kWaitNs) {
                atomicExch(&sm.abort, 1);
                break;
            }
        }
        ok = __all_sync(0xffffffffu, ok);
    }
    return ok;
}

// Byte offset of 16-byte chunk c (of the whole row) of a page's row r: slabs of
// 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ uint32_t at16(int r, int c) {
    return (c >> 3) * (PAGE * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

template <bool kBf>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (kBf)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void warps_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

using Cursor = KvCursor<kRows, PAGE, kOver>;

// ---------------------------------------------------------------- loads

template <int kDim, int kMode>
__device__ void role_load(Smem<kDim, kMode>& sm, const KvAttn& a, const KvMaps& maps, int g, Cursor cur) {
    using S = Smem<kDim, kMode>;
    const int lane = threadIdx.x & 31;
    int st = 0;
    uint32_t phase = 0, used = 0;
    KvFrag f;
    bool alive = true;
    while (alive && cur.next(a, g, f)) {
        const int32_t* table = a.c.page_table + (int64_t)f.b * a.c.max_pages;
        int ids = -1;
        for (int j = f.f0; j < f.f1; ++j) {
            if (j == f.f0 || (j & 31) == 0) {  // 32 page ids at a time, one to a lane
                const int pg = (j & ~31) + lane;
                ids = pg >= f.f0 && pg < f.f1 ? table[pg] : -1;
            }
            const int id = __shfl_sync(0xffffffffu, ids, j & 31);
            const bool good = id >= 0 && id < a.c.num_pages;
            if (used >= S::kStages && !(alive = wait_bar_warp(sm, &sm.empty[st], phase ^ 1))) break;
            ++used;
            if (lane == 0) {
                sm.bad[st] = !good;
                if (!good) atomicOr(a.c.status, CSA2_DEVERR_PAGE);
            }
            __syncwarp();
            mbar_expect_tx_w(&sm.full[st], good ? 2 * S::kPageBytes : 0);
            if (good) {  // the whole warp issues each box
#pragma unroll
                for (int i = 0; i < 2 * S::kSlabs; ++i) {
                    const int v = i / S::kSlabs, c = i % S::kSlabs;
                    tma_load_2d_nohint_w(&sm.kv[st][v][c * PAGE * 128], v ? &maps.v : &maps.k,
                                         64 * c, (id * a.c.kv_heads + f.h) * PAGE, &sm.full[st]);
                }
            }
            __syncwarp();
            if (++st == S::kStages) st = 0, phase ^= 1;
        }
    }
    if (*reinterpret_cast<volatile int*>(&sm.abort)) {  // no copy is in flight when the CTA ends
        for (uint32_t k = 0; k < min(used, (uint32_t)S::kStages); ++k) {
            const int s = (st + S::kStages - 1 - (int)k) % S::kStages;
            (void)mbar_wait(&sm.full[s], s < st ? phase : phase ^ 1);
        }
    }
}

// ---------------------------------------------------------------- rows

// A warp takes what is not finite out of its 16 rows of V that some rows of the item see
// and others do not; true for a lane that found such a value.
template <int kDim, int kMode>
__device__ __forceinline__ bool drop_rows(uint8_t* page, int row0, int page_key, KvCommon common) {
    const int lane = threadIdx.x & 31;
    bool any = false;
    for (int i = lane; i < 16 * (kDim / 8); i += 32) {
        const int r = row0 + (i & 15);
        if (common.has(page_key + r)) continue;
        uint4* at = reinterpret_cast<uint4*>(page + at16(r, i >> 4));
        uint4 v = *at;
        if (drop_unfinite<kMode>(v)) {
            *at = v;
            any = true;
        }
    }
    fence_proxy_async_smem();  // the stage is next written by a TMA
    __syncwarp();
    return any;
}

template <int kDim, int kMode>
__device__ void role_rows(Smem<kDim, kMode>& sm, const KvAttn& a, const KvParts& parts, int64_t per, int g,
                          Cursor cur) {
    using S = Smem<kDim, kMode>;
    constexpr bool kBf = kMode == kBf16;
    constexpr int kKs = kDim / 16, kNt = kDim / 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quad = lane >> 2, qc = lane & 3;
    const float c0 = fmaxf(a.scale * kLog2e, FLT_MIN);
    int st = 0;
    uint32_t phase = 0;
    KvFrag f;
    while (cur.next(a, g, f)) {
        const int nb = f.f1 - f.f0;
        if (nb > 0) {
            // ---- the item's queries, in the operands' type
            constexpr int kCh = kDim / 8;  // 16-byte chunks of a row
            for (int i = threadIdx.x; i < kRows * kCh; i += 32 * kWarps) {
                const int r = i / kCh, c = i % kCh;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (r < f.rows) {
                    const int t = r / g;
                    v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.q.p) +
                                                        (int64_t)(f.s.row0 + t) * a.q.ts +
                                                        (int64_t)(f.h * g + r - t * g) * a.q.hs + 8 * c);
                }
                *reinterpret_cast<uint4*>(&sm.q[r][16 * c]) = v;
            }
            warps_sync();
        }
        uint32_t qf[kKs][4];
        int pos[2], lo[2];
        float mref[2], l[2];
        float o[kNt][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = min(quad + 8 * e, f.rows - 1);
            pos[e] = f.s.n - f.s.m + r / g;
            lo[e] = first_key(pos[e], a.window);
            mref[e] = -INFINITY, l[e] = 0.0f;
        }
        const int pos_min = f.s.n - f.s.m, lo_max = first_key(f.v.hi, a.window);
#pragma unroll
        for (int t = 0; t < kNt; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[t][e] = 0.0f;
        if (nb > 0) {
#pragma unroll
            for (int ks = 0; ks < kKs; ++ks) ldsm4(smem_u32(&sm.q[lane & 15][32 * ks + 16 * (lane >> 4)]), qf[ks]);
        }
        for (int j = f.f0; j < f.f1; ++j) {
            // a wait that gave up does not end the loop: the warps meet at the same barriers
            const bool there = wait_bar_warp(sm, &sm.full[st], phase);
            const int kb = j * PAGE + 16 * warp;  // the warp's keys
            if (there && !sm.bad[st] && kb <= f.v.hi && kb + 15 >= f.v.lo) {
                const uint32_t kp = smem_u32(sm.kv[st][0]), vp = smem_u32(sm.kv[st][1]);
                const bool edge = kb + 15 > f.v.hi || kb < f.v.lo;
                if (edge) {  // rows of V that no query sees: zero, as 0 x NaN is not
                    for (int i = lane; i < 16 * (kDim / 8); i += 32) {
                        const int r = i & 15, key = kb + r;
                        if (key > f.v.hi || key < f.v.lo)
                            *reinterpret_cast<uint4*>(sm.kv[st][1] + at16(16 * warp + r, i >> 4)) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();  // the stage is next written by a TMA
                    __syncwarp();
                }
                // ---- S
                float s[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[t][e] = 0.0f;
                const int kr = 16 * warp + (lane & 7) + ((lane >> 4) << 3);  // ldmatrix row of this lane
#pragma unroll
                for (int ks = 0; ks < kKs; ++ks) {
                    uint32_t b[4];
                    ldsm4(kp + at16(kr, 2 * ks + ((lane >> 3) & 1)), b);
                    mma16816<kBf>(s[0], qf[ks], b[0], b[1]);
                    mma16816<kBf>(s[1], qf[ks], b[2], b[3]);
                }
                // ---- softmax: elements 0, 1 of row quad, 2, 3 of row quad + 8
                if (kb + 15 > pos_min || kb < lo_max) {
                    if (f.s.m > 1 && drop_rows<kDim, kMode>(sm.kv[st][1], 16 * warp, kb - 16 * warp, KvCommon(f, a.window)))
                        sm.unfinite = 1;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = kb + 8 * t + 2 * qc + (e & 1);
                            if (key > pos[e >> 1] || key < lo[e >> 1]) s[t][e] = -INFINITY;
                        }
                }
                float bm[2];
                bool move = false;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = fmaxf(fmaxf(s[0][2 * e], s[0][2 * e + 1]), fmaxf(s[1][2 * e], s[1][2 * e + 1]));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                    bm[e] = x * c0;
                    bm[e] -= below(kMode);
                    move = move || bm[e] > mref[e] + kGap || (mref[e] == -INFINITY && bm[e] > -INFINITY);
                }
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mn = fmaxf(mref[e], bm[e]);
                        const float x = mn == -INFINITY ? 1.0f : ex2(mref[e] - mn);
                        mref[e] = mn;
                        l[e] *= x;
#pragma unroll
                        for (int t = 0; t < kNt; ++t) o[t][2 * e] *= x, o[t][2 * e + 1] *= x;
                    }
                }
                uint32_t p[4];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float ms = mref[e] == -INFINITY ? 0.0f : mref[e];
                        const float x = ex2(fmaf(s[t][2 * e], c0, -ms));
                        const float y = ex2(fmaf(s[t][2 * e + 1], c0, -ms));
                        l[e] += x + y;
                        p[2 * t + e] = pack16(x, y, kBf);
                    }
                // ---- O
                const int vr = 16 * warp + (lane & 15);
#pragma unroll
                for (int t = 0; t < kNt; t += 2) {
                    uint32_t b[4];  // (keys 0-7, 8 channels), (keys 8-15, ..), the next 8 channels
                    ldsm4t(vp + at16(vr, t + (lane >> 4)), b);
                    mma16816<kBf>(o[t], p, b[0], b[1]);
                    mma16816<kBf>(o[t + 1], p, b[2], b[3]);
                }
            }
            __syncwarp();
            mbar_arrive_w(&sm.empty[st]);
            if (++st == S::kStages) st = 0, phase ^= 1;
        }
        // ---- the warps' sums over their keys, joined in a fixed order
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            if (qc == 0) {
                sm.ml[warp][quad + 8 * e][0] = mref[e];
                sm.ml[warp][quad + 8 * e][1] = l[e];
            }
        }
        warps_sync();
        float w[2];  // weight of this warp's sums
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = quad + 8 * e;
            const float M = fmaxf(fmaxf(sm.ml[0][r][0], sm.ml[1][r][0]), fmaxf(sm.ml[2][r][0], sm.ml[3][r][0]));
            w[e] = M == -INFINITY ? 1.0f : ex2(mref[e] - M);  // no key seen: zeros, or NaN scores' NaN
        }
        auto place = [&](bool add, int buf) {
#pragma unroll
            for (int t = 0; t < kNt; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float2* d = reinterpret_cast<float2*>(&sm.red[buf][quad + 8 * e][8 * t + 2 * qc]);
                    float2 v = make_float2(o[t][2 * e] * w[e], o[t][2 * e + 1] * w[e]);
                    if (add) {
                        const float2 u = *d;
                        v.x += u.x, v.y += u.y;
                    }
                    *d = v;
                }
        };
        if (warp < 2) place(false, warp);
        warps_sync();
        if (warp >= 2) place(true, warp - 2);
        warps_sync();
        // ---- the output, or the range's partial sums
        const bool whole = f.first && f.last;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (f.first ? 1 : 0);
        for (int i = threadIdx.x; i < kRows * (kDim / 8); i += 32 * kWarps) {
            const int r = i / (kDim / 8), c = i % (kDim / 8);
            float M = -INFINITY, L = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) M = fmaxf(M, sm.ml[k][r][0]);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) L += sm.ml[k][r][1] * (M == -INFINITY ? 1.0f : ex2(sm.ml[k][r][0] - M));
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 x = *reinterpret_cast<const float4*>(&sm.red[0][r][8 * c + e]);
                const float4 y = *reinterpret_cast<const float4*>(&sm.red[1][r][8 * c + e]);
                v[e] = x.x + y.x, v[e + 1] = x.y + y.y, v[e + 2] = x.z + y.z, v[e + 3] = x.w + y.w;
            }
            if (whole) {
                if (r >= f.rows) continue;
                const int t = r / g, head = f.h * g + r - t * g;
                const int64_t token = f.s.row0 + t;
                const float inv = L == 0.0f ? 0.0f : 1.0f / L;
                uint32_t u[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) u[e] = L == 0.0f ? 0u : pack16(v[2 * e] * inv, v[2 * e + 1] * inv, kBf);
                *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out.p) + token * a.out.ts + (int64_t)head * a.out.hs +
                                          8 * c) = make_uint4(u[0], u[1], u[2], u[3]);
                if (a.lse && c == 0) a.lse[token * a.H + head] = L == 0.0f ? -INFINITY : (M + log2f(L)) * kLn2;
            } else {
                float4* po = parts.o + (slot * kRows + r) * (kDim / 4) + 2 * c;
                po[0] = make_float4(v[0], v[1], v[2], v[3]);
                po[1] = make_float4(v[4], v[5], v[6], v[7]);
                if (c == 0) parts.ml[slot * kRows + r] = make_float2(M, L);
            }
        }
        if (!whole && f.first && threadIdx.x == 0)
            parts.cut[blockIdx.x] = kv_cut<kSnap>(f, blockIdx.x, per, g, kRows);
        warps_sync();  // the buffers are free for the next item
    }
}

template <int kDim, int kMode>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    k_kv_rows(const __grid_constant__ KvAttn a, const __grid_constant__ KvMaps maps, const __grid_constant__ KvPlan plan,
              const __grid_constant__ KvParts parts) {
    extern __shared__ uint8_t smem_raw[];
    using S = Smem<kDim, kMode>;
    S& sm = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    static_assert(sizeof(KvPlanSmem) <= sizeof(sm.kv), "the plan's arrays lie in the ring");
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], kWarps);
        }
        sm.abort = 0;
        sm.unfinite = 0;
        fence_mbar_init();
    }
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    if (threadIdx.x == 0) parts.cut[blockIdx.x].last = -1;
    int64_t per;
    const Cursor cur = kv_plan<kRows, PAGE, kOver, kSnap>(a, plan, *reinterpret_cast<KvPlanSmem*>(sm.kv), &per);
    if (threadIdx.x == 0) sm.cur = cur;
    fence_proxy_async_smem();  // the plan's arrays were written by ordinary stores
    __syncthreads();
    if (threadIdx.x < 32 * kWarps) role_rows<kDim, kMode>(sm, a, parts, per, plan.g, cur);
    else role_load<kDim, kMode>(sm, a, maps, plan.g, cur);
    __syncwarp();
    __syncthreads();
    if (sm.abort && threadIdx.x == 0) atomicOr(a.c.status, CSA2_DEVERR_TIMEOUT);
    if (sm.unfinite && threadIdx.x < 32 * kWarps)
        give_back<kMode, kDim, kRows, PAGE, false>(a, parts, plan.g, sm.cur, 32 * kWarps);
}

template <int kDim, int kMode>
cudaError_t rows_as(const KvAttn& a, cudaStream_t st) {
    using S = Smem<kDim, kMode>;
    constexpr int kSmem = sizeof(S) + 1024;
    static_assert(kCtasPerSm * (kSmem + 1024) <= 233472, "two CTAs an SM");
    static_assert(S::kStages >= 2, "a ring");
    KvMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    const int64_t rows = (int64_t)a.c.num_pages * a.c.kv_heads * PAGE;
    if (!make_pool_map(&maps.k, a.c.k, rows, kDim, kMode, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !make_pool_map(&maps.v, a.c.v, rows, kDim, kMode, 128, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    KvPlan plan;
    plan.g = a.H / a.c.kv_heads;
    plan.grid = kCtasPerSm * device_sm_count();
    plan.min_per = kMinPer;
    const KvParts parts = kv_parts(a.ws, plan.grid, kRows, kDim);
    static std::atomic<uint64_t> attr_done{0};
    cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(k_kv_rows<kDim, kMode>), kSmem, attr_done);
    if (e != cudaSuccess) return e;
    e = launch_behind(k_kv_rows<kDim, kMode>, dim3(plan.grid), kThreads, kSmem, st, a, maps, plan, parts);
    if (e != cudaSuccess) return e;
    constexpr bool kBf = kMode == kBf16;
    return launch_behind(k_kv_join<kDim, kBf, false>, dim3(kJoinBlocksPerSm * device_sm_count()), kJoinThreads, 0, st, a, parts, plan.g, kRows, plan.grid);
}

}  // namespace

size_t kv_rows_workspace_bytes(int head_dim) {
    return kv_parts_bytes(kCtasPerSm * device_sm_count(), kRows, head_dim);
}

cudaError_t launch_kv_rows(const KvAttn& a, int head_dim, int dtype, cudaStream_t st) {
    const bool bf = dtype == CSA2_DTYPE_BF16;
    if (head_dim == 64) return bf ? rows_as<64, kBf16>(a, st) : rows_as<64, kF16>(a, st);
    return bf ? rows_as<128, kBf16>(a, st) : rows_as<128, kF16>(a, st);
}

}  // namespace csa2
