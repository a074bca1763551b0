// Attention over E4M3 pages for few query rows (at most 16 or 32 rows of token x head
// of the group to a sequence and kv head): the tensor cores read the codes themselves
// (tcgen05.mma kind::f8f6f4, fp32 accumulation in TMEM), so no page is widened.
//
// Keys and values are the operand with 128 rows, queries and probabilities the one
// with N columns, each split into three E4M3 terms of four bits (12 bits together,
// one more than fp16):
//
//   S^T [128 keys][3 R]     = K [128][128] . (q1 q2 q3)^T     s = S1 + S2 2^-5 + S3 2^-10
//   O^T [128 channels][3 R] += V^T [128][128] . (p1 p2 p3)    o = O1 + O2 2^-5 + O3 2^-10
//
// where x1 = rn(x), x2 = rn(2^5 (x - x1)), x3 = rn(2^5 (2^5 (x - x1) - x2)); R is 16 or
// 32.  Of |x| <= 2^8 a rounding leaves at most 2^3, so 2^5 times it is in range again.
// A row's queries are scaled by a power of two that takes the largest into [2^7, 2^8),
// undone in the softmax scale; the third term is a multiple of 2^-19, so a query is
// exact to 2^-20, 2^-27 of the largest.
// Probabilities are rounded to fp16 first and then split.  The reference of a row's
// exponentials is its maximum less 4 (log2) when it is taken, and moves when a score
// exceeds it by more than 8: the largest probability lies in [2^4, 2^8], E4M3's range,
// and the third term's rounding, 2^-20, is at most 2^-24 of it.  (Less 5 or 6 would
// move it more often: 4 and 20% longer with 32 rows.)
//
// One CTA an SM, 384 threads, blocks of 128 keys:
//   warps 0-3, 4-7  softmax of even and odd blocks, each with sums and a maximum of
//                   its own: thread = key (TMEM lane of S^T); at an item's end thread
//                   = channel (lane of O^T);
//   warp 8          issues the MMAs;
//   warps 9, 11     load pages by TMA, K and V (one warp for both took 1,600 cycles a
//                   block, more than the bytes);
//   warp 10         loads and splits the queries and tells the others which item is next.
//
// The cache's bytes bound it: one token of 8 sequences over 65,536, 64 / 8 heads of
// 128, takes 174 us (6.2 TB/s, 96% of the copy rate).  With 32 rows (4 tokens each) it
// takes 235 to 253 us by the machine (66 to 71%): no pipe is more than a third busy
// (issue slots 33%), so it waits in the two groups' chains scores - split - product,
// some 470 instructions a thread and block.  Heads of 64, whose blocks have half the
// bytes and the same chain: 126 and 197 us (66%, 42%).
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

constexpr int kBlk = 128;    // keys of a block
constexpr int kOver = 2;     // an item's start and end, in blocks
constexpr int kMinPer = 4;   // least cost of a CTA's range
constexpr int kSnap = 1;
constexpr int kThreads = 384, kRegsLaunch = 168;
// Registers of a softmax thread and of the others.
template <int R>
constexpr int kRegsSoftmax = R == 32 ? 200 : kRegsLaunch;
template <int R>
constexpr int kRegsOther = R == 32 ? 104 : kRegsLaunch;
constexpr int kWarpMma = 8, kWarpK = 9, kWarpQ = 10, kWarpV = 11;
constexpr int places_of(int dim) { return dim == 64 ? 16 : 10; }  // K and V blocks in the order of their use
constexpr int kRing = 16;    // blocks whose masks of bad pages are kept
constexpr uint32_t kTmemCols = 512, kColS = 0, kColO = 256;  // two of each, 128 columns apart
constexpr float kNone = -FLT_MAX / 2;                         // reference before any score
constexpr float kBelow = 4.0f;                                // by which a reference is below the maximum

template <int kDim, int R>
struct Smem {
    static constexpr int kPlaces = places_of(kDim);
    alignas(16) uint8_t kv[kPlaces][kBlk * kDim];  // [key][channel], swizzled by its width
    uint8_t p[2][kBlk * 128];                     // [key][3 R codes], SW128
    uint8_t q[3 * R * kDim];                      // [term][row][channel], as kv
    float4 cm[2][R / 2];                          // (c, -reference) of two rows each
    float factor[2][R];
    float wmax[2][4][32], wsum[2][4][32];
    float2 pair[R];                               // odd blocks' (reference, sum)
    float2 join[R];                               // weights of even and odd blocks' sums
    float c[2][R];                                // softmax scale of each row (per item parity)
    int pos[2][R];                                // its last key
    uint8_t bad[kRing];                           // bit p: page p of the block is outside the pool
    int unfinite;                                 // values were taken out
    KvCursor<R, kBlk, kOver> cur;                 // the CTA's, for them
    uint64_t full[kPlaces], empty[kPlaces];
    uint64_t q_full, q_empty, s_full[2], p_full[2], o_done[2], tail, drained;
    uint64_t frag_full[2], frag_empty[2], pair_full, pair_empty;
    KvFrag frag[2];
    uint32_t tmem_base;
    int abort;
};

// Byte offset of 16-byte chunk c of row r of `width` bytes with the swizzle of that width.
template <int width>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    return width == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Bounded wait of a warp that also gives up when another role has given up.
template <class S>
__device__ __forceinline__ bool wait_bar(S& sm, uint64_t* bar, uint32_t parity) {
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

// The four warps of a group.
__device__ __forceinline__ void group_sync(int t) { asm volatile("bar.sync %0, 128;" ::"r"(1 + t) : "memory"); }
__device__ __forceinline__ bool group_any(int t, bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(1 + t), "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

template <int R>
using Cursor = KvCursor<R, kBlk, kOver>;

__device__ __forceinline__ uint32_t h2_to_codes(uint32_t h) {  // two fp16 to two codes
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}
// The next term's value: 2^5 (h - its code).
__device__ __forceinline__ uint32_t rest16(uint32_t h, uint32_t code) {
    uint32_t b = e4m3x2_to_h2(code), r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(b));
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(r), "r"(0x50005000u));  // 32
    return r;
}
// Two values of fp16 into three terms of two codes.
__device__ __forceinline__ void split(uint32_t h, uint32_t (&e)[3]) {
    e[0] = h2_to_codes(h);
    h = rest16(h, e[0]);
    e[1] = h2_to_codes(h);
    h = rest16(h, e[1]);
    e[2] = h2_to_codes(h);
}

// ---------------------------------------------------------------- MMA

template <int kDim, int R>
__device__ void role_mma(Smem<kDim, R>& sm, uint32_t tb) {
    // kind::f8f6f4 has the fields of kind::f16; format 0 is E4M3
    const uint32_t idesc_s = idesc_f16(128, 3 * R, 0, 0, 0), idesc_o = idesc_f16(128, 3 * R, 0, 1, 1);
    constexpr uint32_t kLayout = kDim == 128 ? kLayoutSw128 : kLayoutSw64;
    const uint64_t desc_q = smem_desc(sm.q, 16, 8 * kDim, kLayout);
    const uint64_t desc_k = smem_desc(sm.kv[0], 16, 8 * kDim, kLayout);
    // heads of 64: the product has 128 rows all the same, those behind the 64th come
    // from what lies behind the block, and nothing reads them
    const uint64_t desc_v = smem_desc(sm.kv[0], kBlk * kDim, 8 * kDim, kLayout);
    const uint64_t desc_p = smem_desc(sm.p[0], 16, 1024, kLayoutSw128);
    int place = 0;
    uint32_t phase = 0, items = 0, np[2] = {0, 0};
    auto step = [&] {
        tc_commit_w(&sm.empty[place]);
        if (++place == Smem<kDim, R>::kPlaces) place = 0, phase ^= 1;
    };
    auto scores = [&](int t) {  // S_t^T = K q^T
        if (!wait_bar(sm, &sm.full[place], phase)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < kDim / 32; ++ks)
            tc_mma_f8_w(tb + kColS + 128 * t, desc_k + (uint32_t)(place * (kBlk * kDim) >> 4) + 2 * ks, desc_q + 2 * ks, idesc_s, ks > 0);
        tc_commit_w(&sm.s_full[t]);
        step();
        return true;
    };
    for (uint32_t n = 0;; ++n) {
        if (!wait_bar(sm, &sm.frag_full[n & 1], (n >> 1) & 1)) return;
        const int nb = sm.frag[n & 1].f1 - sm.frag[n & 1].f0, rows = sm.frag[n & 1].rows;
        if (rows == 0) return;
        __syncwarp();
        mbar_arrive_w(&sm.frag_empty[n & 1]);
        if (nb == 0) continue;
        if (!wait_bar(sm, &sm.q_full, items & 1)) return;
        ++items;
        for (int t = 0; t < min(nb, 2); ++t)
            if (!scores(t)) return;
        if (nb <= 2) tc_commit_w(&sm.q_empty);
        for (int j = 0; j < nb; ++j) {
            const int t = j & 1;
            if (!wait_bar(sm, &sm.full[place], phase)) return;
            if (!wait_bar(sm, &sm.p_full[t], np[t] & 1)) return;
            ++np[t];
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)  // O_t^T += V^T p, 32 keys at a time
                tc_mma_f8_w(tb + kColO + 128 * t, desc_v + (uint32_t)((place * (kBlk * kDim) + ks * 32 * kDim) >> 4),
                            desc_p + (uint32_t)((t * (kBlk * 128) + ks * 4096) >> 4), idesc_o, j > 1 || ks > 0);
            step();
            if (j + 2 < nb) {
                if (!scores(t)) return;
                if (j + 3 == nb) tc_commit_w(&sm.q_empty);
            } else {
                tc_commit_w(&sm.o_done[t]);
            }
        }
    }
}

// ---------------------------------------------------------------- loads

// The ring holds K0 K1 V0 K2 V1 .. of an item's nb blocks, the order of their use.
__device__ __forceinline__ int place_in_item(int j, int nb, bool is_v) {
    if (is_v) return j == nb - 1 ? 2 * nb - 1 : 2 * j + 2;
    return j == 0 ? 0 : 2 * j - 1;
}

template <int kDim, int R, bool kV>
__device__ void role_tma(Smem<kDim, R>& sm, const KvAttn& a, const KvMaps& maps, int g, Cursor<R> cur) {
    constexpr int kPage = PAGE * kDim, kPlaces = Smem<kDim, R>::kPlaces;
    const int lane = threadIdx.x & 31;
    uint32_t base = 0, tails = 0, blocks = 0;
    uint32_t issued = 0, parity = 0;  // places that this warp filled, and in which turn of the ring
    KvFrag f;
    bool alive = true;
    while (alive && cur.next(a, g, f)) {
        const int32_t* table = a.c.page_table + (int64_t)f.b * a.c.max_pages;
        const int nb = f.f1 - f.f0, first = f.v.lo / PAGE, last = f.v.hi / PAGE;
        const KvCommon common(f, a.window);
        int ids = -1, have = -1;  // 32 page ids at a time, one to a lane
        for (int x = 0; x < nb && alive; ++x) {
            const int j = f.f0 + x;
            if (have != 2 * j / 32) {
                have = 2 * j / 32;
                const int pg = 32 * have + lane;
                ids = pg >= first && pg <= last ? table[pg] : -1;
            }
            int page[2], bad = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int id = __shfl_sync(0xffffffffu, ids, (2 * j + i) & 31), pg = 2 * j + i;
                const bool need = pg >= first && pg <= last, good = id >= 0 && id < a.c.num_pages;
                page[i] = need && good ? id : -1;
                if (need && !good) bad |= 1 << i;
            }
            const uint32_t at = base + place_in_item(x, nb, kV), turn = at / kPlaces;
            const int place = at % kPlaces;
            if (turn > 0 && !(alive = wait_bar(sm, &sm.empty[place], (turn - 1) & 1))) break;
            if (!kV) {
                if (lane == 0) {
                    sm.bad[(blocks + x) % kRing] = (uint8_t)bad;
                    if (bad) atomicOr(a.c.status, CSA2_DEVERR_PAGE);
                }
                __syncwarp();
            }
            // rows of V that no query sees are zeroed when they are there, as 0 x NaN is not 0
            const bool part = kV && (common.leaves(j * kBlk, kBlk) || bad);
            uint64_t* bar = part ? &sm.tail : &sm.full[place];
            const uint32_t bytes = ((page[0] >= 0) + (page[1] >= 0)) * kPage;
            if (!part || bytes) {
                mbar_expect_tx_w(bar, bytes);
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (page[i] >= 0)
                        tma_load_2d_nohint_w(&sm.kv[place][i * kPage], kV ? &maps.v : &maps.k, 0, (page[i] * a.c.kv_heads + f.h) * PAGE, bar);
            }
            if (!part) {
                issued |= 1u << place;
                parity = (parity & ~(1u << place)) | (turn & 1) << place;
                continue;
            }
            if (bytes) {
                // its own copy: waited for even when the others have given up
                if (!__all_sync(0xffffffffu, mbar_wait(&sm.tail, tails & 1))) {
                    atomicExch(&sm.abort, 1);
                    alive = false;
                    break;
                }
                ++tails;
            }
            const auto unseen = [&](int r) {
                const int key = j * kBlk + r;
                return key < f.v.lo || key > f.v.hi || (bad >> (r >> 6) & 1);
            };
            if (clear_rows<kE4m3Bf16, kBlk, kDim, 1>(sm.kv[place], common, j * kBlk, unseen)) sm.unfinite = 1;
            fence_proxy_async_smem();
            __syncwarp();
            mbar_arrive_w(&sm.full[place]);
        }
        base += 2 * nb;
        blocks += nb;
    }
    // No copy is in flight when the CTA ends, also after a wait that gave up.  One limit
    // for all: a place that the other warp has filled since may never show its parity.
    if (*reinterpret_cast<volatile int*>(&sm.abort)) {
        const uint64_t t0 = global_ns();
        for (int p = 0; p < kPlaces; ++p)
            while (issued >> p & 1 && !mbar_try(&sm.full[p], parity >> p & 1) && global_ns() - t0 < kWaitNs);
    }
}

// Queries: a pair of lanes to a row, every other eight channels each.
template <int kDim, int R, bool kBf>
__device__ void role_q(Smem<kDim, R>& sm, const KvAttn& a, int g, Cursor<R> cur) {
    const int tid = threadIdx.x - 32 * kWarpQ, odd = tid & 1;
    const float c0 = fmaxf(a.scale * kLog2e, FLT_MIN);
    uint32_t items = 0;
    KvFrag f;
    for (uint32_t n = 0;; ++n) {
        const bool more = cur.next(a, g, f);
        if (n > 1 && !wait_bar(sm, &sm.frag_empty[n & 1], ((n >> 1) - 1) & 1)) return;
        if (tid == 0) {  // tells the others which item is next
            if (!more) f.rows = 0;
            sm.frag[n & 1] = f;
            mbar_arrive(&sm.frag_full[n & 1]);
        }
        __syncwarp();
        if (!more) return;
        if (f.f1 == f.f0) continue;
        if (items > 0 && !wait_bar(sm, &sm.q_empty, (items - 1) & 1)) return;
#pragma unroll 1
        for (int row = tid >> 1; row < R; row += 16) {
            const bool mine = row < f.rows;
            const int r = min(row, f.rows - 1), tok = r / g;
            const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q.p) + (int64_t)(f.s.row0 + tok) * a.q.ts +
                                  (int64_t)(f.h * g + r - tok * g) * a.q.hs + 8 * odd;
            constexpr int kCh = kDim / 16;
            uint4 v[kCh];
            uint32_t top = 0;  // of the magnitudes' bits
#pragma unroll
            for (int k = 0; k < kCh; ++k) {
                v[k] = mine ? *reinterpret_cast<const uint4*>(src + 16 * k) : make_uint4(0, 0, 0, 0);
                top = max(top, top_bits(v[k]));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            float big;
            if constexpr (kBf) big = __uint_as_float(top << 16);
            else big = __half2float(__ushort_as_half((unsigned short)top));
            const int e = big == 0.0f ? 0 : 7 - ((int)max(__float_as_uint(big) >> 23, 1u) - 127);
            // E4M3 has no infinity: a row that holds one becomes NaN, as its softmax is (its
            // scores are infinities, or NaN)
            const float f1 = big < INFINITY ? pow2i(e / 2) : NAN, f2 = pow2i(e - e / 2);
#pragma unroll
            for (int k = 0; k < kCh; ++k) {
                const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
                uint32_t out[3][2] = {};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float lo, hi;
                    if constexpr (kBf) {
                        lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xFFFF0000u);
                    } else {
                        lo = __half2float(__ushort_as_half((unsigned short)(w[i] & 0xFFFF)));
                        hi = __half2float(__ushort_as_half((unsigned short)(w[i] >> 16)));
                    }
                    uint32_t t[3];
                    split(pack16(lo * f1 * f2, hi * f1 * f2, false), t);
#pragma unroll
                    for (int s = 0; s < 3; ++s) out[s][i >> 1] |= t[s] << (16 * (i & 1));
                }
#pragma unroll
                for (int s = 0; s < 3; ++s)  // channels 16 k + 8 odd ..
                    *reinterpret_cast<uint2*>(&sm.q[swizzled<kDim>(s * R + row, k) + 8 * odd]) = make_uint2(out[s][0], out[s][1]);
            }
            if (!odd) {
                sm.c[items & 1][row] = times_pow2(c0, -e);
                sm.pos[items & 1][row] = f.s.n - f.s.m + tok;
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_w(&sm.q_full);
        ++items;
    }
}

// ---------------------------------------------------------------- softmax

// Sum of v[i] over the warp's lanes, for lane i (the upper half of 16 values: twice).
template <int R>
__device__ __forceinline__ float lane_sums(float (&v)[R], int lane) {
#pragma unroll
    for (int d = R / 2; d; d >>= 1) {
#pragma unroll
        for (int i = 0; i < d; ++i) {
            const bool up = lane & d;
            const float give = up ? v[i] : v[i + d], keep = up ? v[i + d] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, d);
        }
    }
    float s = v[0];
    if constexpr (R == 16) s += __shfl_xor_sync(0xffffffffu, s, 16);
    return s;
}

// R columns of a warp's TMEM lanes; the wait is the caller's.
template <int R>
__device__ __forceinline__ void load_cols(uint32_t taddr, float (&v)[R]) {
    if constexpr (R == 32) tmem_ld_32x32b_x32(taddr, v);
    else tmem_ld_32x32b_x16(taddr, v);
}
template <int R>
__device__ __forceinline__ void store_cols(uint32_t taddr, const float (&v)[R]) {
    if constexpr (R == 32) tmem_st_32x32b_x32(taddr, v);
    else tmem_st_32x32b_x16(taddr, v);
}
// The three terms' columns joined.
template <int R>
__device__ __forceinline__ void load_terms(uint32_t taddr, float (&v)[R]) {
    float b[R];
    load_cols<R>(taddr, v);
    load_cols<R>(taddr + R, b);
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = fmaf(b[r], 0x1p-5f, v[r]);
    load_cols<R>(taddr + 2 * R, b);
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = fmaf(b[r], 0x1p-10f, v[r]);
}

// Waits that give up do not end the loops, so that a group's warps meet at the same
// barriers; the results are not used then.
template <int kDim, int R, bool kBf>
__device__ void role_softmax(Smem<kDim, R>& sm, const KvAttn& a, const KvParts& parts, int64_t per, int g, uint32_t tb) {
    const int t = threadIdx.x >> 7, thr = threadIdx.x & 127, warp = thr >> 5, lane = threadIdx.x & 31;
    const uint32_t lane_base = tb + ((uint32_t)(32 * warp) << 16);
    const uint32_t ts = lane_base + kColS + 128 * t, to = lane_base + kColO + 128 * t;
    const int row = lane % R;
    uint32_t ns = 0, no = 0, items = 0, blocks = 0, pairs = 0;
    for (uint32_t n = 0;; ++n) {
        if (group_any(t, !wait_bar(sm, &sm.frag_full[n & 1], (n >> 1) & 1))) return;
        const KvFrag& f = sm.frag[n & 1];
        if (f.rows == 0) return;
        const int nb = f.f1 - f.f0, j0 = f.f0, j1 = f.f1, first = j0 + t;
        const int it = items & 1, blk0 = blocks;
        if (nb > 0) ++items;
        blocks += nb;
        const int pos_min = f.s.n - f.s.m, window = a.window;
        const int lo_max = first_key(f.v.hi, window);
        float l[R];
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] = 0.0f;
        for (int j = first; j < j1; j += 2) {
            wait_bar(sm, &sm.s_full[t], ns & 1);
            ++ns;
            tc_fence_after();
            if (j == first) {  // the scores' arrival tells that the queries and their scales are there
                if (thr < R) reinterpret_cast<float2*>(sm.cm[t])[thr] = make_float2(sm.c[it][thr], -kNone);
                group_sync(t);
            }
            float x[R];
            load_terms<R>(ts, x);
            const int key = j * kBlk + thr;
            const int bad = sm.bad[(blk0 + j - j0) % kRing];
            if (bad || j * kBlk + kBlk - 1 > pos_min || j * kBlk < lo_max) {
                const bool gone = bad >> (thr >> 6) & 1;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int p = sm.pos[it][r];
                    if (gone || key > p || (window > 0 && key <= p - window)) x[r] = -INFINITY;  // p >= -32
                }
            }
            float y[R], top = -INFINITY;
#pragma unroll
            for (int r = 0; r < R; r += 2) {
                const float4 cm = sm.cm[t][r / 2];
                y[r] = fmaf(x[r], cm.x, cm.y);
                y[r + 1] = fmaf(x[r + 1], cm.z, cm.w);
                top = fmaxf(top, fmaxf(y[r], y[r + 1]));
            }
            if (group_any(t, top > kGap)) {
                // each row's largest score over the block: lane r of a warp takes row r's
                float mine = -INFINITY;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    int i = __float_as_int(x[r]);
                    i = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7FFFFFFF));  // in the order of the floats
                    if (row == r) mine = __int_as_float(i ^ ((i >> 31) & 0x7FFFFFFF));
                }
                sm.wmax[t][warp][lane] = mine;
                group_sync(t);
                const float2 cm = reinterpret_cast<const float2*>(sm.cm[t])[row];
                const float most = fmaxf(fmaxf(sm.wmax[t][0][row], sm.wmax[t][1][row]), fmaxf(sm.wmax[t][2][row], sm.wmax[t][3][row])) * cm.x;
                const float old = -cm.y, now = most > old + kGap ? most - kBelow : old;
                group_sync(t);
                if (warp == 0 && lane < R) {
                    sm.factor[t][lane] = ex2(old - now);
                    reinterpret_cast<float2*>(sm.cm[t])[lane] = make_float2(cm.x, -now);
                }
                group_sync(t);
#pragma unroll
                for (int r = 0; r < R; ++r) l[r] *= sm.factor[t][r];
                if (j > first) {  // O holds the blocks before
#pragma unroll 1
                    for (int s = 0; s < 3; ++s) {
                        float o[R];
                        load_cols<R>(to + s * R, o);
#pragma unroll
                        for (int r = 0; r < R; ++r) o[r] *= sm.factor[t][r];
                        store_cols<R>(to + s * R, o);
                    }
                }
#pragma unroll
                for (int r = 0; r < R; r += 2) {
                    const float4 c2 = sm.cm[t][r / 2];
                    y[r] = fmaf(x[r], c2.x, c2.y);
                    y[r + 1] = fmaf(x[r + 1], c2.z, c2.w);
                }
            }
#pragma unroll
            for (int r0 = 0; r0 < R; r0 += 16) {
                uint32_t out[3][4] = {};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float e0 = ex2(y[r0 + 2 * i]), e1 = ex2(y[r0 + 2 * i + 1]);
                    l[r0 + 2 * i] += e0;
                    l[r0 + 2 * i + 1] += e1;
                    uint32_t c[3];
                    split(pack16(e0, e1, false), c);
#pragma unroll
                    for (int s = 0; s < 3; ++s) out[s][i >> 1] |= c[s] << (16 * (i & 1));
                }
#pragma unroll
                for (int s = 0; s < 3; ++s)
                    *reinterpret_cast<uint4*>(&sm.p[t][swizzled<128>(thr, (s * R + r0) >> 4)]) = make_uint4(out[s][0], out[s][1], out[s][2], out[s][3]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            mbar_arrive_w(&sm.p_full[t]);
        }
        // ---- the item's end
        if (first < j1) {
            wait_bar(sm, &sm.o_done[t], no & 1);
            ++no;
            tc_fence_after();
        }
        sm.wsum[t][warp][lane] = lane_sums<R>(l, lane);
        group_sync(t);
        const float L = (sm.wsum[t][0][row] + sm.wsum[t][1][row]) + (sm.wsum[t][2][row] + sm.wsum[t][3][row]);
        const float M = first < j1 ? -reinterpret_cast<const float2*>(sm.cm[t])[row].y : kNone;
        const bool both = nb > 1;  // the even blocks' group joins the two
        if (t == 1) {
            if (both) {
                if (thr < R) sm.pair[thr] = make_float2(M, L);
                tc_fence_before();
                __syncwarp();
                mbar_arrive_w(&sm.pair_full);
                wait_bar(sm, &sm.pair_empty, pairs & 1);
            }
        } else {
            const bool whole = f.first && f.last;
            float m = M, s = L, w0 = 1.0f, w1 = 0.0f;
            if (both) {
                wait_bar(sm, &sm.pair_full, pairs & 1);
                tc_fence_after();
                const float2 o = sm.pair[row];
                m = fmaxf(M, o.x);
                w0 = ex2(M - m), w1 = ex2(o.x - m);
                s = L * w0 + o.y * w1;
            }
            if (m == kNone) m = -INFINITY;
            const int64_t slot = 2 * (int64_t)blockIdx.x + (f.first ? 1 : 0);
            const bool none = whole && s == 0.0f;  // no key was seen: zeros, whatever the sums hold
            const float inv = whole ? 1.0f / s : 1.0f;
            if (thr < f.rows) {
                sm.join[thr] = none ? make_float2(-1.0f, 0.0f) : make_float2(w0 * inv, w1 * inv);
                if (!whole) {
                    parts.ml[slot * R + thr] = make_float2(m, s);
                } else if (a.lse) {
                    const int tok = thr / g;
                    a.lse[(int64_t)(f.s.row0 + tok) * a.H + f.h * g + thr - tok * g] = s == 0.0f ? -INFINITY : (m + log2f(s)) * kLn2;
                }
            }
            group_sync(t);
            float o0[R], o1[R];
            if (nb > 0) load_terms<R>(to, o0);
            if (both) load_terms<R>(to + 128, o1);
            uint16_t* const out = reinterpret_cast<uint16_t*>(a.out.p) + (int64_t)f.s.row0 * a.out.ts + (int64_t)f.h * g * a.out.hs + thr;
            float* const po = reinterpret_cast<float*>(parts.o) + slot * R * kDim + thr;
            int tok = 0, hd = 0;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (r < f.rows && thr < kDim) {
                    const float2 w = sm.join[r];
                    float v = nb > 0 ? o0[r] * w.x : 0.0f;
                    if (both) v = fmaf(o1[r], w.y, v);
                    if (w.x < 0.0f) v = 0.0f;
                    if (!whole) po[r * kDim] = v;
                    else out[tok * a.out.ts + hd * a.out.hs] = (uint16_t)(pack16(v, 0.0f, kBf) & 0xFFFF);
                    if (++hd == g) hd = 0, ++tok;
                }
            }
            if (!whole && f.first && thr == 0) parts.cut[blockIdx.x] = kv_cut<kSnap>(f, blockIdx.x, per, g, R);
            if (both) {
                tc_fence_before();
                __syncwarp();
                mbar_arrive_w(&sm.pair_empty);
            }
            group_sync(t);  // the weights have been read
        }
        if (both) ++pairs;
        tc_fence_before();
        __syncwarp();
        mbar_arrive_w(&sm.frag_empty[n & 1]);
    }
}

template <int kDim, int R, bool kBf>
__global__ void __launch_bounds__(kThreads, 1)
    k_kv_codes(const __grid_constant__ KvAttn a, const __grid_constant__ KvMaps maps, const __grid_constant__ KvPlan plan,
               const __grid_constant__ KvParts parts) {
    extern __shared__ uint8_t smem_raw[];
    using S = Smem<kDim, R>;
    S& sm = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    static_assert(sizeof(KvPlanSmem) <= sizeof(sm.kv), "the plan's arrays lie in the ring");
    static_assert(kRing > S::kPlaces / 2 + 4, "a block's mask is kept until its scores are read");
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i < S::kPlaces; ++i) {
            mbar_init(&sm.full[i], 1);
            mbar_init(&sm.empty[i], 1);
        }
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.q_empty, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sm.s_full[t], 1);
            mbar_init(&sm.p_full[t], 4);
            mbar_init(&sm.o_done[t], 1);
            mbar_init(&sm.frag_full[t], 1);
            mbar_init(&sm.frag_empty[t], 9);
        }
        mbar_init(&sm.pair_full, 4);
        mbar_init(&sm.pair_empty, 4);
        mbar_init(&sm.tail, 1);
        mbar_init(&sm.drained, 1);
        sm.abort = 0;
        sm.unfinite = 0;
        fence_mbar_init();
    }
    if (warp == kWarpMma) tmem_alloc(&sm.tmem_base, kTmemCols);
    cudaTriggerProgrammaticLaunchCompletion();
    cudaGridDependencySynchronize();
    if (tid == 0) parts.cut[blockIdx.x].last = -1;
    int64_t per;
    const Cursor<R> cur = kv_plan<R, kBlk, kOver, kSnap>(a, plan, *reinterpret_cast<KvPlanSmem*>(sm.kv), &per);
    if (tid == 0) sm.cur = cur;
    fence_proxy_async_smem();  // the plan's arrays were written by ordinary stores
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = __shfl_sync(0xffffffffu, sm.tmem_base, 0);
    // the softmax warps take the registers that the others give up
    static_assert(256 * kRegsSoftmax<R> + 128 * kRegsOther<R> <= kThreads * kRegsLaunch,
                  "more registers than the block was launched with");
    if (warp < 8) {
        if constexpr (R == 32) regs_up<kRegsSoftmax<R>>();
        role_softmax<kDim, R, kBf>(sm, a, parts, per, plan.g, tb);
    } else {
        if constexpr (R == 32) regs_down<kRegsOther<R>>();
        if (warp == kWarpMma) role_mma<kDim, R>(sm, tb);
        else if (warp == kWarpK) role_tma<kDim, R, false>(sm, a, maps, plan.g, cur);
        else if (warp == kWarpV) role_tma<kDim, R, true>(sm, a, maps, plan.g, cur);
        else role_q<kDim, R, kBf>(sm, a, plan.g, cur);
    }
    __syncwarp();
    __syncthreads();
    if (sm.abort && tid == 0) atomicOr(a.c.status, CSA2_DEVERR_TIMEOUT);
    if (warp == kWarpMma) {  // every MMA has completed before TMEM is freed
        tc_commit_w(&sm.drained);
        (void)mbar_wait_warp(&sm.drained, 0);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tb, kTmemCols);
    }
    if (sm.unfinite && warp < 8) give_back<kBf ? kE4m3Bf16 : kE4m3F16, kDim, R, kBlk, false>(a, parts, plan.g, sm.cur, 256);
}

template <int kDim, int R, bool kBf>
cudaError_t codes_as(const KvAttn& a, cudaStream_t st) {
    constexpr int kSmem = sizeof(Smem<kDim, R>) + 1024;
    static_assert(kSmem <= 232448, "shared memory beyond the 227 KB per-block limit");
    KvMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    const int64_t rows = (int64_t)a.c.num_pages * a.c.kv_heads * PAGE;
    constexpr CUtensorMapSwizzle kSwizzle = kDim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
    if (!make_pool_map(&maps.k, a.c.k, rows, kDim, kE4m3Bf16, kDim, kSwizzle) ||
        !make_pool_map(&maps.v, a.c.v, rows, kDim, kE4m3Bf16, kDim, kSwizzle))
        return cudaErrorInvalidValue;
    KvPlan plan;
    plan.g = a.H / a.c.kv_heads;
    plan.grid = device_sm_count();
    plan.min_per = kMinPer;
    const KvParts parts = kv_parts(a.ws, plan.grid, R, kDim);
    static std::atomic<uint64_t> attr_done{0};
    cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(k_kv_codes<kDim, R, kBf>), kSmem, attr_done);
    if (e != cudaSuccess) return e;
    e = launch_behind(k_kv_codes<kDim, R, kBf>, dim3(plan.grid), kThreads, kSmem, st, a, maps, plan, parts);
    if (e != cudaSuccess) return e;
    return launch_behind(k_kv_join<kDim, kBf, false>, dim3(kJoinBlocksPerSm * device_sm_count()), kJoinThreads, 0, st, a, parts,
                         plan.g, R, plan.grid);
}

template <int kDim, int R>
cudaError_t codes_type(const KvAttn& a, int dtype, cudaStream_t st) {
    return dtype == CSA2_DTYPE_BF16 ? codes_as<kDim, R, true>(a, st) : codes_as<kDim, R, false>(a, st);
}

}  // namespace

size_t kv_codes_workspace_bytes(bool few, int head_dim) { return kv_parts_bytes(device_sm_count(), few ? 16 : 32, head_dim); }

cudaError_t launch_kv_codes(const KvAttn& a, bool few, int head_dim, int dtype, cudaStream_t st) {
    if (head_dim == 64) return few ? codes_type<64, 16>(a, dtype, st) : codes_type<64, 32>(a, dtype, st);
    return few ? codes_type<128, 16>(a, dtype, st) : codes_type<128, 32>(a, dtype, st);
}

}  // namespace csa2
