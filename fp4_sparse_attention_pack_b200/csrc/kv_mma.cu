// Attention of a chunk of new tokens over the pages on the 5th-generation tensor
// cores (tcgen05.mma kind::f16, fp32 accumulation in TMEM).
//
// An item is 256 query rows (token, head of the group) of one sequence and kv
// head: two tiles of 128 rows that share every block of 128 keys.  Per block
//
//   S = Q K^T   (M = 128 rows, N = 128 keys, K = head_dim; both from shared memory)
//   P = 2^(c S - m)   (c = scale log2 e; 16 bits, written over S in TMEM)
//   O += P V    (M = 128, N = head_dim, K = 128 keys; P from TMEM, V from shared memory)
//
// with an online softmax: m is a maximum of an earlier block that moves only when
// a block exceeds it by more than 8 (then 2^8 fits every type's range), so the
// rescale of O is rare and the softmax warps do it themselves.  The tensor core
// works on one tile while the softmax warps work on the other.
//
// One CTA per SM, 384 threads (512 for an E4M3 cache), the items' work split evenly
// (kv_plan.cuh):
//   warps 0-3, 4-7   softmax of tile 0 and 1: thread = row (TMEM lane); at the
//                    item's end the output, or the partial sums;
//   warp 8           issues the MMAs, a half of P's keys as they arrive;
//   warp 9           loads K and V blocks by TMA: two pages of 64 rows, 64
//                    channels a box, 128-byte swizzle (or raw codes);
//   the last ones    load the queries of the next item while this one ends and
//                    tell the others which item it is.  For an E4M3 cache they
//                    also widen K and V to fp16 (exact); queries are then
//                    brought to fp16 as well: a bf16 row is scaled by a power of
//                    two that takes its largest magnitude into [2^14, 2^15),
//                    undone in c.
// Rows of V that no row of the item sees (behind the last key, before the
// window, on a page that is not loaded) are zeroed in shared memory, because
// 0 x NaN would reach the sums; their scores are masked.  Of rows that only some
// rows see, what is not finite is taken out and given back at the end
// (kv_attn.cuh); the pass that looks for it costs 12 prompts of up to 512 through a
// window of 128 some 2 us of 31, other calls 1% or less.
//
// A chunk of 2,048 tokens over 16,384, 64 / 8 heads of 128, bf16: 1.06 to 1.08 ms
// by the machine (973 TFLOP/s, 57% of the burst rate, 69% of the sustained one).  A block takes 3,650
// cycles for both tiles, of which the tensor pipe works 2,000: the chain scores ->
// softmax (2,400) -> PV and the next scores (1,000) of a tile bounds it.  Chunks of up
// to 1,024 over an E4M3 cache of 8,192: 341 to 346 us (749 TFLOP/s); there the widening warps
// share the issue slots.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cstring>
#include <type_traits>

#include "kv_attn.cuh"
#include "kv_plan.cuh"
#include "sm100.cuh"

namespace csa2 {

namespace {

using namespace sm100;

constexpr int kTile = 256;  // rows of an item
constexpr int kBlk = 128;   // keys of a block
constexpr int kOver = 2;    // an item's start and end, in blocks
constexpr int kMinPer = 4;  // least cost of a CTA's range
constexpr int kSnap = 3;
constexpr int kWarpMma = 8, kWarpTma = 9;
// The last warps load the queries: two, or six that widen an E4M3 cache's blocks too.
constexpr int load_warps(int mode) { return is_e4m3(mode) ? 6 : 2; }
constexpr int kGroupWarps = 3;  // of a group that widens a block
constexpr int threads_of(int mode) { return is_e4m3(mode) ? 512 : 384; }
// Registers of a thread at launch, of a softmax thread and of the others.
constexpr int regs_launch(int mode) { return is_e4m3(mode) ? 128 : 168; }
constexpr int regs_softmax(int mode) { return is_e4m3(mode) ? 176 : 208; }
constexpr int regs_other(int mode) { return is_e4m3(mode) ? 80 : 88; }
constexpr int kMixEvery = 4;  // of so many pairs of exponentials one is a polynomial
constexpr int kExp = 113;     // row_exp's powers lie in [-113, 140]
constexpr int kRing = 16;     // blocks whose masks of bad pages are kept
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // two of each, 128 columns apart

// Laid at a multiple of 1,024 bytes.
template <int kDim, int kMode>
struct Smem {
    static constexpr int kSlabs = kDim / 64;
    static constexpr int kStages = kDim == 64 ? (is_e4m3(kMode) ? 6 : 8) : (is_e4m3(kMode) ? 3 : 5);
    static constexpr int kRaw = is_e4m3(kMode) ? (kDim == 64 ? 8 : 4) : 1;  // blocks of E4M3 codes in flight
    // K and V blocks as the MMAs read them: slabs of 64 channels [key][64], SW128; then
    // the queries of tile 1 and of tile 0 in the same form.  Where every item of a call
    // is one tile, the ring has the place of tile 1's queries too.
    alignas(16) uint8_t kv[kStages + 2][kSlabs][kBlk * 128];
    uint8_t raw[kRaw][is_e4m3(kMode) ? kBlk * kDim : 16];  // slabs of 64 channels [key][64]
    uint8_t qe[2][kMode == kE4m3Bf16 ? kTile : 8];  // power of two of each row, + kExp (per item parity)
    uint8_t bad[kRing];                         // bit p: page p of the block is outside the pool
    int unfinite;                               // values were taken out
    KvCursor<kTile, kBlk, kOver> cur;           // the CTA's, for them
    uint64_t full[kStages + 1], empty[kStages + 1];
    uint64_t raw_full[kRaw], raw_empty[kRaw];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2][2], o_done[2];  // p_full: [tile][half of the keys]
    uint64_t tail;                              // the TMA of a V block that needs zeroing landed
    uint64_t drained;
    uint64_t frag_full[2], frag_empty[2];
    uint64_t pair_full, pair_empty;             // the places' results of an item of one tile
    float2 pair[128];                           // tile 1's (maximum, sum) of an item of one tile
    KvFrag frag[2];                             // this item and the next (rows = 0: no more)
    uint32_t tmem_base;
    int abort;
};

__device__ __forceinline__ uint32_t sw128(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// Bounded wait that also gives up when another role has given up.
template <class S>
__device__ __forceinline__ bool wait_bar(S& sm, uint64_t* bar, uint32_t parity) {
    if (mbar_try(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    while (true) {
        if (*reinterpret_cast<volatile int*>(&sm.abort)) return false;
        if (mbar_try_sleep(bar, parity, 20000u)) return true;
        if (global_ns() - t0 > kWaitNs) {
            atomicExch(&sm.abort, 1);
            return false;
        }
    }
}
template <class S>
__device__ __forceinline__ bool wait_bar_warp(S& sm, uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_bar(sm, bar, parity));
}

using Cursor = KvCursor<kTile, kBlk, kOver>;

// Stage counter of a ring.
struct Ring {
    int n, i = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ explicit Ring(int n) : n(n) {}
    __device__ __forceinline__ void step() {
        if (++i == n) i = 0, phase ^= 1;
    }
};

template <class S>
__device__ __forceinline__ int stages_of(const KvAttn& a, int g) { return S::kStages + (a.max_new <= 128 / g ? 1 : 0); }

// An item of at most 128 rows is one tile: the two tiles' places in TMEM then take
// its blocks by turns, each with its own maximum and sums, joined at the item's
// end.  (With one place the tensor core and the softmax warps wait for each other:
// 8 tokens of 8 sequences over 32,768, 64 / 8 heads of 128, 216 us, now 194.)
__device__ __forceinline__ bool one_tile(const KvFrag& f) { return f.rows <= 128; }

// What the x-th place in the ring holds, of an item's 2 nb: K and V by turns, or
// for one tile K a block ahead (K0 K1 V0 K2 V1 ..), the order of their use.
struct Part {
    int j;
    bool is_v;
};
__device__ __forceinline__ Part part_of(int x, int nb, bool one) {
    if (!one) return {x >> 1, (x & 1) != 0};
    if (x == 0) return {0, false};
    if (x == 2 * nb - 1) return {nb - 1, true};
    return x & 1 ? Part{(x + 1) >> 1, false} : Part{(x >> 1) - 1, true};
}

// ---------------------------------------------------------------- MMA

template <int kDim, int kMode>
__device__ void role_mma(Smem<kDim, kMode>& sm, int stages, uint32_t tb) {
    using S = Smem<kDim, kMode>;
    constexpr uint32_t kFmt = kMode == kBf16 ? 1 : 0;
    const uint32_t idesc_s = idesc_f16(128, kBlk, kFmt, 0, 0);
    const uint32_t idesc_o = idesc_f16(128, kDim, kFmt, 0, 1);
    constexpr uint32_t kStageBytes = S::kSlabs * kBlk * 128;
    const uint64_t desc_q = smem_desc(sm.kv[S::kStages + 1][0], 16, 1024, kLayoutSw128);
    const uint64_t desc_k = smem_desc(sm.kv[0][0], 16, 1024, kLayoutSw128);
    const uint64_t desc_v = smem_desc(sm.kv[0][0], kBlk * 128, 1024, kLayoutSw128);
    Ring ring(stages);
    uint32_t items = 0, np[2] = {0, 0};  // items with keys; P hand-overs of each tile
    auto scores = [&](int t, int q, int stage) {  // S_t = Q_q K^T
#pragma unroll
        for (int ks = 0; ks < kDim / 16; ++ks) {
            const uint32_t off = ((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4;
            tc_mma_f16_w(tb + kColS + 128 * t, desc_q + off - ((q * kStageBytes) >> 4),
                         desc_k + off + ((stage * kStageBytes) >> 4), idesc_s, ks > 0);
        }
        tc_commit_w(&sm.s_full[t]);
    };
    auto values = [&](int t, int stage, bool first) {  // O_t += P_t V, as P arrives
        for (int half = 0; half < 2; ++half) {
            if (!wait_bar_warp(sm, &sm.p_full[t][half], np[t] & 1)) return false;
            tc_fence_after();
#pragma unroll
            for (int i2 = 0; i2 < kBlk / 32; ++i2) {
                const int i = i2 + half * (kBlk / 32);
                tc_mma_f16_ta_w(tb + kColO + 128 * t, tb + kColS + 128 * t + 8 * i,
                                desc_v + ((stage * kStageBytes + 2048 * i) >> 4), idesc_o, !first || i > 0);
            }
        }
        ++np[t];
        return true;
    };
    for (uint32_t n = 0;; ++n) {
        if (!wait_bar_warp(sm, &sm.frag_full[n & 1], (n >> 1) & 1)) return;
        const int nb = sm.frag[n & 1].f1 - sm.frag[n & 1].f0, rows = sm.frag[n & 1].rows;
        const bool one = one_tile(sm.frag[n & 1]);
        if (rows == 0) return;
        __syncwarp();
        mbar_arrive_w(&sm.frag_empty[n & 1]);
        if (nb == 0) continue;
        if (!wait_bar_warp(sm, &sm.q_full, items & 1)) return;
        ++items;
        // the first scores: of the first block for both tiles, or of the first two blocks
        for (int t = 0; t < 2; ++t) {
            if (one && t >= nb) break;
            if (t == 0 || one) {
                if (!wait_bar_warp(sm, &sm.full[ring.i], ring.phase)) return;
                tc_fence_after();
            }
            scores(t, one ? 0 : t, ring.i);
            if (t == 1 || one) {
                tc_commit_w(&sm.empty[ring.i]);
                ring.step();
            }
        }
        if (nb == 1 || (one && nb == 2)) tc_commit_w(&sm.q_empty);
        for (int j = 0; j < nb; ++j) {
            const int sv = ring.i;
            const uint32_t pv = ring.phase;
            ring.step();
            const int sk = ring.i;
            const uint32_t pk = ring.phase;
            const bool more = j + (one ? 2 : 1) < nb;
            if (!wait_bar_warp(sm, &sm.full[sv], pv)) return;
            for (int t = one ? j & 1 : 0; t < (one ? (j & 1) + 1 : 2); ++t) {
                if (!values(t, sv, j < (one ? 2 : 1))) return;
                if (one || t == 1) tc_commit_w(&sm.empty[sv]);
                if (!more) {
                    tc_commit_w(&sm.o_done[t]);
                    continue;
                }
                if (!wait_bar_warp(sm, &sm.full[sk], pk)) return;
                tc_fence_after();
                scores(t, one ? 0 : t, sk);  // in order behind the MMAs that read P, which S overwrites
            }
            if (more) {
                tc_commit_w(&sm.empty[sk]);
                if (j + (one ? 3 : 2) == nb) tc_commit_w(&sm.q_empty);
                ring.step();
            }
        }
    }
}

// ---------------------------------------------------------------- loads

// Pages of a block: ids (or -1: not needed or outside the pool) and bad bits.
struct PagePair {
    int p[2];
    int bad;
};
__device__ __forceinline__ PagePair pages_of(const KvAttn& a, const KvFrag& f, int j, int id0, int id1) {
    PagePair r;
    r.bad = 0;
    const int id[2] = {id0, id1};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int pg = 2 * j + i;
        const bool need = pg * PAGE <= f.v.hi && pg * PAGE + PAGE > f.v.lo;
        const bool good = id[i] >= 0 && id[i] < a.c.num_pages;
        r.p[i] = need && good ? id[i] : -1;
        if (need && !good) r.bad |= 1 << i;
    }
    return r;
}

// A row of V that no query row of the item sees, or that is not loaded.
__device__ __forceinline__ bool v_row_unseen(const KvFrag& f, int bad, int j, int r) {
    const int key = j * kBlk + r;
    return key < f.v.lo || key > f.v.hi || (bad >> (r >> 6) & 1);
}

template <int kDim, int kMode>
__device__ void role_tma(Smem<kDim, kMode>& sm, const KvAttn& a, const KvMaps& maps, int g, Cursor cur) {
    using S = Smem<kDim, kMode>;
    constexpr bool kRawCodes = is_e4m3(kMode);
    constexpr int kPageBytes = PAGE * kDim * (kRawCodes ? 1 : 2);
    const int places = kRawCodes ? S::kRaw : stages_of<S>(a, g);
    uint64_t* const fulls = kRawCodes ? sm.raw_full : sm.full;
    uint64_t* const empties = kRawCodes ? sm.raw_empty : sm.empty;
    const int lane = threadIdx.x & 31;
    Ring ring(places);
    uint32_t used = 0, tails = 0, blocks = 0;
    KvFrag f;
    // the whole warp issues each box (a lane for each box took 1,000 cycles a block, as
    // the lanes' copies are issued one after another with their operands moved first)
    auto load = [&](const PagePair& pp, bool is_v, int h, uint64_t* bar) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (pp.p[i] < 0) continue;
            const int y = (pp.p[i] * a.c.kv_heads + h) * PAGE;
#pragma unroll
            for (int c = 0; c < S::kSlabs; ++c)
                tma_load_2d_nohint_w(kRawCodes ? &sm.raw[ring.i][(c * kBlk + i * PAGE) * 64] : &sm.kv[ring.i][c][i * PAGE * 128],
                                     is_v ? &maps.v : &maps.k, 64 * c, y, bar);
        }
    };
    // block j's K or V to the next place of the ring
    auto put = [&](const PagePair& pp, int j, int place, bool is_v, const KvCommon& common) {
        if (used >= places && !wait_bar_warp(sm, &empties[ring.i], ring.phase ^ 1)) return false;
        ++used;
        uint64_t* full = &fulls[ring.i];
        const uint32_t bytes = ((pp.p[0] >= 0) + (pp.p[1] >= 0)) * kPageBytes;
        if (!is_v) {
            if (lane == 0) {
                sm.bad[place % kRing] = (uint8_t)pp.bad;
                if (pp.bad) atomicOr(a.c.status, CSA2_DEVERR_PAGE);
            }
            __syncwarp();
        }
        if (kRawCodes || !is_v || !(common.leaves(j * kBlk, kBlk) || pp.bad)) {
            mbar_expect_tx_w(full, bytes);
            load(pp, is_v, f.h, full);
        } else {
            if (bytes) {
                mbar_expect_tx_w(&sm.tail, bytes);
                load(pp, true, f.h, &sm.tail);
                // its own copy: waited for even when the others have given up
                if (!__all_sync(0xffffffffu, mbar_wait(&sm.tail, tails & 1))) {
                    atomicExch(&sm.abort, 1);
                    return false;
                }
                ++tails;
            }
            if (clear_rows<kMode, kBlk, 128, S::kSlabs>(sm.kv[ring.i][0], common, j * kBlk, [&](int r) { return v_row_unseen(f, pp.bad, j, r); }))
                sm.unfinite = 1;
            fence_proxy_async_smem();
            __syncwarp();
            mbar_arrive_w(full);
        }
        ring.step();
        return true;
    };
    bool alive = true;
    while (alive && cur.next(a, g, f)) {
        const int32_t* table = a.c.page_table + (int64_t)f.b * a.c.max_pages;
        const int nb = f.f1 - f.f0, ahead = one_tile(f) ? 1 : 0;
        const KvCommon common(f, a.window);
        int ids = -1, have = -1;  // 32 page ids at a time, one to a lane
        PagePair pp = {{-1, -1}, 0};
        for (int x = -ahead; x < nb && alive; ++x) {  // K of block x + ahead, then V of block x
            const PagePair before = pp;
            if (x + ahead < nb) {
                const int j = f.f0 + x + ahead;
                if (have != 2 * j / 32) {
                    have = 2 * j / 32;
                    const int pg = 32 * have + lane;
                    ids = pg >= f.v.lo / PAGE && pg <= f.v.hi / PAGE ? table[pg] : -1;
                }
                pp = pages_of(a, f, j, __shfl_sync(0xffffffffu, ids, 2 * j & 31), __shfl_sync(0xffffffffu, ids, (2 * j + 1) & 31));
                alive = put(pp, j, blocks + x + ahead, false, common);
            }
            if (x >= 0 && alive) alive = put(ahead ? before : pp, f.f0 + x, 0, true, common);
        }
        blocks += nb;
    }
    // no copy is in flight when the CTA ends, also after a wait that gave up
    if (*reinterpret_cast<volatile int*>(&sm.abort)) {
        for (uint32_t k = 0; k < min(used, (uint32_t)places); ++k) {
            const int st = (ring.i + places - 1 - (int)k) % places;
            (void)mbar_wait(&fulls[st], st < ring.i ? ring.phase : ring.phase ^ 1);
        }
    }
}

// 16 codes to 32 bytes of fp16.
__device__ __forceinline__ void widen16(const uint4& v, uint4& lo, uint4& hi) {
    e4m3x4_to_h2(v.x, lo.x, lo.y);
    e4m3x4_to_h2(v.y, lo.z, lo.w);
    e4m3x4_to_h2(v.z, hi.x, hi.y);
    e4m3x4_to_h2(v.w, hi.z, hi.w);
}

// A block of codes, slabs of 64 channels [key][64], to fp16 as the MMAs read it: a warp
// takes 8 rows of a slab at a time, 512 bytes to 1,024, four lanes to a row (the two
// rows of a quarter warp write all eight chunks of a line).
template <int kDim, int kUnroll, class Clear>
__device__ __forceinline__ void widen(const uint8_t* raw, uint8_t* kv, int thread, const Clear& clear) {
    constexpr int kAll = kBlk * kDim / 512;
    const int lane = thread & 31, r8 = lane >> 2;
    const uint8_t* src = raw + 16 * lane;
    uint8_t* lo_at = kv + sw128(r8, 2 * (lane & 3));
    uint8_t* hi_at = kv + sw128(r8, 2 * (lane & 3) + 1);
#pragma unroll kUnroll
    for (int u = thread >> 5; u < kAll; u += kGroupWarps) {
        uint4 v = *reinterpret_cast<const uint4*>(src + 512 * u), lo, hi;
        clear((8 * u + r8) % kBlk, v);
        widen16(v, lo, hi);
        *reinterpret_cast<uint4*>(lo_at + 1024 * u) = lo;
        *reinterpret_cast<uint4*>(hi_at + 1024 * u) = hi;
    }
}

// Queries and, for E4M3, the widening of K and V.
template <int kDim, int kMode>
__device__ void role_load(Smem<kDim, kMode>& sm, const KvAttn& a, int g, Cursor cur) {
    using S = Smem<kDim, kMode>;
    constexpr int kLoaders = 32 * load_warps(kMode);
    const int tid = threadIdx.x - (threads_of(kMode) - kLoaders);
    uint32_t used = 0, items = 0, blocks = 0;
    const uint32_t inv_g = 65536u / g + 1;  // x / g = x * inv_g >> 16 for x < 256 + g
    KvFrag f;
    for (uint32_t n = 0;; ++n) {
        const bool more = cur.next(a, g, f);
        if (tid < 32) {  // the first loader warp tells the others which item is next
            if (n > 1 && !wait_bar_warp(sm, &sm.frag_empty[n & 1], ((n >> 1) - 1) & 1)) return;
            if (tid == 0) {
                if (!more) f.rows = 0;
                sm.frag[n & 1] = f;
                mbar_arrive(&sm.frag_full[n & 1]);
            }
            __syncwarp();
        }
        if (!more) return;
        if (f.f1 == f.f0) continue;
        // ---- queries
        if (items > 0 && !wait_bar_warp(sm, &sm.q_empty, (items - 1) & 1)) return;
        constexpr int kChunks = kDim / 8;  // of 16 bytes a row
        const int rem0 = f.tile * kTile - f.v.t0 * g;
        const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q.p) + (int64_t)(f.s.row0 + f.v.t0) * a.q.ts +
                            (int64_t)f.h * g * a.q.hs;
        const int rows = f.rows > 128 ? 256 : 128;
        for (int r = tid >> 1; r < rows; r += kLoaders / 2) {  // a pair of lanes to a row
            const int x = rem0 + r, t = (x * inv_g) >> 16;
            const uint16_t* src = q + (int64_t)t * a.q.ts + (int64_t)(x - t * g) * a.q.hs + 8 * (tid & 1);
#pragma unroll
            for (int c = 0; c < kChunks; c += 2) {
                uint8_t* d = &sm.kv[S::kStages + 1 - (r >> 7)][c >> 3][sw128(r & 127, (c & 7) + (tid & 1))];
                if (r < f.rows) cp_async16(d, src + 8 * c);
                else *reinterpret_cast<uint4*>(d) = make_uint4(0, 0, 0, 0);
            }
        }
        cp_async_commit();
        cp_async_wait_all();
        if constexpr (kMode == kE4m3Bf16) {
            for (int r = tid >> 1; r < rows; r += kLoaders / 2) {
                auto at = [&](int c) { return reinterpret_cast<uint4*>(&sm.kv[S::kStages + 1 - (r >> 7)][c >> 3][sw128(r & 127, (c & 7) + (tid & 1))]); };
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < kChunks; c += 2) top = max(top, top_bits(*at(c)));
                top = max(top, __shfl_xor_sync(3u << (tid & 30), top, 1));
                const int e = row_exp(top);
#pragma unroll
                for (int c = 0; c < kChunks; c += 2) *at(c) = scaled(*at(c), e);
                if ((tid & 1) == 0) sm.qe[items & 1][r] = (uint8_t)(e + kExp);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_w(&sm.q_full);
        ++items;
        if constexpr (is_e4m3(kMode)) {
            // ---- K and V: two groups of warps take the blocks by turns, so that one waits
            // while the other works
            const uint32_t stages = stages_of<S>(a, g);
            const int nb = f.f1 - f.f0, group = tid / (32 * kGroupWarps), gt = tid % (32 * kGroupWarps);
            const bool one = one_tile(f);
            const KvCommon common(f, a.window);
            constexpr int kGroups = kLoaders / (32 * kGroupWarps);
            // a place's parity says which turn of the ring it is only within one turn
            static_assert(kGroups <= S::kStages && kGroups <= S::kRaw, "more groups than places");
            for (int x = (group + kGroups - used % kGroups) % kGroups; x < 2 * nb; x += kGroups) {  // places group, group + kGroups, ..
                const Part part = part_of(x, nb, one);
                const int j = f.f0 + part.j;
                const uint32_t place = used + x;
                const int ri = place % stages, rw = place % S::kRaw;
                if (place >= stages && !wait_bar_warp(sm, &sm.empty[ri], (place / stages - 1) & 1)) return;
                if (!wait_bar_warp(sm, &sm.raw_full[rw], (place / S::kRaw) & 1)) return;
                const int bad = sm.bad[(blocks + part.j) % kRing];
                // Two tiles' softmax warps need the issue slots, so few loads are in flight
                // then; for one tile widening is what bounds the kernel.
                const auto nothing = [](int, uint4&) {};
                if (part.is_v && (common.leaves(j * kBlk, kBlk) || bad)) {
                    Unfinite<kMode> found;
                    widen<kDim, 2>(sm.raw[rw], sm.kv[ri][0], gt, [&](int r, uint4& v) {
                        if (v_row_unseen(f, bad, j, r)) v = make_uint4(0, 0, 0, 0);
                        if (!common.has(j * kBlk + r)) found.see(v);
                    });
                    if (__any_sync(0xffffffffu, found.any())) {  // once more, without them
                        widen<kDim, 1>(sm.raw[rw], sm.kv[ri][0], gt, [&](int r, uint4& v) {
                            if (v_row_unseen(f, bad, j, r)) v = make_uint4(0, 0, 0, 0);
                            if (!common.has(j * kBlk + r)) drop_unfinite<kMode>(v);
                        });
                        sm.unfinite = 1;
                    }
                } else if (one) widen<kDim, 4>(sm.raw[rw], sm.kv[ri][0], gt, nothing);
                else widen<kDim, 2>(sm.raw[rw], sm.kv[ri][0], gt, nothing);
                fence_proxy_async_smem();
                __syncwarp();
                mbar_arrive_w(&sm.full[ri]);
                mbar_arrive_w(&sm.raw_empty[rw]);
            }
            used += 2 * nb;
            blocks += nb;
        }
    }
}

// ---------------------------------------------------------------- softmax

// 2^t of two values in fp32 arithmetic, for t in [-126, 127.5) (its callers' are at most
// kGap + 7 = 15): t = n + f with |f| <= 1/2, a polynomial for 2^f (the minimax one of
// degree 4, computed for this file by Remez exchange: relative error 2.6e-6, far below
// the rounding to 16 bits) times 2^n.  Below -126 the value is that of -126; NaN stays
// NaN.
__device__ __forceinline__ float2 ex2_poly(float2 t) {
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(t.x) : "f"(-126.0f));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(t.y) : "f"(-126.0f));
    constexpr float kRound = 12582912.0f;  // 1.5 x 2^23: the sum's low bits are n
    const float2 r = add2(t, splat2(kRound));
    const float2 f = sub2(t, sub2(r, splat2(kRound)));
    float2 p = fma2(splat2(9.570101912e-3f), f, splat2(5.591786032e-2f));
    p = fma2(p, f, splat2(0.2402474483f));
    p = fma2(p, f, splat2(0.6931218147f));
    p = fma2(p, f, splat2(0.9999992614f));
    return mul2(p, make_float2(__uint_as_float((__float_as_uint(r.x) << 23) + 0x3F800000u),
                               __uint_as_float((__float_as_uint(r.y) << 23) + 0x3F800000u)));
}

// P of 32 keys, 2^(c s - m), in 16 bits, and its sums.  kMix: some pairs by
// polynomial, as the special-function units (16 values a clock) would bound the
// kernel otherwise; without it masked scores give exact zeros.
template <bool kMix, bool kBf>
__device__ __forceinline__ void exps(const uint32_t (&s)[32], float2 c, float2 m, float2 (&sum)[2], uint32_t (&p)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float2 e = fma2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c, m);
        if (kMix && i % kMixEvery == kMixEvery - 1) e = ex2_poly(e);
        else e = make_float2(ex2(e.x), ex2(e.y));
        sum[i & 1] = add2(sum[i & 1], e);
        p[i] = pack16(e.x, e.y, kBf);
    }
}
__device__ __forceinline__ float max32(const uint32_t (&x)[32]) {
    float m[2] = {__uint_as_float(x[0]), __uint_as_float(x[1])};
#pragma unroll
    for (int i = 2; i < 30; i += 4) {
#pragma unroll
        for (int k = 0; k < 2; ++k) m[k] = fmaxf(fmaxf(m[k], __uint_as_float(x[i + 2 * k])), __uint_as_float(x[i + 2 * k + 1]));
    }
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(__uint_as_float(x[30]), __uint_as_float(x[31])));
}

template <int kDim, int kMode>
__device__ void role_softmax(Smem<kDim, kMode>& sm, const KvAttn& a, const KvParts& parts, int64_t per, int g, uint32_t tb) {
    const int t = threadIdx.x >> 7, row = threadIdx.x & 127, lane = threadIdx.x & 31;  // tile; row = TMEM lane
    const uint32_t lane_base = tb + ((uint32_t)(32 * ((threadIdx.x >> 5) & 3)) << 16);
    const uint32_t ts = lane_base + kColS + 128 * t, to = lane_base + kColO + 128 * t;
    constexpr bool kP16Bf = kMode == kBf16;  // P in V's type
    constexpr bool kOutBf = kMode == kBf16 || kMode == kE4m3Bf16;
    uint32_t ns = 0, no = 0, items = 0, blocks = 0, pairs = 0;
    for (uint32_t n = 0;; ++n) {
        if (!wait_bar_warp(sm, &sm.frag_full[n & 1], (n >> 1) & 1)) return;
        const KvFrag& f = sm.frag[n & 1];
        if (f.rows == 0) return;
        const int nb = f.f1 - f.f0;
        const int it = items;
        if (nb > 0) ++items;
        const int blk0 = blocks;
        blocks += nb;
        const bool one = one_tile(f);
        if (!one || t == 0 || nb > 1) {
            const int ri = one ? row : 128 * t + row;  // row of the item
            const bool idle = ri - lane >= f.rows;     // a warp without rows: what it leaves in P reaches no row that counts
            int pos, lo;  // the row sees keys lo .. pos
            {
                const int x = f.tile * kTile - f.v.t0 * g + min(ri, f.rows - 1);
                pos = f.s.n - f.s.m + f.v.t0 + x / g;
                lo = first_key(pos, a.window);
            }
            float mref = -INFINITY, l = 0.0f;
            float c = fmaxf(a.scale * kLog2e, FLT_MIN);  // never 0: a masked score is -infinity
            const int j0 = f.f0, j1 = f.f1, first = one ? j0 + t : j0;
            for (int j = first; j < j1; j += one ? 2 : 1) {
                if (!wait_bar_warp(sm, &sm.s_full[t], ns & 1)) return;
                ++ns;
                __syncwarp();
                tc_fence_after();
                if (idle) {
                    mbar_arrive_w(&sm.p_full[t][0]);
                    mbar_arrive_w(&sm.p_full[t][1]);
                    continue;
                }
                if constexpr (kMode == kE4m3Bf16) {
                    if (j == first) c = times_pow2(c, kExp - sm.qe[it & 1][ri]);
                }
                uint32_t r[4][32];
#pragma unroll
                for (int k = 0; k < 4; ++k) tmem_ld_x32_nowait(ts + 32 * k, r[k]);
                const int bad = sm.bad[(blk0 + j - j0) % kRing], k0 = j * kBlk;
                const bool part = __any_sync(0xffffffffu, pos - k0 < kBlk - 1 || lo - k0 > 0) || bad;
                auto masked = [&](int k, uint32_t(&x)[32]) {
                    const int c_hi = bad >> (k >> 1) & 1 ? -1 : pos - k0 - 32 * k, c_lo = lo - k0 - 32 * k;
                    if (!__any_sync(0xffffffffu, c_hi < 31 || c_lo > 0)) return;
                    const uint32_t below = c_hi >= 31 ? ~0u : c_hi < 0 ? 0u : (2u << c_hi) - 1;  // keys up to c_hi
                    const uint32_t seen = c_lo <= 0 ? below : c_lo > 31 ? 0u : below & (~0u << c_lo);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!(seen >> i & 1)) x[i] = 0xFF800000u;  // -infinity
                    tmem_st_x32_nowait(ts + 32 * k, x);  // they are read again
                };
                tmem_wait_ld2(r[0], r[1]);
                tmem_wait_ld2(r[2], r[3]);
                if (part) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) masked(k, r[k]);
                    tmem_wait_st();
                }
                const float bm = fmaxf(fmaxf(max32(r[0]), max32(r[1])), fmaxf(max32(r[2]), max32(r[3]))) * c - below(kMode);
                const bool move = bm > mref + kGap || (mref == -INFINITY && bm > -INFINITY);
                if (__any_sync(0xffffffffu, move)) {
                    const float f1 = move ? ex2(mref - bm) : 1.0f;  // mref = -inf: 0
                    if (move) mref = bm;
                    l *= f1;
                    if (j > first) {  // O holds the blocks before
#pragma unroll 1
                        for (int k = 0; k < kDim; k += 16) {
                            float o[16];
                            tmem_ld_32x32b_x16(to + k, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] *= f1;
                            tmem_st_32x32b_x16(to + k, o);
                        }
                    }
                }
                const float2 c2 = splat2(c), m2 = splat2(mref == -INFINITY ? 0.0f : -mref);
                float2 sum[2] = {make_float2(l, 0.f), splat2(0.f)};
                // 64 keys at a time, their scores read again: a short loop and few registers
                // (one pass over 128 scores in registers took 4% longer, one over 32 10%)
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[16];
                    tmem_ld_x32_nowait(ts + 64 * h, r[0]);
                    tmem_ld_x32_nowait(ts + 64 * h + 32, r[1]);
                    tmem_wait_ld2(r[0], r[1]);
                    if (part) {
                        exps<false, kP16Bf>(r[0], c2, m2, sum, p);
                        tmem_st_x16_nowait(ts + 32 * h, p);
                        exps<false, kP16Bf>(r[1], c2, m2, sum, p);
                    } else {
                        exps<true, kP16Bf>(r[0], c2, m2, sum, p);
                        tmem_st_x16_nowait(ts + 32 * h, p);
                        exps<true, kP16Bf>(r[1], c2, m2, sum, p);
                    }
                    tmem_st_x16_nowait(ts + 32 * h + 16, p);
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    mbar_arrive_w(&sm.p_full[t][h]);  // the product with these keys' values begins
                }
                l = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            }
            // ---- the item's end
            if (nb > 0) {
                if (!wait_bar_warp(sm, &sm.o_done[t], no & 1)) return;
                ++no;
                __syncwarp();
                tc_fence_after();
            }
            const bool both = one && nb > 1;  // tile 0 joins the two places' results
            float w0 = 1.0f, w1 = 0.0f;
            if (both && t == 1) {
                sm.pair[row] = make_float2(mref, l);
                tc_fence_before();
                __syncwarp();
                mbar_arrive_w(&sm.pair_full);
                if (!wait_bar_warp(sm, &sm.pair_empty, pairs & 1)) return;
            } else {
                if (both) {
                    if (!wait_bar_warp(sm, &sm.pair_full, pairs & 1)) return;
                    __syncwarp();
                    tc_fence_after();
                    const float2 o = sm.pair[row];
                    const float m = fmaxf(mref, o.x), ms = m == -INFINITY ? 0.0f : m;
                    w0 = ex2(mref - ms), w1 = ex2(o.x - ms);  // a maximum of -infinity: 0
                    l = l * w0 + o.y * w1;
                    mref = m;
                }
                const bool mine = ri < f.rows;
                const bool whole = f.first && f.last;
                const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                const float k0 = whole ? w0 * inv : w0, k1 = whole ? w1 * inv : w1;
                const int64_t slot = 2 * (int64_t)blockIdx.x + (f.first ? 1 : 0);
                float4* po = parts.o + slot * (kDim / 4) * kTile + ri;
                const int x = f.tile * kTile - f.v.t0 * g + min(ri, f.rows - 1);
                const int64_t token = f.s.row0 + f.v.t0 + x / g;
                const int head = f.h * g + x % g;
                uint16_t* out = reinterpret_cast<uint16_t*>(a.out.p) + token * a.out.ts + (int64_t)head * a.out.hs;
                uint16_t* to_row[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    to_row[i] = reinterpret_cast<uint16_t*>(__shfl_sync(
                        0xffffffffu, reinterpret_cast<unsigned long long>(mine ? out : nullptr), (lane & 28) + i));
#pragma unroll 1
                for (int k = 0; k < kDim; k += 32) {
                    float o[32];
                    if (nb > 0) tmem_ld_32x32b_x32(to + k, o);
                    if (both) {
                        float o1[32];
                        tmem_ld_32x32b_x32(to + 128 + k, o1);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = o[i] * k0 + o1[i] * k1;
                    } else if (whole) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= k0;
                    }
                    if (!whole) {
                        if (idle) break;
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            po[(int64_t)((k + i) / 4) * kTile] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    } else {
                        // four lanes exchange their 16-byte chunks, so that a store takes 64
                        // bytes of each of eight rows, not 16 of 32
                        uint32_t w[4][4];
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i >> 2][i & 3] = l == 0.0f ? 0u : pack16(o[2 * i], o[2 * i + 1], kOutBf);
#pragma unroll
                        for (int d = 1; d < 4; d *= 2)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (i & d) continue;
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const uint32_t give = lane & d ? w[i][e] : w[i | d][e];
                                    const uint32_t got = __shfl_xor_sync(0xffffffffu, give, d);
                                    if (lane & d) w[i][e] = got;
                                    else w[i | d][e] = got;
                                }
                            }
#pragma unroll
                        for (int i = 0; i < 4; ++i)  // chunk lane % 4 of the i-th of the four rows
                            if (to_row[i]) *reinterpret_cast<uint4*>(to_row[i] + k + 8 * (lane & 3)) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
                    }
                }
                if (!whole) {
                    parts.ml[slot * kTile + ri] = make_float2(mref, l);
                    if (f.first && threadIdx.x == 0)
                        parts.cut[blockIdx.x] = kv_cut<kSnap>(f, blockIdx.x, per, g, kTile);
                } else if (mine && a.lse) {
                    a.lse[token * a.H + head] = l == 0.0f ? -INFINITY : (mref + log2f(l)) * kLn2;
                }
                if (both) {
                    tc_fence_before();
                    __syncwarp();
                    mbar_arrive_w(&sm.pair_empty);
                }
            }
            if (both) ++pairs;
            tc_fence_before();
        }
        __syncwarp();
        mbar_arrive_w(&sm.frag_empty[n & 1]);
    }
}

template <int kDim, int kMode>
__global__ void __launch_bounds__(threads_of(kMode), 1)
    k_kv_mma(const __grid_constant__ KvAttn a, const __grid_constant__ KvMaps maps, const __grid_constant__ KvPlan plan,
             const __grid_constant__ KvParts parts) {
    extern __shared__ uint8_t smem_raw[];
    using S = Smem<kDim, kMode>;
    S& sm = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    static_assert(sizeof(KvPlanSmem) <= sizeof(sm.kv), "the plan's arrays lie in the ring");
    const int tid = threadIdx.x, warp = tid >> 5;
    if (tid == 0) {
        for (int i = 0; i <= S::kStages; ++i) {
            mbar_init(&sm.full[i], is_e4m3(kMode) ? kGroupWarps : 1);
            mbar_init(&sm.empty[i], 1);
        }
        mbar_init(&sm.q_full, load_warps(kMode));
        mbar_init(&sm.q_empty, 1);
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sm.s_full[t], 1);
            mbar_init(&sm.p_full[t][0], 4);
            mbar_init(&sm.p_full[t][1], 4);
            mbar_init(&sm.frag_full[t], 1);
            mbar_init(&sm.frag_empty[t], 9);
            mbar_init(&sm.o_done[t], 1);
        }
        for (int i = 0; i < S::kRaw; ++i) {
            mbar_init(&sm.raw_full[i], 1);
            mbar_init(&sm.raw_empty[i], kGroupWarps);
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
    Cursor cur = kv_plan<kTile, kBlk, kOver, kSnap>(a, plan, *reinterpret_cast<KvPlanSmem*>(sm.kv), &per);
    if (tid == 0) sm.cur = cur;
    fence_proxy_async_smem();  // the plan's arrays were written by ordinary stores
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tb = __shfl_sync(0xffffffffu, sm.tmem_base, 0);
    // the softmax warps take the registers that the others give up
    static_assert(threads_of(kMode) * regs_launch(kMode) <= 65536 &&
                      256 * regs_softmax(kMode) + (threads_of(kMode) - 256) * regs_other(kMode) <=
                          threads_of(kMode) * regs_launch(kMode),
                  "more registers than the block was launched with");
    if (warp < 8) {
        regs_up<regs_softmax(kMode)>();
        role_softmax<kDim, kMode>(sm, a, parts, per, plan.g, tb);
    } else {
        regs_down<regs_other(kMode)>();
        if (warp == kWarpMma) role_mma<kDim, kMode>(sm, stages_of<S>(a, plan.g), tb);
        else if (warp == kWarpTma) role_tma<kDim, kMode>(sm, a, maps, plan.g, cur);
        else role_load<kDim, kMode>(sm, a, plan.g, cur);
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
    if (sm.unfinite && warp < 8) give_back<kMode, kDim, kTile, kBlk, true>(a, parts, plan.g, sm.cur, 256);
}

template <int kDim, int kMode>
cudaError_t mma_as(const KvAttn& a, cudaStream_t st) {
    using S = Smem<kDim, kMode>;
    constexpr int kSmem = sizeof(S) + 1024;
    static_assert(kSmem <= 232448, "shared memory beyond the 227 KB per-block limit");
    KvMaps maps;
    std::memset(&maps, 0, sizeof(maps));
    const int64_t rows = (int64_t)a.c.num_pages * a.c.kv_heads * PAGE;
    constexpr int kWidth = is_e4m3(kMode) ? 64 : 128;  // bytes of 64 channels
    constexpr CUtensorMapSwizzle kSwizzle = is_e4m3(kMode) ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
    if (!make_pool_map(&maps.k, a.c.k, rows, kDim, kMode, kWidth, kSwizzle) ||
        !make_pool_map(&maps.v, a.c.v, rows, kDim, kMode, kWidth, kSwizzle))
        return cudaErrorInvalidValue;
    KvPlan plan;
    plan.g = a.H / a.c.kv_heads;
    plan.grid = device_sm_count();
    plan.min_per = kMinPer;
    const KvParts parts = kv_parts(a.ws, plan.grid, kTile, kDim);
    static std::atomic<uint64_t> attr_done{0};
    cudaError_t e = smem_opt_in(reinterpret_cast<const void*>(k_kv_mma<kDim, kMode>), kSmem, attr_done);
    if (e != cudaSuccess) return e;
    e = launch_behind(k_kv_mma<kDim, kMode>, dim3(plan.grid), threads_of(kMode), kSmem, st, a, maps, plan, parts);
    if (e != cudaSuccess) return e;
    constexpr bool kBf = kMode == kBf16 || kMode == kE4m3Bf16;
    return launch_behind(k_kv_join<kDim, kBf, true>, dim3(kJoinBlocksPerSm * device_sm_count()), kJoinThreads, 0, st, a, parts, plan.g, kTile, plan.grid);
}

}  // namespace

size_t kv_mma_workspace_bytes(int head_dim) { return kv_parts_bytes(device_sm_count(), kTile, head_dim); }

cudaError_t launch_kv_mma(const KvAttn& a, int head_dim, int dtype, int kv_dtype, cudaStream_t st) {
    const bool e4m3 = kv_dtype == CSA2_KV_E4M3, bf = dtype == CSA2_DTYPE_BF16;
    if (head_dim == 64)
        return e4m3 ? (bf ? mma_as<64, kE4m3Bf16>(a, st) : mma_as<64, kE4m3F16>(a, st))
                    : (bf ? mma_as<64, kBf16>(a, st) : mma_as<64, kF16>(a, st));
    return e4m3 ? (bf ? mma_as<128, kE4m3Bf16>(a, st) : mma_as<128, kE4m3F16>(a, st))
                : (bf ? mma_as<128, kBf16>(a, st) : mma_as<128, kF16>(a, st));
}

}  // namespace csa2
