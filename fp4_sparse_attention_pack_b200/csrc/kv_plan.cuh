// Work plan of the attention over pages, computed by every CTA from the counts
// on the device (they change between replays of a captured call).
//
// An item is a tile of query rows of one sequence and kv head: rows of a
// sequence are (token, head of the group) in that order, `kTile` to an item.  It
// costs one unit for each block of `kBlk` keys that its rows see and
// `kOver` more for its start and end.  The items' costs are laid end to end and
// cut into equal ranges, one for each CTA, so the work is even whatever the
// sequences' lengths; an item that a cut divides leaves partial results
// (unnormalised sums, maxima) in the workspace, which a second kernel joins.  A
// cut that falls within `kSnap` units of an item's start or end moves there, as
// the partial results cost about as much.  A CTA has at most two of them: the end
// of an item begun earlier (slot 2 c) and the beginning of one that goes on (slot
// 2 c + 1).  The joins' order is fixed,
// so equal calls give equal bits.
#pragma once

#include "kv.cuh"

namespace csa2 {

// A finite bound on the work of one call keeps the sums in 63 bits.
struct KvPlan {
    int g;        // query heads per kv head
    int grid;     // CTAs
    int min_per;  // least cost of a range
};

struct KvSeq {
    int row0, m, n;  // first row, new tokens (0: none, or left out), tokens held
};

__device__ __forceinline__ KvSeq kv_seq(const KvAttn& a, int b) {
    const NewTokens t = new_tokens(a.cu, b, a.total, a.max_new);
    if (t.m <= 0) return {0, 0, 0};
    return {t.row0, t.m, kv_held(a.c, b)};
}

// The first key that a row at position `pos` sees.  A position may lie 2^31 - 4096 below
// 0 (more new tokens than the cache holds), so the window is subtracted only where it
// begins behind key 0.
__device__ __forceinline__ int first_key(int pos, int window) {
    return window > 0 && pos >= window ? pos - window + 1 : 0;
}

// The keys [lo, hi] and blocks [b0, b1) that the rows of a tile see.
struct KvSpan {
    int t0, lo, hi, b0, b1;
};
template <int kTile, int kBlk>
__device__ __forceinline__ KvSpan kv_span(const KvSeq& s, int g, int window, int tile) {
    const int r1 = min((tile + 1) * (int64_t)kTile, (int64_t)s.m * g) - 1;
    KvSpan v;
    v.t0 = tile * kTile / g;
    v.hi = s.n - s.m + r1 / g;
    v.lo = first_key(s.n - s.m + v.t0, window);
    v.b0 = v.lo / kBlk;
    v.b1 = v.hi < 0 ? v.b0 : v.hi / kBlk + 1;
    return v;
}

__device__ __forceinline__ int kv_tiles(const KvSeq& s, int g, int tile) { return (s.m * g + tile - 1) / tile; }

// One CTA's share of an item: blocks [f0, f1).  first / last: it holds the
// item's first / last block (both: the whole item).
struct KvFrag {
    KvSeq s;
    KvSpan v;
    int b, h, tile, rows, f0, f1;
    int cost, rest;  // of the item; of what is behind this share
    bool first, last;
};

template <int kTile, int kBlk, int kOver>
struct KvCursor {
    KvSeq s;
    int b, h, tile, tiles, off;
    int64_t left;

    __device__ bool next(const KvAttn& a, int g, KvFrag& f) {
        while (left > 0) {
            if (tile >= tiles) {
                tile = 0;
                if (tiles == 0 || ++h >= a.c.kv_heads) {
                    h = 0;
                    if (++b >= a.c.batch) return false;
                    s = kv_seq(a, b);
                    tiles = kv_tiles(s, g, kTile);
                    if (tiles == 0) continue;
                }
            }
            const KvSpan v = kv_span<kTile, kBlk>(s, g, a.window, tile);
            const int nb = v.b1 - v.b0, cost = kOver + nb;
            const int take = (int)min(left, (int64_t)(cost - off));
            const int s0 = max(off - kOver, 0), s1 = max(off + take - kOver, 0);
            const bool some = s1 > s0 || (nb == 0 && off == 0);  // a tile that sees no key writes its zeros
            if (some) {
                f.s = s;
                f.v = v;
                f.b = b, f.h = h, f.tile = tile;
                f.rows = (int)min((int64_t)kTile, (int64_t)s.m * g - (int64_t)tile * kTile);
                f.f0 = v.b0 + s0, f.f1 = v.b0 + s1;
                f.first = s0 == 0, f.last = s1 == nb;
                f.cost = cost, f.rest = cost - off - take;
            }
            left -= take;
            off += take;
            if (off == cost) off = 0, ++tile;
            if (some) return true;
        }
        return false;
    }
};

// Where a cut at unit `off` of an item of cost `cost` goes.
template <int kSnap>
__device__ __forceinline__ int64_t snapped(int64_t off, int64_t cost) {
    if (off <= kSnap && off <= cost - off) return 0;
    return cost - off <= kSnap ? cost : off;
}

// What the plan needs in shared memory while it is made.
struct KvPlanSmem {
    int64_t cum[CSA2_KV_MAX_BATCH + 1], head[CSA2_KV_MAX_BATCH];  // running cost; that of one head
    int row0[CSA2_KV_MAX_BATCH], m[CSA2_KV_MAX_BATCH], n[CSA2_KV_MAX_BATCH];
    int64_t end[2];  // the range
    int first[7];    // b, h, tile, off; row0, m, n
};

// The whole block calls it; every thread gets its CTA's cursor.  cost_per: the
// range's length before cuts move.  The shared memory is free again after the call.
template <int kTile, int kBlk, int kOver, int kSnap>
__device__ __forceinline__ KvCursor<kTile, kBlk, kOver> kv_plan(const KvAttn& a, const KvPlan& p, KvPlanSmem& sm,
                                                                int64_t* cost_per) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int B = a.c.batch;
    for (int b = tid; b < B; b += blockDim.x) {
        const NewTokens t = new_tokens(a.cu, b, a.total, a.max_new);
        const int n = a.c.n_tokens[b];  // loaded beside the bounds
        if (t.m < 0 && blockIdx.x == 0) atomicOr(a.c.status, CSA2_DEVERR_COUNT);
        sm.row0[b] = t.row0;
        sm.m[b] = max(t.m, 0);
        sm.n[b] = t.m > 0 ? kv_held_of(a.c, n) : 0;
    }
    __syncthreads();
    for (int b = warp; b < B; b += warps) {
        const KvSeq s{0, sm.m[b], sm.n[b]};
        const int tiles = kv_tiles(s, p.g, kTile);
        int64_t cost = 0;
        for (int t = lane; t < tiles; t += 32) {
            const KvSpan v = kv_span<kTile, kBlk>(s, p.g, a.window, t);
            cost += kOver + v.b1 - v.b0;
        }
        if (tiles > 1) {
#pragma unroll
            for (int d = 16; d; d >>= 1) cost += __shfl_xor_sync(0xffffffffu, cost, d);
        }
        if (lane == 0) sm.cum[b + 1] = cost * a.c.kv_heads, sm.head[b] = cost;
    }
    __syncthreads();
    if (warp == 0) {  // running sums
        int64_t base = 0;
        for (int b0 = 0; b0 < B; b0 += 32) {
            int64_t v = b0 + lane < B ? sm.cum[b0 + lane + 1] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t u = __shfl_up_sync(0xffffffffu, v, d);
                if (lane >= d) v += u;
            }
            if (b0 + lane < B) sm.cum[b0 + lane + 1] = base + v;
            base += __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0) sm.cum[0] = 0;
    }
    __syncthreads();
    const int64_t W = sm.cum[B];
    const int64_t per = max((W + p.grid - 1) / p.grid, (int64_t)p.min_per);
    *cost_per = per;
    // a warp finds the item at one of the range's ends: warp 0 its start, warp 1 its end
    if (warp < 2) {
        const int64_t w = min((int64_t)(blockIdx.x + warp) * per, W);
        KvCursor<kTile, kBlk, kOver> c;
        c.b = 0, c.h = 0, c.tile = 0, c.tiles = 0, c.off = 0;
        c.s = {0, 0, 0};
        c.left = w;  // for now the end's place
        if (w < W) {
            int lo = 0, hi = B;  // the last b with cum[b] <= w (it has a cost: w < W)
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (sm.cum[mid] <= w) lo = mid;
                else hi = mid;
            }
            c.b = lo;
            c.s = {sm.row0[lo], sm.m[lo], sm.n[lo]};
            c.tiles = kv_tiles(c.s, p.g, kTile);
            const int64_t per_head = sm.head[lo];
            int64_t rem = w - sm.cum[lo];
            c.h = (int)(rem / per_head);
            rem -= c.h * per_head;
            for (int t0 = 0; t0 < c.tiles; t0 += 32) {
                int64_t cost = 0;
                if (t0 + lane < c.tiles) {
                    const KvSpan v = kv_span<kTile, kBlk>(c.s, p.g, a.window, t0 + lane);
                    cost = kOver + v.b1 - v.b0;
                }
                int64_t sum = cost;
#pragma unroll
                for (int d = 1; d < 32; d <<= 1) {
                    const int64_t u = __shfl_up_sync(0xffffffffu, sum, d);
                    if (lane >= d) sum += u;
                }
                const unsigned over = __ballot_sync(0xffffffffu, sum > rem);
                if (over) {
                    const int l = __ffs(over) - 1;
                    c.tile = t0 + l;
                    c.off = (int)(rem - __shfl_sync(0xffffffffu, sum - cost, l));
                    const int64_t item = __shfl_sync(0xffffffffu, cost, l);
                    const int64_t to = snapped<kSnap>(c.off, item);
                    c.left = w + to - c.off;
                    if (to == item) ++c.tile, c.off = 0;  // the next item, wherever it is
                    else c.off = (int)to;
                    break;
                }
                rem -= __shfl_sync(0xffffffffu, sum, 31);
            }
        }
        if (lane == 0) sm.end[warp] = c.left;
        if (warp == 0 && lane == 0) {
            sm.first[0] = c.b, sm.first[1] = c.h, sm.first[2] = c.tile, sm.first[3] = c.off;
            sm.first[4] = c.s.row0, sm.first[5] = c.s.m, sm.first[6] = c.s.n;
        }
    }
    __syncthreads();
    KvCursor<kTile, kBlk, kOver> c;
    c.b = sm.first[0], c.h = sm.first[1], c.tile = sm.first[2], c.off = sm.first[3];
    c.s = {sm.first[4], sm.first[5], sm.first[6]};
    c.tiles = kv_tiles(c.s, p.g, kTile);
    c.left = sm.end[1] - sm.end[0];
    __syncthreads();
    return c;
}

// The last CTA that has a share of an item which goes on behind CTA `cta`'s range.
template <int kSnap>
__device__ __forceinline__ int kv_last(int cta, int64_t per, const KvFrag& f) {
    const int k = (int)((f.rest + per - 1) / per);      // the cut k ranges on is the last inside the item
    const int64_t off = f.cost - f.rest + (k - 1) * per;  // its place in the item
    return cta + (k > 1 && snapped<kSnap>(off, f.cost) == f.cost ? k - 1 : k);
}

// Workspace: partial sums of a slot, (maximum in log2 units, sum) [slot][kTile],
// and for each CTA the item that goes on behind its range.
struct KvCut {
    int last;         // the last CTA that has a share of it, or -1: none
    int token0;       // row of the sequence's first new token
    int head0;        // first query head of the kv head
    int row0, rows;   // the item's first row (token, head) in the sequence, and how many
    int pad[3];
};
struct KvParts {
    float4* o;
    float2* ml;
    KvCut* cut;
};
inline size_t kv_parts_bytes(int grid, int tile, int dim) {
    return (size_t)2 * grid * tile * (dim * sizeof(float) + sizeof(float2)) + (size_t)grid * sizeof(KvCut);
}
inline KvParts kv_parts(void* ws, int grid, int tile, int dim) {
    KvParts p;
    p.o = static_cast<float4*>(ws);
    p.ml = reinterpret_cast<float2*>(p.o + (size_t)2 * grid * tile * (dim / 4));
    p.cut = reinterpret_cast<KvCut*>(p.ml + (size_t)2 * grid * tile);
    return p;
}
template <int kSnap>
__device__ __forceinline__ KvCut kv_cut(const KvFrag& f, int cta, int64_t per, int g, int tile_rows) {
    return {kv_last<kSnap>(cta, per, f), f.s.row0, f.h * g, f.tile * tile_rows, f.rows, {0, 0, 0}};
}

}  // namespace csa2
