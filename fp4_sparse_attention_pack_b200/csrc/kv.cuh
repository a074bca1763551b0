// Shared definitions of the paged key/value cache operators (kv_*.cu).
#pragma once

#include "common.cuh"
#include "kernels.cuh"

namespace csa2 {

// Device view of a key/value cache (plain values, passed by value to kernels).
struct KvView {
    uint8_t* k;
    uint8_t* v;
    const int32_t* page_table;
    int32_t* n_tokens;
    uint32_t* status;
    int batch, max_pages, num_pages, kv_heads;
};

struct HeadsView {
    uint8_t* p;
    int64_t ts, hs;  // strides in elements
};

// A rotation as kernels take it: two bits of axis for each pair.
struct RotaryView {
    const float* inv_freq;
    const int32_t* pos;   // [n_axes][pos_stride], or null: the slot number on every axis
    int64_t pos_stride;
    uint32_t axis[CSA2_MAX_ROT / 2 / 16];
    int rot, offset, neighbours;
    float sign;           // -1: the inverse
};

// The new tokens of sequence b: rows row0 .. row0 + m - 1; m = -1 when the bounds
// are not 0 <= cu[b] <= cu[b + 1] <= total with at most max_new tokens.
struct NewTokens {
    int row0, m;
};
__device__ __forceinline__ NewTokens new_tokens(const int32_t* cu, int b, int total, int max_new) {
    const int a = cu[b], e = cu[b + 1];
    if (a < 0 || e < a || e > total || e - a > max_new) return {0, -1};
    return {a, e - a};
}

// Tokens that sequence b holds, clamped to the table's capacity; n: its count as stored.
__device__ __forceinline__ int kv_held_of(const KvView& c, int n) {
    const int cap = c.max_pages * PAGE;
    if (n < 0 || n > cap) {
        atomicOr(c.status, CSA2_DEVERR_COUNT);
        n = n < 0 ? 0 : cap;
    }
    return n;
}
__device__ __forceinline__ int kv_held(const KvView& c, int b) { return kv_held_of(c, c.n_tokens[b]); }

// Physical page of a sequence's logical page, or -1 (and a status bit) when the
// table points outside the pool.
__device__ __forceinline__ int kv_page(const KvView& c, int b, int logical) {
    const int p = c.page_table[(int64_t)b * c.max_pages + logical];
    if (p < 0 || p >= c.num_pages) {
        atomicOr(c.status, CSA2_DEVERR_PAGE);
        return -1;
    }
    return p;
}

cudaError_t launch_rotate(const RotaryView& r, const HeadsView& x, const HeadsView& y, int dtype, int64_t n_tokens,
                          int heads, int head_dim, cudaStream_t st);

struct KvAppend {
    KvView c;
    HeadsView k, v;
    const int32_t* cu;
    const int32_t* start;  // null: behind n_tokens
    int total, max_new;
};
cudaError_t launch_kv_append(const KvAppend& a, const RotaryView* r, int head_dim, int dtype, int kv_dtype,
                             cudaStream_t st);

struct KvAttn {
    KvView c;
    HeadsView q, out;
    const int32_t* cu;
    float* lse;
    void* ws;
    int H, total, max_new, window;
    float scale;
};
size_t kv_attn_workspace_bytes(int max_new, int H, const csa2_kv_cache& c);
cudaError_t launch_kv_attn(const KvAttn& a, int head_dim, int dtype, int kv_dtype, cudaStream_t st);

}  // namespace csa2
