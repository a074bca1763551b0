// C ABI of the paged key/value cache operators: argument checks and descriptors.
// Everything is checked before the first launch, as in api.cu.
#include <cmath>
#include <cstring>

#include "kv.cuh"

using namespace csa2;

namespace {

inline bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_kv_cache(const csa2_kv_cache* c) {
    if (!c || !c->k_pages || !c->v_pages || !c->page_table || !c->n_tokens || !c->status) return CSA2_ERR_INVALID_ARG;
    if (c->batch < 1 || c->max_pages < 1 || c->num_pages < 1 || c->kv_heads < 1) return CSA2_ERR_INVALID_ARG;
    if (c->dtype != CSA2_KV_BF16 && c->dtype != CSA2_KV_F16 && c->dtype != CSA2_KV_E4M3) return CSA2_ERR_INVALID_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return CSA2_ERR_UNSUPPORTED;
    if (c->batch > CSA2_KV_MAX_BATCH || c->kv_heads > CSA2_MAX_H) return CSA2_ERR_UNSUPPORTED;
    if ((int64_t)c->max_pages * PAGE > (int64_t)1 << 30) return CSA2_ERR_UNSUPPORTED;
    if ((int64_t)c->num_pages * c->kv_heads * PAGE >= (int64_t)1 << 31) return CSA2_ERR_UNSUPPORTED;
    if (!a16(c->k_pages) || !a16(c->v_pages) || !a16(c->page_table) || !a16(c->n_tokens) || !a16(c->status))
        return CSA2_ERR_ALIGN;
    return CSA2_OK;
}

KvView kv_view(const csa2_kv_cache& c) {
    return KvView{static_cast<uint8_t*>(c.k_pages), static_cast<uint8_t*>(c.v_pages), c.page_table, c.n_tokens,
                  c.status, c.batch, c.max_pages, c.num_pages, c.kv_heads};
}

// A tensor of tokens x heads x dim; an output's rows must not overlap.
int check_heads(const csa2_heads* x, int64_t tokens, int heads, int dim, bool output) {
    if (!x || !x->data || x->token_stride < 0 || x->head_stride < 0) return CSA2_ERR_INVALID_ARG;
    if (output && ((tokens > 1 && x->token_stride < dim) || (heads > 1 && x->head_stride < dim)))
        return CSA2_ERR_INVALID_ARG;
    if (output && tokens > 1 && heads > 1 &&
        x->token_stride < (heads - 1) * x->head_stride + dim && x->head_stride < (tokens - 1) * x->token_stride + dim)
        return CSA2_ERR_INVALID_ARG;  // neither is the outer dimension: rows could meet
    if (!a16(x->data) || x->token_stride % 8 || x->head_stride % 8) return CSA2_ERR_ALIGN;
    return CSA2_OK;
}

HeadsView heads_view(const csa2_heads& x) {
    return HeadsView{static_cast<uint8_t*>(x.data), x.token_stride, x.head_stride};
}

int check_rotary(const csa2_rotary* r, int head_dim) {
    if (!r || !r->inv_freq) return CSA2_ERR_INVALID_ARG;
    if (r->rot_dim < 16 || r->rot_dim % 16 || r->rot_dim > CSA2_MAX_ROT || r->rot_offset < 0 || r->rot_offset % 8 ||
        r->rot_offset > head_dim - r->rot_dim)
        return CSA2_ERR_INVALID_ARG;
    if ((r->neighbours != 0 && r->neighbours != 1) || r->n_axes < 1 || r->n_axes > CSA2_MAX_AXES)
        return CSA2_ERR_INVALID_ARG;
    if (r->axis)
        for (int i = 0; i < r->rot_dim / 2; ++i)
            if (r->axis[i] >= r->n_axes) return CSA2_ERR_INVALID_ARG;
    if (!a16(r->inv_freq)) return CSA2_ERR_ALIGN;
    return CSA2_OK;
}

RotaryView rotary_view(const csa2_rotary& r, const int32_t* pos, int64_t pos_stride, bool inverse) {
    RotaryView v;
    std::memset(&v, 0, sizeof(v));
    v.inv_freq = r.inv_freq;
    v.pos = pos;
    v.pos_stride = pos_stride;
    if (r.axis)
        for (int i = 0; i < r.rot_dim / 2; ++i) v.axis[i / 16] |= (uint32_t)r.axis[i] << (2 * (i % 16));
    v.rot = r.rot_dim;
    v.offset = r.rot_offset;
    v.neighbours = r.neighbours;
    v.sign = inverse ? -1.0f : 1.0f;
    return v;
}

// The cache's type for inputs of `dtype`: the same 16-bit type, or E4M3.
bool kv_types_match(int dtype, int kv_dtype) {
    if (dtype == CSA2_DTYPE_BF16) return kv_dtype == CSA2_KV_BF16 || kv_dtype == CSA2_KV_E4M3;
    if (dtype == CSA2_DTYPE_F16) return kv_dtype == CSA2_KV_F16 || kv_dtype == CSA2_KV_E4M3;
    return false;
}

int cuda_status(cudaError_t e) { return e == cudaSuccess ? CSA2_OK : CSA2_ERR_CUDA; }

}  // namespace

extern "C" {

int csa2_rotate(const csa2_rotary* rot, const csa2_heads* x, const csa2_heads* y, int dtype, int64_t n_tokens,
                int heads, int head_dim, const int32_t* pos, int inverse, csa2_stream stream) {
    if (dtype != CSA2_DTYPE_BF16 && dtype != CSA2_DTYPE_F16 && dtype != CSA2_DTYPE_F32) return CSA2_ERR_INVALID_ARG;
    if (n_tokens < 0 || heads < 1 || head_dim < 8 || head_dim % 8 || head_dim > D || (inverse != 0 && inverse != 1))
        return CSA2_ERR_INVALID_ARG;
    int rc = check_rotary(rot, head_dim);
    if (rc) return rc;
    if (n_tokens == 0) return CSA2_OK;
    if (n_tokens > (int64_t)1 << 30 || heads > CSA2_ROTATE_MAX_HEADS) return CSA2_ERR_UNSUPPORTED;
    if ((rc = check_heads(x, n_tokens, heads, head_dim, false)) || (rc = check_heads(y, n_tokens, heads, head_dim, true)))
        return rc;
    if (!pos) return CSA2_ERR_INVALID_ARG;
    if (!a16(pos)) return CSA2_ERR_ALIGN;
    if (x->data == y->data && (x->token_stride != y->token_stride || x->head_stride != y->head_stride) &&
        n_tokens * heads > 1)
        return CSA2_ERR_INVALID_ARG;  // in place only with the same strides
    if (inject_fault("csa2_rotate")) return CSA2_ERR_CUDA;
    return cuda_status(launch_rotate(rotary_view(*rot, pos, n_tokens, inverse == 1), heads_view(*x), heads_view(*y),
                                     dtype, n_tokens, heads, head_dim, (cudaStream_t)stream));
}

int csa2_kv_append(const csa2_kv_cache* cache, const csa2_heads* k, const csa2_heads* v, int dtype, const int32_t* cu,
                   int total, int max_new, const int32_t* start, const csa2_rotary* rot, const int32_t* pos,
                   csa2_stream stream) {
    int rc = check_kv_cache(cache);
    if (rc) return rc;
    if (!kv_types_match(dtype, cache->dtype) || total < 0 || max_new < 0) return CSA2_ERR_INVALID_ARG;
    if (rot && (rc = check_rotary(rot, cache->head_dim))) return rc;
    if (!rot && pos) return CSA2_ERR_INVALID_ARG;
    if (!cu) return CSA2_ERR_INVALID_ARG;
    if (!a16(cu) || !a16(start) || !a16(pos)) return CSA2_ERR_ALIGN;
    if (start && start != cache->n_tokens && start < cache->n_tokens + cache->batch &&
        cache->n_tokens < start + cache->batch)
        return CSA2_ERR_INVALID_ARG;  // start overlaps n_tokens
    if (total > 1 << 30) return CSA2_ERR_UNSUPPORTED;
    if (total > 0) {
        if ((rc = check_heads(k, total, cache->kv_heads, cache->head_dim, false)) ||
            (rc = check_heads(v, total, cache->kv_heads, cache->head_dim, false)))
            return rc;
    }
    if (inject_fault("csa2_kv_append")) return CSA2_ERR_CUDA;
    KvAppend a;
    std::memset(&a, 0, sizeof(a));
    a.c = kv_view(*cache);
    if (total > 0) {
        a.k = heads_view(*k);
        a.v = heads_view(*v);
    }
    a.cu = cu;
    a.start = start == cache->n_tokens ? nullptr : start;
    a.total = total;
    a.max_new = max_new;
    RotaryView r;
    if (rot) r = rotary_view(*rot, pos, total, false);
    return cuda_status(launch_kv_append(a, rot ? &r : nullptr, cache->head_dim, dtype, cache->dtype,
                                        (cudaStream_t)stream));
}

size_t csa2_kv_attn_workspace(const csa2_kv_cache* cache, int total, int max_new, int H) {
    if (check_kv_cache(cache) || total < 0 || max_new < 0 || H < 1 || H > CSA2_MAX_H || H % cache->kv_heads) return 0;
    return kv_attn_workspace_bytes(max_new, H, *cache);
}

int csa2_kv_attn(const csa2_kv_cache* cache, const csa2_heads* q, int H, int dtype, const int32_t* cu, int total,
                 int max_new, float scale, int window, const csa2_heads* out, float* lse, void* ws, size_t ws_bytes,
                 csa2_stream stream) {
    int rc = check_kv_cache(cache);
    if (rc) return rc;
    if (!kv_types_match(dtype, cache->dtype) || total < 0 || max_new < 0 || window < 0 || H < 1 || H > CSA2_MAX_H ||
        H % cache->kv_heads || !std::isfinite(scale) || scale <= 0.0f || !cu)
        return CSA2_ERR_INVALID_ARG;
    if ((int64_t)total * H > ((int64_t)1 << 31) - 4096) return CSA2_ERR_UNSUPPORTED;  // rows are counted in 32 bits
    if (total == 0) return CSA2_OK;
    if ((rc = check_heads(q, total, H, cache->head_dim, false)) || (rc = check_heads(out, total, H, cache->head_dim, true)))
        return rc;
    if (q->data == out->data) return CSA2_ERR_INVALID_ARG;
    if (!a16(cu) || !a16(lse) || !a16(ws)) return CSA2_ERR_ALIGN;
    const size_t need = kv_attn_workspace_bytes(max_new, H, *cache);
    if (need > 0 && (!ws || ws_bytes < need)) return CSA2_ERR_WORKSPACE;
    if (inject_fault("csa2_kv_attn")) return CSA2_ERR_CUDA;
    KvAttn a;
    std::memset(&a, 0, sizeof(a));
    a.c = kv_view(*cache);
    a.q = heads_view(*q);
    a.out = heads_view(*out);
    a.cu = cu;
    a.lse = lse;
    a.ws = ws;
    a.H = H;
    a.total = total;
    a.max_new = max_new;
    a.window = window < cache->max_pages * PAGE ? window : 0;  // one of the whole capacity hides nothing
    a.scale = scale;
    return cuda_status(launch_kv_attn(a, cache->head_dim, dtype, cache->dtype, (cudaStream_t)stream));
}

}  // extern "C"
