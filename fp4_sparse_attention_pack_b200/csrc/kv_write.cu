// Rotary positions, and the append of new keys and values to the pages with the
// rotation on the way.
//
// Pair i of a token turns by the angle pos * inv_freq[i].  The angle is formed
// in turns (revolutions) in fp64 and reduced to [-1/2, 1/2] there, so positions
// of a million and more keep an error near 2^-25 of a turn; sine and cosine of
// the reduced angle and the rotation are fp32, rounded once to the output type.
// The angles of a token are the same for all its heads: a CTA computes them once
// into shared memory and then streams its rows.
//
// Both kernels are bound by memory (large calls) or by latency (a decode step).
// A thread's unit of work is 8 channels of a row, or 8 + 8 when the pair's two
// channels are half a rotation apart, so every access is 16 bytes (8 for the
// write of E4M3 codes) and a warp covers whole lines.
#include <algorithm>

#include "kv.cuh"

namespace csa2 {

namespace {

constexpr int kThreads = 256;

template <typename T>
struct Vec8;  // 8 channels as they lie in memory
template <>
struct Vec8<float> {
    float4 a, b;
};
template <>
struct Vec8<__nv_bfloat16> {
    uint4 a;
};
template <>
struct Vec8<__half> {
    uint4 a;
};
template <>
struct Vec8<__nv_fp8_e4m3> {
    uint2 a;
};

__device__ __forceinline__ void unpack(const Vec8<float>& v, float (&f)[8]) {
    f[0] = v.a.x, f[1] = v.a.y, f[2] = v.a.z, f[3] = v.a.w;
    f[4] = v.b.x, f[5] = v.b.y, f[6] = v.b.z, f[7] = v.b.w;
}
__device__ __forceinline__ void unpack(const Vec8<__nv_bfloat16>& v, float (&f)[8]) {
    const uint32_t w[4] = {v.a.x, v.a.y, v.a.z, v.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void unpack(const Vec8<__half>& v, float (&f)[8]) {
    const uint32_t w[4] = {v.a.x, v.a.y, v.a.z, v.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        __half2 h;
        memcpy(&h, &w[i], 4);
        const float2 p = __half22float2(h);
        f[2 * i] = p.x, f[2 * i + 1] = p.y;
    }
}

__device__ __forceinline__ void pack(const float (&f)[8], Vec8<float>& v) {
    v.a = make_float4(f[0], f[1], f[2], f[3]);
    v.b = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void pack(const float (&f)[8], Vec8<__nv_bfloat16>& v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        memcpy(&w[i], &h, 4);
    }
    v.a = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(const float (&f)[8], Vec8<__half>& v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
        memcpy(&w[i], &h, 4);
    }
    v.a = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(const float (&f)[8], Vec8<__nv_fp8_e4m3>& v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // nearest even, saturating at +-448, NaN kept
        w[i] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    v.a = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

template <typename T>
__device__ __forceinline__ Vec8<T> load8(const T* p) {
    return *reinterpret_cast<const Vec8<T>*>(p);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const Vec8<T>& v) {
    *reinterpret_cast<Vec8<T>*>(p) = v;
}

// 8 channels unchanged but for the type.
template <typename In, typename Out>
__device__ __forceinline__ void copy8(const In* src, Out* dst) {
    if constexpr (std::is_same<In, Out>::value) {
        store8(dst, load8(src));
    } else {
        float f[8];
        Vec8<Out> o;
        unpack(load8(src), f);
        pack(f, o);
        store8(dst, o);
    }
}

// Units of a row that rotate; the other channels are (dim - rot) / 8 more.
__host__ __device__ __forceinline__ int rot_units(int rot, int neighbours) { return neighbours ? rot / 8 : rot / 16; }

// Unit u of a row whose first R units rotate by cs (one (cos, sin) per pair).
template <typename In, typename Out>
__device__ __forceinline__ void row_unit(const In* src, Out* dst, int u, int R, const RotaryView& r, const float2* cs) {
    if (u >= R) {
        int c = 8 * (u - R);
        if (c >= r.offset) c += r.rot;
        copy8(src + c, dst + c);
    } else if (r.neighbours) {
        const int c = r.offset + 8 * u;
        float f[8], g[8];
        unpack(load8(src + c), f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 w = cs[4 * u + i];
            g[2 * i] = f[2 * i] * w.x - f[2 * i + 1] * w.y;
            g[2 * i + 1] = f[2 * i + 1] * w.x + f[2 * i] * w.y;
        }
        Vec8<Out> o;
        pack(g, o);
        store8(dst + c, o);
    } else {
        const int c = r.offset + 8 * u, h = r.rot / 2;
        float a[8], b[8], x[8], y[8];
        const Vec8<In> va = load8(src + c), vb = load8(src + c + h);
        unpack(va, a);
        unpack(vb, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 w = cs[8 * u + i];
            x[i] = a[i] * w.x - b[i] * w.y;
            y[i] = b[i] * w.x + a[i] * w.y;
        }
        Vec8<Out> o;
        pack(x, o);
        store8(dst + c, o);
        pack(y, o);
        store8(dst + c + h, o);
    }
}

// (cos, sin) of pair i at a position.
__device__ __forceinline__ float2 turn_of(const RotaryView& r, int i, int position) {
    constexpr double kTurns = 0.15915494309189533577;  // 1 / (2 pi)
    const double t = (double)position * ((double)r.inv_freq[i] * kTurns);
    const float f = (float)(t - rint(t));
    float s, c;
    sincospif(2.0f * f, &s, &c);
    return make_float2(c, r.sign * s);
}

__device__ __forceinline__ int axis_of(const RotaryView& r, int i) { return (r.axis[i / 16] >> (2 * (i % 16))) & 3; }

// Rows of `tt` tokens x `ht` heads a CTA: blockIdx.x tokens, blockIdx.y heads.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_rotate(const __grid_constant__ RotaryView r, HeadsView x, HeadsView y,
                                                     int64_t n_tokens, int heads, int tt, int ht, int units) {
    extern __shared__ float2 cs[];  // [tt][rot / 2]
    const int64_t t0 = (int64_t)blockIdx.x * tt;
    const int nt = (int)min((int64_t)tt, n_tokens - t0);
    const int h0 = blockIdx.y * ht, nh = min(ht, heads - h0);
    const int half = r.rot / 2;
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, p = i - t * half;
        cs[i] = turn_of(r, p, r.pos[axis_of(r, p) * r.pos_stride + t0 + t]);
    }
    __syncthreads();
    const int R = rot_units(r.rot, r.neighbours);
    for (int i = threadIdx.x; i < nt * nh * units; i += kThreads) {
        const int row = i / units, u = i - row * units;
        const int t = row / nh, h = row - t * nh;
        const T* src = reinterpret_cast<const T*>(x.p) + (t0 + t) * x.ts + (h0 + h) * x.hs;
        T* dst = reinterpret_cast<T*>(y.p) + (t0 + t) * y.ts + (h0 + h) * y.hs;
        row_unit(src, dst, u, R, r, cs + t * half);
    }
}

// What an append does with sequence b: its first row and token count, and the
// slot of its first token; m = -1 when the sequence is left out (the bits say why).
struct Placed {
    int row0, m, slot0;
    uint32_t bits;
};
__device__ __forceinline__ Placed place(const KvAppend& a, const int32_t* cu, int b) {
    const NewTokens n = new_tokens(cu, b, a.total, a.max_new);
    if (n.m < 0) return {0, -1, 0, CSA2_DEVERR_COUNT};
    const int cap = a.c.max_pages * PAGE;
    int s = a.start ? a.start[b] : a.c.n_tokens[b];
    uint32_t bits = 0;
    if (!a.start && (s < 0 || s > cap)) {  // a held count is clamped, as wherever it is read
        bits = CSA2_DEVERR_COUNT;
        s = s < 0 ? 0 : cap;
    }
    if (s < 0 || (int64_t)s + n.m > cap) return {0, -1, 0, bits | CSA2_DEVERR_CAPACITY};
    return {n.row0, n.m, s, bits};
}

// n_tokens of sequences t, t + step, ... and the bits of those left out.
__device__ __forceinline__ void count_tokens(const KvAppend& a, const int32_t* cu, int t, int step) {
    for (int b = t; b < a.c.batch; b += step) {
        const Placed p = place(a, cu, b);
        if (p.bits) atomicOr(a.c.status, p.bits);
        if (p.m >= 0) a.c.n_tokens[b] = p.slot0 + p.m;
    }
}

// `tt` new tokens a CTA (blockIdx.x), `ht` kv heads (blockIdx.y).  A CTA first
// finds its tokens' sequences (cu in shared memory), slots and pages.  With an
// explicit start the first CTA also writes the counts, which nothing reads here.
template <typename In, typename Out>
__global__ void __launch_bounds__(kThreads) k_kv_append(const __grid_constant__ KvAppend a,
                                                        const __grid_constant__ RotaryView r, int dim, int tt, int ht,
                                                        int units_k) {
    extern __shared__ float2 cs[];                                // [tt][rot / 2]
    const int half = r.rot / 2;
    int64_t* row = reinterpret_cast<int64_t*>(cs + tt * half);    // [tt] element of head 0 in the pools, or -1
    int* slot = reinterpret_cast<int*>(row + tt);                 // [tt]
    int* cu = slot + tt;                                          // [batch + 1]
    const int t0 = blockIdx.x * tt, nt = min(tt, a.total - t0);
    const int h0 = blockIdx.y * ht, nh = min(ht, a.c.kv_heads - h0);
    for (int i = threadIdx.x; i <= a.c.batch; i += kThreads) cu[i] = a.cu[i];
    __syncthreads();
    for (int i = threadIdx.x; i < nt; i += kThreads) {
        const int t = t0 + i;
        int lo = 0, hi = a.c.batch;  // the last b with cu[b] <= t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t) lo = mid;
            else hi = mid;
        }
        const Placed p = place(a, cu, lo);
        int64_t at = -1;
        int s = 0;
        if (p.m > 0 && t >= p.row0 && t < p.row0 + p.m) {
            s = p.slot0 + (t - p.row0);
            const int page = kv_page(a.c, lo, s / PAGE);
            if (page >= 0) at = ((int64_t)page * a.c.kv_heads * PAGE + s % PAGE) * dim;
        }
        row[i] = at;
        slot[i] = s;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, p = i - t * half;
        if (row[t] >= 0)
            cs[i] = turn_of(r, p, r.pos ? r.pos[axis_of(r, p) * r.pos_stride + t0 + t] : slot[t]);
    }
    __syncthreads();
    const int R = rot_units(r.rot, r.neighbours), units = units_k + dim / 8;
    for (int i = threadIdx.x; i < nt * nh * units; i += kThreads) {
        const int rw = i / units, u = i - rw * units;
        const int t = rw / nh, h = rw - t * nh + h0;
        if (row[t] < 0) continue;
        const int64_t at = row[t] + (int64_t)h * PAGE * dim;
        if (u < units_k) {
            row_unit(reinterpret_cast<const In*>(a.k.p) + (int64_t)(t0 + t) * a.k.ts + h * a.k.hs,
                     reinterpret_cast<Out*>(a.c.k) + at, u, R, r, cs + t * half);
        } else {
            const int c = 8 * (u - units_k);
            copy8(reinterpret_cast<const In*>(a.v.p) + (int64_t)(t0 + t) * a.v.ts + h * a.v.hs + c,
                  reinterpret_cast<Out*>(a.c.v) + at + c);
        }
    }
    if (a.start && blockIdx.x == 0 && blockIdx.y == 0) count_tokens(a, cu, threadIdx.x, kThreads);
}

// The counts when they are also the start: after every CTA has read them.
__global__ void k_kv_count(const __grid_constant__ KvAppend a) {
    count_tokens(a, a.cu, threadIdx.x, blockDim.x);
}

// Tokens and heads of a CTA: about 2,048 units, fewer (down to one unit a
// thread) while the CTAs would not fill the SMs twice.
void tile_rows(int64_t tokens, int heads, int units, int half, int& tt, int& ht) {
    const int64_t want = 2 * device_sm_count();
    int per = 2048;
    while (per > kThreads && tokens * heads * units / per < want) per /= 2;
    ht = std::max(1, std::min(heads, per / units));
    tt = ht < heads ? 1 : (int)std::max<int64_t>(1, std::min<int64_t>(per / (units * heads), 64));
    tt = (int)std::min<int64_t>(tt, tokens);
    if (half > 0) tt = std::min(tt, 4096 / half);  // 32 KB of (cos, sin)
}

template <typename T>
cudaError_t rotate_as(const RotaryView& r, const HeadsView& x, const HeadsView& y, int64_t n_tokens, int heads, int dim,
                      cudaStream_t st) {
    const bool in_place = x.p == y.p;  // the other channels are there already
    const int units = rot_units(r.rot, r.neighbours) + (in_place ? 0 : (dim - r.rot) / 8);
    int tt, ht;
    tile_rows(n_tokens, heads, units, r.rot / 2, tt, ht);
    const dim3 grid((unsigned)((n_tokens + tt - 1) / tt), (heads + ht - 1) / ht);
    k_rotate<T><<<grid, kThreads, (size_t)tt * (r.rot / 2) * sizeof(float2), st>>>(r, x, y, n_tokens, heads, tt, ht,
                                                                                   units);
    return cudaGetLastError();
}

template <typename In, typename Out>
cudaError_t append_as(const KvAppend& a, const RotaryView& r, int dim, cudaStream_t st) {
    if (a.total > 0) {
        const int units_k = rot_units(r.rot, r.neighbours) + (dim - r.rot) / 8;
        int tt, ht;
        tile_rows(a.total, a.c.kv_heads, units_k + dim / 8, r.rot / 2, tt, ht);
        const dim3 grid((a.total + tt - 1) / tt, (a.c.kv_heads + ht - 1) / ht);
        const size_t smem = (size_t)tt * (r.rot / 2 * sizeof(float2) + sizeof(int64_t) + sizeof(int)) +
                            (size_t)(a.c.batch + 1) * sizeof(int);
        k_kv_append<In, Out><<<grid, kThreads, smem, st>>>(a, r, dim, tt, ht, units_k);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        if (a.start) return cudaSuccess;
    }
    k_kv_count<<<1, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rotate(const RotaryView& r, const HeadsView& x, const HeadsView& y, int dtype, int64_t n_tokens,
                          int heads, int head_dim, cudaStream_t st) {
    if (dtype == CSA2_DTYPE_BF16) return rotate_as<__nv_bfloat16>(r, x, y, n_tokens, heads, head_dim, st);
    if (dtype == CSA2_DTYPE_F16) return rotate_as<__half>(r, x, y, n_tokens, heads, head_dim, st);
    return rotate_as<float>(r, x, y, n_tokens, heads, head_dim, st);
}

cudaError_t launch_kv_append(const KvAppend& a, const RotaryView* rot, int head_dim, int dtype, int kv_dtype,
                             cudaStream_t st) {
    RotaryView r = {};
    if (rot) r = *rot;
    const bool e4m3 = kv_dtype == CSA2_KV_E4M3;
    if (dtype == CSA2_DTYPE_BF16)
        return e4m3 ? append_as<__nv_bfloat16, __nv_fp8_e4m3>(a, r, head_dim, st)
                    : append_as<__nv_bfloat16, __nv_bfloat16>(a, r, head_dim, st);
    return e4m3 ? append_as<__half, __nv_fp8_e4m3>(a, r, head_dim, st)
                : append_as<__half, __half>(a, r, head_dim, st);
}

}  // namespace csa2
