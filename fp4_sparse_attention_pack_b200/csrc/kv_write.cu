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
// A thread's unit of work is 8 or 16 neighbouring channels of a row, or 8 + 8 when
// the pair's two channels are half a rotation apart, so every access is 16 bytes
// (8 for some writes of E4M3 codes) and a warp covers whole lines.  A thread has at
// most four units and loads all of them before it looks up positions, slots and pages
// and computes the angles, so those chains of small loads lie under the large ones.
//
// 4,096 tokens of 64 heads of 512, the last 64 rotating, bf16: 92 us (5.9 TB/s, 91% of
// the copy rate).  8,191 tokens of 16 heads of 128, three axes, fp16: 15 us (70%; issue
// slots 67% busy).  Append of 16 x 8,192 tokens, 8 heads of 128, to E4M3 pages: 170 us
// (4.7 TB/s, 73%; issue slots 63% busy; a cheaper sine and cosine, packed products and
// other tile sizes changed nothing).
#include <algorithm>

#include "kv.cuh"

namespace csa2 {

namespace {

constexpr int kThreads = 128;  // (256 and 512: 3% and 18% slower for the large append)
template <typename In>
constexpr int kUnits = sizeof(In) == 4 ? 2 : 4;  // units of a thread
constexpr int kMaxTokens = 64;                   // of a CTA

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

template <typename In, typename Out>
__device__ __forceinline__ void convert8(const Vec8<In>& v, Vec8<Out>& o) {
    if constexpr (std::is_same<In, Out>::value) {
        o = v;
    } else {
        float f[8];
        unpack(v, f);
        pack(f, o);
    }
}

// Units of a row that rotate; the other channels are (dim - rot) / 8 more.
__host__ __device__ __forceinline__ int rot_units(int rot, int neighbours) { return neighbours ? rot / 8 : rot / 16; }

// First channel of a unit of `width` channels that does not rotate, the u-th such one of a row.
__device__ __forceinline__ int other_channel(const RotaryView& r, int u, int width) {
    const int c = width * u;
    return c >= r.offset ? c + r.rot : c;
}
template <typename In>
struct Unit {
    Vec8<In> a, b;  // b: the pairs' other channels, half a rotation behind, or the next 8
};
// Units that do not rotate: 8 channels, or 16.
template <typename In>
__device__ __forceinline__ void load_plain(Unit<In>& x, const In* src, int width) {
    x.a = load8(src);
    if (width == 16) x.b = load8(src + 8);
}
template <typename In, typename Out>
__device__ __forceinline__ void store_plain(const Unit<In>& v, Out* dst, int width) {
    Vec8<Out> o;
    convert8(v.a, o);
    if constexpr (sizeof(Out) == 1) {
        if (width == 16) {
            Vec8<Out> p;
            convert8(v.b, p);
            *reinterpret_cast<uint4*>(dst) = make_uint4(o.a.x, o.a.y, p.a.x, p.a.y);
            return;
        }
    }
    store8(dst, o);
    if (width == 16) {
        convert8(v.b, o);
        store8(dst + 8, o);
    }
}
// Unit u of a row that rotates.
template <typename In>
__device__ __forceinline__ void load_turn(Unit<In>& x, const In* src, int u, const RotaryView& r) {
    src += r.offset + 8 * u;
    x.a = load8(src);
    if (!r.neighbours) x.b = load8(src + r.rot / 2);
}
template <typename In, typename Out>
__device__ __forceinline__ void store_turn(const Unit<In>& v, Out* dst, int u, const RotaryView& r, const float2* cs) {
    Vec8<Out> o;
    float a[8], x[8];
    dst += r.offset + 8 * u;
    unpack(v.a, a);
    if (r.neighbours) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 w = cs[u + i * (r.rot / 8)];
            x[2 * i] = a[2 * i] * w.x - a[2 * i + 1] * w.y;
            x[2 * i + 1] = a[2 * i + 1] * w.x + a[2 * i] * w.y;
        }
    } else {
        float b[8], y[8];
        unpack(v.b, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 w = cs[u + i * (r.rot / 16)];
            x[i] = a[i] * w.x - b[i] * w.y;
            y[i] = b[i] * w.x + a[i] * w.y;
        }
        pack(y, o);
        store8(dst + r.rot / 2, o);
    }
    pack(x, o);
    store8(dst, o);
}

// Division of x < 2^16 by d < 2^16: m = 2^32 / d + 1 (0 for d = 1).
struct Divisor {
    uint32_t d, m;
};
__device__ __forceinline__ int divide(int x, const Divisor& v) { return v.m ? (int)__umulhi((uint32_t)x, v.m) : x; }
__host__ __device__ __forceinline__ Divisor divisor(int d) {
    return {(uint32_t)d, d > 1 ? 0xFFFFFFFFu / (uint32_t)d + 1 : 0};
}

// The units of a CTA's rows, kind after kind, so that a warp's are nearly always
// of one kind: those that rotate, the other channels of the same rows, and (an
// append) the values'.
struct Kinds {
    Divisor turn, other, value;  // units of a row
    int width;                   // channels of a unit of the others
};
struct Where {
    uint32_t bits;  // the unit of the row 0-7, head 8-18, token 19-25, kind 26-27
    __device__ __forceinline__ int u() const { return bits & 0xFF; }
    __device__ __forceinline__ int h() const { return bits >> 8 & 0x7FF; }
    __device__ __forceinline__ int t() const { return bits >> 19 & 0x7F; }
    __device__ __forceinline__ int kind() const { return bits >> 26; }
};
__device__ __forceinline__ Where where(int i, int nt, int nh, const Divisor& per_token, const Kinds& k) {
    const int n0 = nt * nh * k.turn.d, n1 = nt * nh * k.other.d;
    const int kind = i < n0 ? 0 : i < n0 + n1 ? 1 : 2;
    const Divisor& v = kind == 0 ? k.turn : kind == 1 ? k.other : k.value;
    i -= kind == 0 ? 0 : kind == 1 ? n0 : n0 + n1;
    const int row = divide(i, v), t = divide(row, per_token);
    return {(uint32_t)(i - row * (int)v.d) | (uint32_t)(row - t * nh) << 8 | (uint32_t)t << 19 | (uint32_t)kind << 26};
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

// Place of a token's pair p in shared memory: neighbouring units' (cos, sin) side
// by side, so that a warp reads them without bank conflicts.
__device__ __forceinline__ int cs_at(const RotaryView& r, int p) {
    return r.neighbours ? (p >> 2) + (p & 3) * (r.rot / 8) : (p >> 3) + (p & 7) * (r.rot / 16);
}

__device__ __forceinline__ int axis_of(const RotaryView& r, int i) { return (r.axis[i / 16] >> (2 * (i % 16))) & 3; }

// `tt` tokens (blockIdx.x) x `ht` heads (blockIdx.y) a CTA.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_rotate(const __grid_constant__ RotaryView r, HeadsView x, HeadsView y,
                                                     int64_t n_tokens, int heads, int tt, int ht, Kinds kinds,
                                                     Divisor pairs) {
    extern __shared__ float2 cs[];  // [tt][rot / 2]
    const int64_t t0 = (int64_t)blockIdx.x * tt;
    const int nt = (int)min((int64_t)tt, n_tokens - t0);
    const int h0 = blockIdx.y * ht, nh = min(ht, heads - h0);
    const int half = r.rot / 2, total = nt * nh * (int)(kinds.turn.d + kinds.other.d);
    const Divisor per_token = divisor(nh);
    Unit<T> v[kUnits<T>];
    Where w[kUnits<T>];
#pragma unroll
    for (int k = 0; k < kUnits<T>; ++k) {
        const int i = threadIdx.x + k * kThreads;
        if (i >= total) continue;
        w[k] = where(i, nt, nh, per_token, kinds);
        const T* src = reinterpret_cast<const T*>(x.p) + (t0 + w[k].t()) * x.ts + (h0 + w[k].h()) * x.hs;
        if (w[k].kind() == 0) load_turn(v[k], src, w[k].u(), r);
        else load_plain(v[k], src + other_channel(r, w[k].u(), kinds.width), kinds.width);
    }
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = divide(i, pairs), p = i - t * half;
        cs[t * half + cs_at(r, p)] = turn_of(r, p, r.pos[axis_of(r, p) * r.pos_stride + t0 + t]);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kUnits<T>; ++k) {
        const int i = threadIdx.x + k * kThreads;
        if (i >= total) continue;
        T* dst = reinterpret_cast<T*>(y.p) + (t0 + w[k].t()) * y.ts + (h0 + w[k].h()) * y.hs;
        if (w[k].kind() == 0) store_turn(v[k], dst, w[k].u(), r, cs + w[k].t() * half);
        else store_plain(v[k], dst + other_channel(r, w[k].u(), kinds.width), kinds.width);
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
                                                        Kinds kinds, Divisor pairs) {
    extern __shared__ float2 cs[];                                // [tt][rot / 2]
    const int half = r.rot / 2;
    int64_t* row = reinterpret_cast<int64_t*>(cs + tt * half);    // [tt] element of head 0 in the pools, or -1
    int* slot = reinterpret_cast<int*>(row + tt);                 // [tt]
    int* cu = slot + tt;                                          // [batch + 1]
    const int t0 = blockIdx.x * tt, nt = min(tt, a.total - t0);
    const int h0 = blockIdx.y * ht, nh = min(ht, a.c.kv_heads - h0);
    const int total = nt * nh * (int)(kinds.turn.d + kinds.other.d + kinds.value.d);
    const Divisor per_token = divisor(nh);
    const auto load = [&](Unit<In>& v, const Where& w) {
        const HeadsView& x = w.kind() == 2 ? a.v : a.k;
        const In* src = reinterpret_cast<const In*>(x.p) + (int64_t)(t0 + w.t()) * x.ts + (h0 + w.h()) * x.hs;
        if (w.kind() == 0) load_turn(v, src, w.u(), r);
        else if (w.kind() == 1) load_plain(v, src + other_channel(r, w.u(), kinds.width), kinds.width);
        else load_plain(v, src + 16 * w.u(), 16);
    };
    const auto store = [&](const Unit<In>& v, const Where& w) {
        const int64_t at = row[w.t()];
        if (at < 0) return;
        Out* dst = reinterpret_cast<Out*>(w.kind() == 2 ? a.c.v : a.c.k) + at + (int64_t)(h0 + w.h()) * PAGE * dim;
        if (w.kind() == 0) store_turn(v, dst, w.u(), r, cs + w.t() * half);
        else if (w.kind() == 1) store_plain(v, dst + other_channel(r, w.u(), kinds.width), kinds.width);
        else store_plain(v, dst + 16 * w.u(), 16);
    };
    // Where token threadIdx.x goes if it belongs to sequence b.
    const auto locate = [&](int b) {
        const int t = t0 + threadIdx.x;
        int64_t at = -1;
        int s = 0;
        const Placed p = place(a, cu, b);
        if (p.m > 0 && t >= p.row0 && t < p.row0 + p.m) {
            s = p.slot0 + (t - p.row0);
            const int page = kv_page(a.c, b, s / PAGE);
            if (page >= 0) at = ((int64_t)page * a.c.kv_heads * PAGE + s % PAGE) * dim;
        }
        row[threadIdx.x] = at;
        slot[threadIdx.x] = s;
    };
    const auto turns = [&] {
        for (int i = threadIdx.x; i < nt * half; i += kThreads) {
            const int t = divide(i, pairs), p = i - t * half;
            if (row[t] >= 0)
                cs[t * half + cs_at(r, p)] = turn_of(r, p, r.pos ? r.pos[axis_of(r, p) * r.pos_stride + t0 + t] : slot[t]);
        }
    };
    static_assert(kMaxTokens <= kThreads, "a thread looks up one token");
    Unit<In> v[kUnits<In>];
    Where w[kUnits<In>];
#pragma unroll
    for (int k = 0; k < kUnits<In>; ++k) {
        const int i = threadIdx.x + k * kThreads;
        if (i >= total) continue;
        w[k] = where(i, nt, nh, per_token, kinds);
        load(v[k], w[k]);
    }
    bool ordered = true;
    for (int i = threadIdx.x; i <= a.c.batch; i += kThreads) {
        cu[i] = a.cu[i];
        if (i < a.c.batch) ordered = ordered && cu[i] <= a.cu[i + 1];
    }
    ordered = __syncthreads_and(ordered);
    if (ordered) {
        if (threadIdx.x < nt) {
            int lo = 0, hi = a.c.batch;  // the last b with cu[b] <= t: no other sequence has the row
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (cu[mid] <= t0 + (int)threadIdx.x) lo = mid;
                else hi = mid;
            }
            locate(lo);
        }
        __syncthreads();
        turns();
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kUnits<In>; ++k)
            if (threadIdx.x + k * kThreads < total) store(v[k], w[k]);
    } else {
        // Bounds out of order: each sequence whose own bounds are in order gets its rows, and
        // a row may belong to several of them.
        for (int b = 0; b < a.c.batch; ++b) {
            if (max(cu[b], t0) >= min(cu[b + 1], t0 + nt)) continue;
            __syncthreads();  // the sequence before has been written
            if (threadIdx.x < nt) locate(b);
            __syncthreads();
            turns();
            __syncthreads();
#pragma unroll 1
            for (int i = threadIdx.x; i < total; i += kThreads) {
                const Where at = where(i, nt, nh, per_token, kinds);
                Unit<In> x;
                load(x, at);
                store(x, at);
            }
        }
    }
    if (a.start && blockIdx.x == 0 && blockIdx.y == 0) count_tokens(a, cu, threadIdx.x, kThreads);
}

// The counts when they are also the start: after every CTA has read them.
__global__ void k_kv_count(const __grid_constant__ KvAppend a) {
    count_tokens(a, a.cu, threadIdx.x, blockDim.x);
}

// Units of a row of dim channels, `others` of which are only moved, and of its values.
Kinds kinds_of(const RotaryView& r, int others, int values) {
    const int width = r.offset % 16 == 0 && others % 16 == 0 ? 16 : 8;
    return {divisor(rot_units(r.rot, r.neighbours)), divisor(others / width), divisor(values / 16), width};
}

// Tokens and heads of a CTA: as many as its threads have units for, or fewer
// (down to one unit a thread) while the CTAs would not fill the SMs twice.
void tile_rows(int64_t tokens, int heads, int units, int half, int most, int& tt, int& ht) {
    const int64_t want = 2 * device_sm_count();
    int per = most * kThreads;
    while (per > kThreads && tokens * heads * units / per < want) per /= 2;
    const int parts = (heads * units + per - 1) / per;  // of a token's heads
    ht = std::min((heads + parts - 1) / parts, per / units);
    tt = ht < heads ? 1 : per / (units * heads);
    tt = (int)std::min<int64_t>(std::min(tt, kMaxTokens), tokens);
    if (half > 0) tt = std::min(tt, 4096 / half);  // 32 KB of (cos, sin)
}

template <typename T>
cudaError_t rotate_as(const RotaryView& r, const HeadsView& x, const HeadsView& y, int64_t n_tokens, int heads, int dim,
                      cudaStream_t st) {
    const bool in_place = x.p == y.p;  // the other channels are there already
    const Kinds kinds = kinds_of(r, in_place ? 0 : dim - r.rot, 0);
    const int units = kinds.turn.d + kinds.other.d;
    int tt, ht;
    tile_rows(n_tokens, heads, units, r.rot / 2, kUnits<T>, tt, ht);
    const dim3 grid((unsigned)((n_tokens + tt - 1) / tt), (heads + ht - 1) / ht);
    k_rotate<T><<<grid, kThreads, (size_t)tt * (r.rot / 2) * sizeof(float2), st>>>(r, x, y, n_tokens, heads, tt, ht,
                                                                                   kinds, divisor(r.rot / 2));
    return cudaGetLastError();
}

template <typename In, typename Out>
cudaError_t append_as(const KvAppend& a, const RotaryView& r, int dim, cudaStream_t st) {
    if (a.total > 0) {
        const Kinds kinds = kinds_of(r, dim - r.rot, dim);
        int tt, ht;
        const int units = kinds.turn.d + kinds.other.d + kinds.value.d;
        tile_rows(a.total, a.c.kv_heads, units, r.rot / 2, kUnits<In>, tt, ht);
        const dim3 grid((a.total + tt - 1) / tt, (a.c.kv_heads + ht - 1) / ht);
        const size_t smem = (size_t)tt * (r.rot / 2 * sizeof(float2) + sizeof(int64_t) + sizeof(int)) +
                            (size_t)(a.c.batch + 1) * sizeof(int);
        k_kv_append<In, Out><<<grid, kThreads, smem, st>>>(a, r, dim, tt, ht, kinds, divisor(r.rot / 2));
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
