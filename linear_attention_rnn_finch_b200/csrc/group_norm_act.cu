// Group norm over channels-last tensors with an activation, forward and backward (sm_100a).
//
// x [N][L][C]; for each n and group of per = C / groups channels, over its L positions:
//     h = (x - mean) / sqrt(var + eps),   z = h gamma + beta,   y = act(z), or z act(gate).
// Backward, with dz = dy act'(z) (or dy act(gate), and then dgate = dy z act'(gate)):
//     dbeta = sum dz,   dgamma = sum dz h   (over n and positions),
//     dh = dz gamma,    dx = (dh - mean(dh) - h mean(dh h)) / sqrt(var + eps).
// Every pass is bound by memory; sums are fp32, the squares' of differences from the mean (over
// positions from a value of the data), so that a mean far from zero costs the variance no digits.
//
// One position (L = 1, each token's heads): a group is a contiguous run of `per` values held
// in the registers of a few adjacent lanes, read once and written once in one launch.  A set of
// lanes keeps its group and walks rows, the next row's loads issued before the present one is
// worked on, with gamma and beta in registers.
//
// Several positions: a thread owns 8 adjacent channels (one, where the groups do not allow it)
// and walks positions, so that accesses are whole rows whatever the group's width.  A CTA takes
// whole groups (or a part of one wide group) over a split of the positions and leaves one
// (mean, sum of squares about it) a group; the next launch's CTAs join those of their groups
// themselves.  Two launches forward, three backward.
#include <type_traits>

#include "common.cuh"
#include "dependent_launch.cuh"
#include "group_norm_act.h"

namespace goldwkv {

namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ element access
template <int V>
__device__ __forceinline__ void load(const float* p, float (&v)[V]) {
    if (V == 1) {
        v[0] = p[0];
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 a = *reinterpret_cast<const float4*>(p + i);
            v[i] = a.x; v[i + 1] = a.y; v[i + 2] = a.z; v[i + 3] = a.w;
        }
    }
}
template <int V>
__device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[V]) {
    if (V == 1) {
        v[0] = __bfloat162float(p[0]);
    } else {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}
template <int V>
__device__ __forceinline__ void store(float* p, const float (&v)[V]) {
    if (V == 1) {
        p[0] = v[0];
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}
template <int V>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[V]) {
    if (V == 1) {
        p[0] = __float2bfloat16_rn(v[0]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&t);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// sigmoid: the approximate exponential and reciprocal where the result is rounded to bf16
// (relative error about 2^-21), the accurate ones for fp32.  The gradient over rows issues 40
// to 70 instructions a value, which bound it before memory did.
template <typename IO> __device__ __forceinline__ float sigmoid(float x);
template <> __device__ __forceinline__ float sigmoid<float>(float x) { return 1.f / (1.f + expf(-x)); }
template <> __device__ __forceinline__ float sigmoid<__nv_bfloat16>(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}
template <typename IO>
__device__ __forceinline__ float act(float x, bool silu) { return silu ? x * sigmoid<IO>(x) : x; }
// act(x) and act'(x)
template <typename IO>
__device__ __forceinline__ float2 act_grad(float x, bool silu) {
    if (!silu) return make_float2(x, 1.f);
    const float s = sigmoid<IO>(x), xs = x * s;
    return make_float2(xs, fmaf(xs, 1.f - s, s));
}

// sum over the `lanes` (a power of two) adjacent lanes of a group
__device__ __forceinline__ float lanes_sum(float x, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// What a lane loads, before conversion.
template <typename IO, int V> struct Raw;
template <> struct Raw<float, 8> { float4 a, b; };
template <> struct Raw<__nv_bfloat16, 8> { uint4 a; };
template <> struct Raw<float, 1> { float a; };
template <> struct Raw<__nv_bfloat16, 1> { __nv_bfloat16 a; };
template <typename IO, int V>
__device__ __forceinline__ Raw<IO, V> load_raw(const IO* p) { return *reinterpret_cast<const Raw<IO, V>*>(p); }
template <int V>
__device__ __forceinline__ void convert(const Raw<float, V>& r, float (&v)[V]) {
    const float* p = reinterpret_cast<const float*>(&r);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = p[i];
}
__device__ __forceinline__ void convert(const Raw<__nv_bfloat16, 1>& r, float (&v)[1]) { v[0] = __bfloat162float(r.a); }
__device__ __forceinline__ void convert(const Raw<__nv_bfloat16, 8>& r, float (&v)[8]) {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// ------------------------------------------------------------------ one position
// A group's `units` (of V values) lie on `lanes` adjacent lanes, U a lane (unit = lane +
// lanes * i), in registers.  U = 0: more than the registers hold, read again for each pass.
// Set s of lanes keeps group s % groups and takes rows s / groups, + streams, ...
struct RowShape {
    long rows;       // N
    int C, groups, per, units, lanes;
    long streams;
};
struct RowSet {
    bool in;
    int g, l;
    long n;          // first row
};
__device__ __forceinline__ RowSet row_set(const RowShape& s) {
    RowSet r;
    const unsigned set = blockIdx.x * (kThreads / s.lanes) + threadIdx.x / s.lanes;
    r.l = threadIdx.x & (s.lanes - 1);
    r.n = set / (unsigned)s.groups;
    r.g = (int)(set - (unsigned)r.n * s.groups);
    r.in = r.n < s.streams;
    if (!r.in) r.n = r.g = 0;
    return r;
}

template <typename IO, int V, int U, bool kGate, bool kSilu>
__global__ void __launch_bounds__(kThreads)
group_norm_rows_kernel(const IO* __restrict__ x, const IO* __restrict__ gate,
                       const float* __restrict__ gamma, const float* __restrict__ beta, float eps,
                       IO* __restrict__ y, RowShape s) {
    const RowSet set = row_set(s);
    const int l = set.l, c0 = set.g * s.per;
    const float inv_n = 1.f / (float)s.per;
    // every lane of a warp runs the same number of rows: the shuffles need them all
    const long turns = (s.rows + s.streams - 1) / s.streams;
    if (U > 0) {
        constexpr int K = U > 0 ? U : 1;
        float ga[K][V], be[K][V];
        Raw<IO, V> rx[K], rg[K];
        bool has[K];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int u = l + s.lanes * i;
            has[i] = set.in && u < s.units;
            if (has[i]) {
                load<V>(gamma + c0 + u * V, ga[i]);
                load<V>(beta + c0 + u * V, be[i]);
            }
        }
        const int apart = s.lanes * V;
        const size_t stride = (size_t)s.streams * s.C;
        auto fetch = [&](size_t o) {
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (has[i]) {
                    rx[i] = load_raw<IO, V>(x + o + i * apart);
                    if (kGate) rg[i] = load_raw<IO, V>(gate + o + i * apart);
                }
        };
        size_t o = (size_t)set.n * s.C + c0 + l * V;
        int left = (int)((s.rows - set.n + s.streams - 1) / s.streams);   // rows of this set
        fetch(o);
        for (int it = 0; it < turns; ++it, --left, o += stride) {
            const bool row = left > 0;
            float v[K][V], gt[K][V], sum = 0.f;
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (has[i] && row) {
                    convert(rx[i], v[i]);
                    if (kGate) convert(rg[i], gt[i]);
#pragma unroll
                    for (int e = 0; e < V; ++e) sum += v[i][e];
                }
            if (left > 1) fetch(o + stride);
            const float mean = lanes_sum(sum, s.lanes) * inv_n;
            float sq = 0.f;
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (has[i] && row) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        v[i][e] -= mean;
                        sq = fmaf(v[i][e], v[i][e], sq);
                    }
                }
            const float r = rsqrtf(lanes_sum(sq, s.lanes) * inv_n + eps);
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (has[i] && row) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float z = fmaf(v[i][e] * r, ga[i][e], be[i][e]);
                        v[i][e] = kGate ? z * act<IO>(gt[i][e], kSilu) : act<IO>(z, kSilu);
                    }
                    store<V>(y + o + i * apart, v[i]);
                }
        }
    } else {
        for (long it = 0; it < turns; ++it) {
            const long n = set.n + it * s.streams;
            const int units = set.in && n < s.rows ? s.units : 0;
            const size_t base = (size_t)n * s.C + c0;
            float v[V], gt[V], sum = 0.f, sq = 0.f;
            for (int u = l; u < units; u += s.lanes) {
                load<V>(x + base + (size_t)u * V, v);
#pragma unroll
                for (int e = 0; e < V; ++e) sum += v[e];
            }
            const float mean = lanes_sum(sum, s.lanes) * inv_n;
            for (int u = l; u < units; u += s.lanes) {
                load<V>(x + base + (size_t)u * V, v);
#pragma unroll
                for (int e = 0; e < V; ++e) sq = fmaf(v[e] - mean, v[e] - mean, sq);
            }
            const float r = rsqrtf(lanes_sum(sq, s.lanes) * inv_n + eps);
            for (int u = l; u < units; u += s.lanes) {
                float ga[V], be[V];
                load<V>(x + base + (size_t)u * V, v);
                if (kGate) load<V>(gate + base + (size_t)u * V, gt);
                load<V>(gamma + c0 + u * V, ga);
                load<V>(beta + c0 + u * V, be);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float z = fmaf((v[e] - mean) * r, ga[e], be[e]);
                    v[e] = kGate ? z * act<IO>(gt[e], kSilu) : act<IO>(z, kSilu);
                }
                store<V>(y + base + (size_t)u * V, v);
            }
        }
    }
}

// dz and, with a gate, dgate (in gt) of one value: h the normalised value, d the output's gradient.
template <typename IO, bool kGate>
__device__ __forceinline__ float value_grad(float h, float ga, float be, float d, float& gt, bool silu) {
    const float z = fmaf(h, ga, be);
    if (!kGate) return d * act_grad<IO>(z, silu).y;
    const float2 a = act_grad<IO>(gt, silu);
    gt = d * z * a.y;
    return d * a.x;
}

// Backward over rows: a set's channels' dgamma and dbeta sums stay in registers (U > 0) and leave
// as one row of partial sums a stream.  U = 0 (wide groups): the sums are kept in the partial
// row itself, which no one else touches.
template <typename IO, int V, int U, bool kGate, bool kSilu>
__global__ void __launch_bounds__(kThreads, U == 1 ? 3 : 1)
group_norm_rows_bwd_kernel(const IO* __restrict__ x, const IO* __restrict__ gate,
                           const float* __restrict__ gamma, const float* __restrict__ beta,
                           float eps, const IO* __restrict__ dy, IO* __restrict__ dx,
                           IO* __restrict__ dgate, float* __restrict__ part, RowShape s) {
    const RowSet set = row_set(s);
    const int l = set.l, c0 = set.g * s.per;
    const float inv_n = 1.f / (float)s.per;
    // partial rows: dgamma then dbeta, [streams][2][C]
    float* pg = part + (size_t)set.n * 2 * s.C + c0;
    float* pb = pg + s.C;
    const long turns = (s.rows + s.streams - 1) / s.streams;
    if (U > 0) {
        constexpr int K = U > 0 ? U : 1;
        float dga[K][V], dbe[K][V], ga[K][V], be[K][V];
        Raw<IO, V> rx[K], rd[K], rg[K];
        bool has[K];
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int u = l + s.lanes * i;
            has[i] = set.in && u < s.units;
#pragma unroll
            for (int e = 0; e < V; ++e) dga[i][e] = dbe[i][e] = 0.f;
            if (has[i]) {
                load<V>(gamma + c0 + u * V, ga[i]);
                load<V>(beta + c0 + u * V, be[i]);
            }
        }
        const int apart = s.lanes * V;
        const size_t stride = (size_t)s.streams * s.C;
        auto fetch = [&](size_t o) {
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (has[i]) {
                    rx[i] = load_raw<IO, V>(x + o + i * apart);
                    rd[i] = load_raw<IO, V>(dy + o + i * apart);
                    if (kGate) rg[i] = load_raw<IO, V>(gate + o + i * apart);
                }
        };
        size_t o = (size_t)set.n * s.C + c0 + l * V;
        int left = (int)((s.rows - set.n + s.streams - 1) / s.streams);   // rows of this set
        fetch(o);
        for (int it = 0; it < turns; ++it, --left, o += stride) {
            const bool row = left > 0;
            float v[K][V], d[K][V], gt[K][V], sum = 0.f;
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (has[i] && row) {
                    convert(rx[i], v[i]);
                    convert(rd[i], d[i]);
                    if (kGate) convert(rg[i], gt[i]);
#pragma unroll
                    for (int e = 0; e < V; ++e) sum += v[i][e];
                }
            if (left > 1) fetch(o + stride);
            const float mean = lanes_sum(sum, s.lanes) * inv_n;
            float sq = 0.f;
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (has[i] && row) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        v[i][e] -= mean;
                        sq = fmaf(v[i][e], v[i][e], sq);
                    }
                }
            const float r = rsqrtf(lanes_sum(sq, s.lanes) * inv_n + eps);
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (has[i] && row) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float h = v[i][e] * r;
                        const float dz = value_grad<IO, kGate>(h, ga[i][e], be[i][e], d[i][e], gt[i][e], kSilu);
                        dga[i][e] = fmaf(dz, h, dga[i][e]);
                        dbe[i][e] += dz;
                        const float dh = dz * ga[i][e];
                        s1 += dh;
                        s2 = fmaf(dh, h, s2);
                        d[i][e] = dh;
                        v[i][e] = h;
                    }
                    if (kGate) store<V>(dgate + o + i * apart, gt[i]);
                }
            s1 = lanes_sum(s1, s.lanes) * inv_n;
            s2 = lanes_sum(s2, s.lanes) * inv_n;
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (has[i] && row) {
#pragma unroll
                    for (int e = 0; e < V; ++e) d[i][e] = r * (d[i][e] - s1 - v[i][e] * s2);
                    store<V>(dx + o + i * apart, d[i]);
                }
        }
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (has[i]) {
                store<V>(pg + (l + s.lanes * i) * V, dga[i]);
                store<V>(pb + (l + s.lanes * i) * V, dbe[i]);
            }
    } else {
        float zero[V];
#pragma unroll
        for (int e = 0; e < V; ++e) zero[e] = 0.f;
        if (set.in)
            for (int u = l; u < s.units; u += s.lanes) {
                store<V>(pg + u * V, zero);
                store<V>(pb + u * V, zero);
            }
        for (long it = 0; it < turns; ++it) {
            const long n = set.n + it * s.streams;
            const int units = set.in && n < s.rows ? s.units : 0;
            const size_t base = (size_t)n * s.C + c0;
            float v[V], d[V], gt[V], gg[V], bb[V];
            float sum = 0.f, sq = 0.f, s1 = 0.f, s2 = 0.f;
            for (int u = l; u < units; u += s.lanes) {
                load<V>(x + base + (size_t)u * V, v);
#pragma unroll
                for (int e = 0; e < V; ++e) sum += v[e];
            }
            const float mean = lanes_sum(sum, s.lanes) * inv_n;
            for (int u = l; u < units; u += s.lanes) {
                load<V>(x + base + (size_t)u * V, v);
#pragma unroll
                for (int e = 0; e < V; ++e) sq = fmaf(v[e] - mean, v[e] - mean, sq);
            }
            const float r = rsqrtf(lanes_sum(sq, s.lanes) * inv_n + eps);
            for (int pass = 0; pass < 2; ++pass) {
                for (int u = l; u < units; u += s.lanes) {
                    load<V>(x + base + (size_t)u * V, v);
                    load<V>(dy + base + (size_t)u * V, d);
                    if (kGate) load<V>(gate + base + (size_t)u * V, gt);
                    load<V>(gamma + c0 + u * V, gg);
                    load<V>(beta + c0 + u * V, bb);
                    float a1[V], a2[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float h = (v[e] - mean) * r;
                        const float dz = value_grad<IO, kGate>(h, gg[e], bb[e], d[e], gt[e], kSilu);
                        const float dh = dz * gg[e];
                        a1[e] = dz * h;
                        a2[e] = dz;
                        if (pass == 0) {
                            s1 += dh;
                            s2 = fmaf(dh, h, s2);
                        } else {
                            d[e] = r * (dh - s1 - h * s2);
                        }
                    }
                    if (pass == 0) {
                        float o1[V], o2[V];
                        load<V>(pg + u * V, o1);
                        load<V>(pb + u * V, o2);
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            o1[e] += a1[e];
                            o2[e] += a2[e];
                        }
                        store<V>(pg + u * V, o1);
                        store<V>(pb + u * V, o2);
                        if (kGate) store<V>(dgate + base + (size_t)u * V, gt);
                    } else {
                        store<V>(dx + base + (size_t)u * V, d);
                    }
                }
                if (pass == 0) {
                    s1 = lanes_sum(s1, s.lanes) * inv_n;
                    s2 = lanes_sum(s2, s.lanes) * inv_n;
                }
            }
        }
    }
}

// Groups of 8 kL channels, kL a power of two: every lane of a set holds one vector, so that
// nothing is left to test in the loop (a set whose turns end leaves; the shuffles are among a
// set's lanes only), and the sums' steps are known.  The gradient issues 49 instructions a value
// instead of 57 and takes 32768 rows of 2048 from 156 to 136 us, the norm itself from 76 to 69.
template <int kL>
__device__ __forceinline__ float set_sum(float x, unsigned lanes) {
#pragma unroll
    for (int o = kL >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(lanes, x, o);
    return x;
}
template <int kL>
__device__ __forceinline__ unsigned set_lanes() {
    return kL == 32 ? 0xffffffffu : ((1u << (kL & 31)) - 1) << (threadIdx.x & 31 & ~(kL - 1));
}

template <typename IO, int kL, bool kGate, bool kSilu>
__global__ void __launch_bounds__(kThreads)
group_norm_full_rows_kernel(const IO* __restrict__ x, const IO* __restrict__ gate,
                            const float* __restrict__ gamma, const float* __restrict__ beta, float eps,
                            IO* __restrict__ y, RowShape s) {
    constexpr int V = 8;
    const RowSet set = row_set(s);
    if (!set.in) return;
    const unsigned lanes = set_lanes<kL>();
    const int c0 = set.g * s.per + set.l * V;
    constexpr float inv_n = 1.f / (kL * V);
    float ga[V], be[V];
    load<V>(gamma + c0, ga);
    load<V>(beta + c0, be);
    const size_t stride = (size_t)s.streams * s.C;
    size_t o = (size_t)set.n * s.C + c0;
    int left = (int)((s.rows - set.n + s.streams - 1) / s.streams);   // rows of this set
    Raw<IO, V> rx = load_raw<IO, V>(x + o), rg;
    if (kGate) rg = load_raw<IO, V>(gate + o);
    for (; left > 0; --left, o += stride) {
        float v[V], gt[V], sum = 0.f, sq = 0.f;
        convert(rx, v);
        if (kGate) convert(rg, gt);
        if (left > 1) {
            rx = load_raw<IO, V>(x + o + stride);
            if (kGate) rg = load_raw<IO, V>(gate + o + stride);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) sum += v[e];
        const float mean = set_sum<kL>(sum, lanes) * inv_n;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            v[e] -= mean;
            sq = fmaf(v[e], v[e], sq);
        }
        const float r = rsqrtf(set_sum<kL>(sq, lanes) * inv_n + eps);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float z = fmaf(v[e] * r, ga[e], be[e]);
            v[e] = kGate ? z * act<IO>(gt[e], kSilu) : act<IO>(z, kSilu);
        }
        store<V>(y + o, v);
    }
}

template <typename IO, int kL, bool kGate, bool kSilu>
__global__ void __launch_bounds__(kThreads, sizeof(IO) == 4 ? 2 : 3)
group_norm_full_rows_bwd_kernel(const IO* __restrict__ x, const IO* __restrict__ gate,
                                const float* __restrict__ gamma, const float* __restrict__ beta,
                                float eps, const IO* __restrict__ dy, IO* __restrict__ dx,
                                IO* __restrict__ dgate, float* __restrict__ part, RowShape s) {
    constexpr int V = 8;
    const RowSet set = row_set(s);
    if (!set.in) return;
    const unsigned lanes = set_lanes<kL>();
    const int c0 = set.g * s.per + set.l * V;
    constexpr float inv_n = 1.f / (kL * V);
    float ga[V], be[V], dga[V], dbe[V];
    load<V>(gamma + c0, ga);
    load<V>(beta + c0, be);
#pragma unroll
    for (int e = 0; e < V; ++e) dga[e] = dbe[e] = 0.f;
    const size_t stride = (size_t)s.streams * s.C;
    size_t o = (size_t)set.n * s.C + c0;
    int left = (int)((s.rows - set.n + s.streams - 1) / s.streams);
    Raw<IO, V> rx = load_raw<IO, V>(x + o), rd = load_raw<IO, V>(dy + o), rg;
    if (kGate) rg = load_raw<IO, V>(gate + o);
    for (; left > 0; --left, o += stride) {
        float v[V], d[V], gt[V], sum = 0.f, sq = 0.f, s1 = 0.f, s2 = 0.f;
        convert(rx, v);
        convert(rd, d);
        if (kGate) convert(rg, gt);
        if (left > 1) {
            rx = load_raw<IO, V>(x + o + stride);
            rd = load_raw<IO, V>(dy + o + stride);
            if (kGate) rg = load_raw<IO, V>(gate + o + stride);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) sum += v[e];
        const float mean = set_sum<kL>(sum, lanes) * inv_n;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            v[e] -= mean;
            sq = fmaf(v[e], v[e], sq);
        }
        const float r = rsqrtf(set_sum<kL>(sq, lanes) * inv_n + eps);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            v[e] *= r;
            const float dz = value_grad<IO, kGate>(v[e], ga[e], be[e], d[e], gt[e], kSilu);
            dga[e] = fmaf(dz, v[e], dga[e]);
            dbe[e] += dz;
            d[e] = dz * ga[e];
            s1 += d[e];
            s2 = fmaf(d[e], v[e], s2);
        }
        if (kGate) store<V>(dgate + o, gt);
        s1 = set_sum<kL>(s1, lanes) * inv_n * r;
        s2 = set_sum<kL>(s2, lanes) * inv_n * r;
#pragma unroll
        for (int e = 0; e < V; ++e) d[e] = fmaf(-v[e], s2, fmaf(d[e], r, -s1));
        store<V>(dx + o, d);
    }
    // partial rows: dgamma then dbeta, [streams][2][C]
    float* pg = part + (size_t)set.n * 2 * s.C + c0;
    store<V>(pg, dga);
    store<V>(pg + s.C, dbe);
}

// dgamma[c], dbeta[c] = the sums of `rows` partial rows ([rows][2][C]), in a fixed order: 32
// columns a CTA, kWarps row lanes each, joined through shared memory.  A lane takes eight rows at a
// time, all their loads in flight, and carries on what rounding takes from its sum (Kahan's): with
// a row for each n it adds up tens of thousands, which plainly leave 3e-6 of 800,000 values of one
// sign.
template <int kWarps>
__device__ __forceinline__ void sum_params(const float* __restrict__ part, long rows, int C, int cta,
                                           float* __restrict__ dgamma, float* __restrict__ dbeta) {
    __shared__ float red[kWarps][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = cta * 32 + lane;   // column of the 2 C
    float sum = 0.f, lost = 0.f;
    if (i < 2 * C)
        for (long r = warp; r < rows; r += 8 * kWarps) {
            float v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = r + u * kWarps < rows ? part[(size_t)(r + u * kWarps) * 2 * C + i] : 0.f;
            const float add = (((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]))) - lost;
            const float next = sum + add;
            lost = isfinite(next) ? (next - sum) - add : 0.f;   // an infinite sum stays one
            sum = next;
        }
    red[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && i < 2 * C) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) t += red[w][lane];
        if (i < C) dgamma[i] = t;
        else dbeta[i - C] = t;
    }
}
constexpr int kParamWarps = 32;   // few rows a warp: the loads' latency is all that counts
__global__ void __launch_bounds__(32 * kParamWarps)
group_norm_param_kernel(const float* __restrict__ part, long rows, int C, float* __restrict__ dgamma,
                        float* __restrict__ dbeta) {
    previous_ended();
    sum_params<kParamWarps>(behind(part), rows, C, blockIdx.x, dgamma, dbeta);
}

// ------------------------------------------------------------------ several positions
// A CTA covers positions [l0, l1) of one n and a tile of at most kThreads channel vectors: whole
// groups, or one of the `parts` of a group wider than that.  Thread = (row lane, vector): row
// lane i walks positions l0 + i, l0 + i + lanes, ...
struct Tiling {
    long N, L;
    int C, groups, per;
    int V;           // channels of a vector
    int width;       // channels of a tile
    int parts;       // tiles of a group (1: a tile holds width / per whole groups)
    int tiles;       // channel tiles
    int vecs, lanes; // vectors of a tile, position lanes
    int splits;      // splits of the positions
    long span;       // positions of a split
};
struct Place {
    long n;
    int split, tile;
    int c_begin, c_end;  // the tile's channels
    int g_begin, g_count;
    int c0;              // first channel of the thread's vector
    long first, count;   // the split's positions
    long l0, l1;         // the thread's: l0, l0 + lanes, ... < l1
    bool in;
};
__device__ __forceinline__ Place place(const Tiling& t) {
    Place p;
    const unsigned i = blockIdx.x, ns = i / (unsigned)t.tiles;
    p.tile = (int)(i - ns * t.tiles);
    p.n = ns / (unsigned)t.splits;
    p.split = (int)(ns - (unsigned)p.n * t.splits);
    if (t.parts == 1) {
        p.c_begin = p.tile * t.width;
        p.c_end = min(t.C, p.c_begin + t.width);
        p.g_begin = p.c_begin / t.per;
        p.g_count = (p.c_end - p.c_begin) / t.per;
    } else {
        p.g_begin = p.tile / t.parts;
        p.g_count = 1;
        p.c_begin = p.g_begin * t.per + (p.tile - p.g_begin * t.parts) * t.width;
        p.c_end = min((p.g_begin + 1) * t.per, p.c_begin + t.width);
    }
    const int lane = threadIdx.x / t.vecs;
    p.c0 = p.c_begin + (threadIdx.x - lane * t.vecs) * t.V;
    p.first = p.split * t.span;
    p.count = min(t.L, p.first + t.span) - p.first;
    p.l0 = p.first + lane;
    p.l1 = p.first + p.count;
    p.in = lane < t.lanes && p.c0 < p.c_end;
    return p;
}
// Partial sums of group g of n: [n][group][split][part].
__device__ __forceinline__ size_t partial(const Tiling& t, long n, int g) {
    return ((size_t)n * t.groups + g) * t.splits * t.parts;
}
// Values behind partial i of a group.
__device__ __forceinline__ float partial_count(const Tiling& t, int i) {
    const int split = t.parts == 1 ? i : i / t.parts, part = i - split * t.parts;
    const int channels = t.parts == 1 ? t.per : min(t.width, t.per - part * t.width);
    return (float)(min(t.L, (split + 1) * t.span) - split * t.span) * (float)channels;
}

// f(e, group) for the V channels from c0 on.
template <int V, typename F>
__device__ __forceinline__ void each_group(const Tiling& t, int c0, F f) {
    int g = c0 / t.per, left = (g + 1) * t.per - c0;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        if (left == 0) {
            ++g;
            left = t.per;
        }
        --left;
        f(e, g);
    }
}
// Adjacent lanes that take a group together, so that a tile's groups are joined at once.
__device__ __forceinline__ int group_lanes(int groups) {
    int n = 32;
    while (n > 1 && n * groups > kThreads) n >>= 1;
    return n;
}
// (mean, 1 / sqrt(var + eps)) of the tile's groups into stat[].
__device__ __forceinline__ void join_stats(const float2* __restrict__ part, float eps, const Tiling& t,
                                           const Place& p, float2* stat) {
    const int lanes = group_lanes(p.g_count), lane = threadIdx.x & (lanes - 1), items = t.splits * t.parts;
    const float inv = 1.f / ((float)t.L * (float)t.per);
    // whole warps run the loop: the shuffles need them
    for (int g0 = 0; g0 < p.g_count; g0 += kThreads / lanes) {
        const int g = g0 + threadIdx.x / lanes;
        const float2* pp = part + partial(t, p.n, p.g_begin + (g < p.g_count ? g : 0));
        float s = 0.f, q = 0.f;
#pragma unroll 4
        for (int i = lane; i < items; i += lanes) s = fmaf(partial_count(t, i), pp[i].x, s);
        const float mean = lanes_sum(s, lanes) * inv;
#pragma unroll 4
        for (int i = lane; i < items; i += lanes) {
            const float2 r = pp[i];
            const float d = r.x - mean;
            q += fmaf(partial_count(t, i) * d, d, r.y);
        }
        q = lanes_sum(q, lanes) * inv;
        if (lane == 0 && g < p.g_count) stat[g] = make_float2(mean, rsqrtf(q + eps));
    }
    __syncthreads();
}

// A group's mean and sum of squares about it over a split.
template <typename IO, int V>
__global__ void __launch_bounds__(kThreads, 4)   // otherwise 80 registers, [8, 16384, 512] with a gate 111 us instead of 106
group_norm_stats_kernel(const IO* __restrict__ x, float2* __restrict__ part, Tiling t) {
    __shared__ float2 red[kThreads * V];   // (lane, channel): mean, M2
    const Place p = place(t);
    const IO* xp = x + ((size_t)p.n * t.L) * t.C + p.c0;
    // Runs of positions: the sums of differences from k and of their squares, joined to the mean
    // (k + lo) and the sum of squares so far (m2).  k is the thread's first value, then the mean so
    // far, so that what cancels in q - a m is at most kRun squares of an outlying first value, and
    // sums stay short; lo is what rounding took from the mean, which a mean far from zero would
    // otherwise lose at every join.  Between runs lo and m2 wait in the thread's places of red.
    // (One run however long: 2.3e-4 of the largest value in [300, 1000, 2048] behind a first position
    // 1000 deviations away; 103 us instead of 106 at [8, 16384, 512] with a gate.)
    constexpr int kRun = 64;
    if (p.in && p.l0 < p.l1) {
        float k[V];
        load<V>(xp + (size_t)p.l0 * t.C, k);
        float2* own = red + threadIdx.x * V;
        int before = 0;
        for (long l = p.l0; l < p.l1;) {
            const long end = min(p.l1, l + (long)kRun * t.lanes);
            float a[V], q[V];
            int cnt = 0;
#pragma unroll
            for (int e = 0; e < V; ++e) a[e] = q[e] = 0.f;
#pragma unroll 8
            for (; l < end; l += t.lanes) {
                float v[V];
                load<V>(xp + (size_t)l * t.C, v);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float d = v[e] - k[e];
                    a[e] += d;
                    q[e] = fmaf(d, d, q[e]);
                }
                ++cnt;
            }
            const float inv = 1.f / (float)cnt;
            const bool first = before == 0, last = l >= p.l1;
            const float share = first ? 1.f : (float)cnt / (float)(before + cnt), weight = (float)before * share;
            before += cnt;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float2 so = first ? make_float2(0.f, 0.f) : own[e];   // lo, m2
                const float m = a[e] * inv, g = m - so.x, off = fmaf(g, share, so.x), mean = k[e] + off;
                const float m2 = so.y + fmaf(weight * g, g, fmaxf(q[e] - a[e] * m, 0.f));
                own[e] = make_float2(last ? mean : off - (mean - k[e]), m2);
                k[e] = mean;
            }
        }
    }
    __syncthreads();
    // join the position lanes of each channel
    const int width = t.vecs * V, channels = p.c_end - p.c_begin;
    const int count = (int)p.count, each = count / t.lanes, more = count - each * t.lanes;
    const int have = min(count, t.lanes);   // lanes with a position: each or each + 1 of them
    for (int c = threadIdx.x; c < channels; c += kThreads) {
        float mean = 0.f, m2 = 0.f;
        for (int i = 0; i < have; ++i) mean += (float)(each + (i < more)) * red[i * width + c].x;
        mean /= (float)count;
        for (int i = 0; i < have; ++i) {
            const float2 r = red[i * width + c];
            const float d = r.x - mean;
            m2 += fmaf((float)(each + (i < more)) * d, d, r.y);
        }
        red[c] = make_float2(mean, m2);   // lane 0's place: no one else's of this channel
    }
    __syncthreads();
    // and the channels of each group
    const int gl = group_lanes(p.g_count), lane = threadIdx.x & (gl - 1), per = channels / p.g_count;
    for (int g0 = 0; g0 < p.g_count; g0 += kThreads / gl) {
        const int g = g0 + threadIdx.x / gl, own = g < p.g_count ? per : 0;
        float m = 0.f, q2 = 0.f;
        for (int c = lane; c < own; c += gl) m += red[g * per + c].x;
        m = lanes_sum(m, gl) / (float)per;
        for (int c = lane; c < own; c += gl) {
            const float2 r = red[g * per + c];
            const float d = r.x - m;
            q2 += fmaf((float)count * d, d, r.y);
        }
        q2 = lanes_sum(q2, gl);
        if (lane == 0 && own)
            part[partial(t, p.n, p.g_begin + g) + (size_t)p.split * t.parts + p.tile % t.parts] = make_float2(m, q2);
    }
}

template <typename IO, int V, bool kGate, bool kSilu>
__global__ void __launch_bounds__(kThreads)
group_norm_apply_kernel(const IO* __restrict__ x, const IO* __restrict__ gate,
                        const float* __restrict__ gamma, const float* __restrict__ beta, float eps,
                        const float2* __restrict__ part, IO* __restrict__ y, Tiling t) {
    __shared__ float2 stat[kThreads * V];
    const Place p = place(t);
    const size_t base = ((size_t)p.n * t.L) * t.C + p.c0;
    // A turn of positions' loads is issued before the turn ahead of it is worked on; the first needs
    // no statistics.  [8, 16384, 512] bf16 with a gate 138 -> 100 us, [2, 16384, 512] fp32 59 -> 48;
    // eight positions a turn 104 and 67.
    constexpr int kTurn = sizeof(IO) == 4 ? 2 : 4;
    Raw<IO, V> rx[kTurn], rg[kTurn];
    float mean[V], r[V], be[V];
    auto fetch = [&](long l) {
#pragma unroll
        for (int i = 0; i < kTurn; ++i, l += t.lanes)
            if (l < p.l1) {
                rx[i] = load_raw<IO, V>(x + base + (size_t)l * t.C);
                if (kGate) rg[i] = load_raw<IO, V>(gate + base + (size_t)l * t.C);
            }
    };
    if (p.in) {
        load<V>(gamma + p.c0, r);
        load<V>(beta + p.c0, be);
        fetch(p.l0);
    }
    previous_ended();
    join_stats(behind(part), eps, t, p, stat);
    if (!p.in) return;
    each_group<V>(t, p.c0, [&](int e, int g) {
        const float2 st = stat[g - p.g_begin];
        mean[e] = st.x;
        r[e] *= st.y;
    });
    for (long l = p.l0; l < p.l1; l += kTurn * t.lanes) {
        Raw<IO, V> cx[kTurn], cg[kTurn];
#pragma unroll
        for (int i = 0; i < kTurn; ++i) {
            cx[i] = rx[i];
            if (kGate) cg[i] = rg[i];
        }
        fetch(l + kTurn * t.lanes);
#pragma unroll
        for (int i = 0; i < kTurn; ++i) {
            const long at = l + i * t.lanes;
            if (at >= p.l1) break;
            float v[V], gt[V];
            convert(cx[i], v);
            if (kGate) convert(cg[i], gt);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float z = fmaf(v[e] - mean[e], r[e], be[e]);
                v[e] = kGate ? z * act<IO>(gt[e], kSilu) : act<IO>(z, kSilu);
            }
            store<V>(y + base + (size_t)at * t.C, v);
        }
    }
}

// Per channel of a split: sums of dz h and of dz ([n][split][2][C]); from them each group's sums
// of dh and dh h; dgate.  The statistics are handed on to the next launch.
template <typename IO, int V, bool kGate, bool kSilu>
__global__ void __launch_bounds__(kThreads)
group_norm_bwd_sums_kernel(const IO* __restrict__ x, const IO* __restrict__ gate,
                           const float* __restrict__ gamma, const float* __restrict__ beta, float eps,
                           const float2* __restrict__ part, const IO* __restrict__ dy,
                           IO* __restrict__ dgate, float2* __restrict__ stats,
                           float* __restrict__ rows, float2* __restrict__ sums, Tiling t) {
    __shared__ float2 red[kThreads * V];
    const Place p = place(t);
    float2* stat = red;
    const size_t base = ((size_t)p.n * t.L) * t.C + p.c0;
    // as in group_norm_apply_kernel: [8, 16384, 512] bf16 with a gate 296 -> 212 us for this launch
    // and the next, [2, 16384, 512] fp32 108 -> 90; with a position more a turn 241 and 123
    constexpr int kTurn = sizeof(IO) == 4 ? 1 : 2;
    Raw<IO, V> rx[kTurn], rd[kTurn], rg[kTurn];
    float mean[V], r[V], ga[V], be[V], sg[V], sb[V];
    auto fetch = [&](long l) {
#pragma unroll
        for (int i = 0; i < kTurn; ++i, l += t.lanes)
            if (l < p.l1) {
                const size_t o = base + (size_t)l * t.C;
                rx[i] = load_raw<IO, V>(x + o);
                rd[i] = load_raw<IO, V>(dy + o);
                if (kGate) rg[i] = load_raw<IO, V>(gate + o);
            }
    };
    if (p.in) {
        load<V>(gamma + p.c0, ga);
        load<V>(beta + p.c0, be);
        fetch(p.l0);
    }
    previous_ended();
    join_stats(behind(part), eps, t, p, stat);
    if (p.split == 0 && p.tile % t.parts == 0)
        for (int g = threadIdx.x; g < p.g_count; g += kThreads) stats[p.n * t.groups + p.g_begin + g] = stat[g];
#pragma unroll
    for (int e = 0; e < V; ++e) sg[e] = sb[e] = 0.f;
    if (p.in) {
        each_group<V>(t, p.c0, [&](int e, int g) {
            const float2 st = stat[g - p.g_begin];
            mean[e] = st.x;
            r[e] = st.y;
        });
        for (long l = p.l0; l < p.l1; l += kTurn * t.lanes) {
            Raw<IO, V> cx[kTurn], cd[kTurn], cg[kTurn];
#pragma unroll
            for (int i = 0; i < kTurn; ++i) {
                cx[i] = rx[i];
                cd[i] = rd[i];
                if (kGate) cg[i] = rg[i];
            }
            fetch(l + kTurn * t.lanes);
#pragma unroll
            for (int i = 0; i < kTurn; ++i) {
                const long at = l + i * t.lanes;
                if (at >= p.l1) break;
                float v[V], d[V], gt[V];
                convert(cx[i], v);
                convert(cd[i], d);
                if (kGate) convert(cg[i], gt);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float h = (v[e] - mean[e]) * r[e];
                    const float dz = value_grad<IO, kGate>(h, ga[e], be[e], d[e], gt[e], kSilu);
                    sg[e] = fmaf(dz, h, sg[e]);
                    sb[e] += dz;
                }
                if (kGate) store<V>(dgate + base + (size_t)at * t.C, gt);
            }
        }
    }
    __syncthreads();   // stat is read
#pragma unroll
    for (int e = 0; e < V; ++e) red[threadIdx.x * V + e] = make_float2(sg[e], sb[e]);
    __syncthreads();
    const int width = t.vecs * V, channels = p.c_end - p.c_begin;
    float* row = rows + ((size_t)p.n * t.splits + p.split) * 2 * t.C + p.c_begin;
    for (int c = threadIdx.x; c < channels; c += kThreads) {
        float a = 0.f, b = 0.f;
        for (int i = 0; i < t.lanes; ++i) {
            a += red[i * width + c].x;
            b += red[i * width + c].y;
        }
        row[c] = a;
        row[t.C + c] = b;
        const float gm = gamma[p.c_begin + c];
        red[c] = make_float2(gm * b, gm * a);   // dh, dh h
    }
    __syncthreads();
    const int gl = group_lanes(p.g_count), lane = threadIdx.x & (gl - 1), per = channels / p.g_count;
    for (int g0 = 0; g0 < p.g_count; g0 += kThreads / gl) {
        const int g = g0 + threadIdx.x / gl, own = g < p.g_count ? per : 0;
        float s1 = 0.f, s2 = 0.f;
        for (int c = lane; c < own; c += gl) {
            s1 += red[g * per + c].x;
            s2 += red[g * per + c].y;
        }
        s1 = lanes_sum(s1, gl);
        s2 = lanes_sum(s2, gl);
        if (lane == 0 && own)
            sums[partial(t, p.n, p.g_begin + g) + (size_t)p.split * t.parts + p.tile % t.parts] = make_float2(s1, s2);
    }
}

// dx; the CTAs behind the tiles' sum up dgamma and dbeta.
template <typename IO, int V, bool kGate, bool kSilu>
__global__ void __launch_bounds__(kThreads)
group_norm_bwd_apply_kernel(const IO* __restrict__ x, const IO* __restrict__ gate,
                            const float* __restrict__ gamma, const float* __restrict__ beta,
                            const float2* __restrict__ stats,
                            const float2* __restrict__ sums, const IO* __restrict__ dy,
                            IO* __restrict__ dx, const float* __restrict__ rows,
                            float* __restrict__ dgamma, float* __restrict__ dbeta, unsigned ctas,
                            Tiling t) {
    __shared__ float2 sum[kThreads * V];
    if (blockIdx.x >= ctas) {
        previous_ended();
        sum_params<kThreads / 32>(behind(rows), t.N * t.splits, t.C, (int)(blockIdx.x - ctas), dgamma, dbeta);
        return;
    }
    const Place p = place(t);
    const size_t base = ((size_t)p.n * t.L) * t.C + p.c0;
    constexpr int kTurn = sizeof(IO) == 4 ? 1 : 2;
    Raw<IO, V> rx[kTurn], rd[kTurn], rg[kTurn];
    float mean[V], r[V], ga[V], be[V], s1[V], s2[V];
    auto fetch = [&](long l) {
#pragma unroll
        for (int i = 0; i < kTurn; ++i, l += t.lanes)
            if (l < p.l1) {
                const size_t o = base + (size_t)l * t.C;
                rx[i] = load_raw<IO, V>(x + o);
                rd[i] = load_raw<IO, V>(dy + o);
                if (kGate) rg[i] = load_raw<IO, V>(gate + o);
            }
    };
    if (p.in) {
        load<V>(gamma + p.c0, ga);
        load<V>(beta + p.c0, be);
        fetch(p.l0);
    }
    previous_ended();
    stats = behind(stats);
    sums = behind(sums);
    {
        const int lanes = group_lanes(p.g_count), lane = threadIdx.x & (lanes - 1), items = t.splits * t.parts;
        const float inv = 1.f / ((float)t.L * (float)t.per);
        for (int g0 = 0; g0 < p.g_count; g0 += kThreads / lanes) {
            const int g = g0 + threadIdx.x / lanes;
            const float2* pp = sums + partial(t, p.n, p.g_begin + (g < p.g_count ? g : 0));
            float s1 = 0.f, s2 = 0.f;
#pragma unroll 4
            for (int i = lane; i < items; i += lanes) {
                s1 += pp[i].x;
                s2 += pp[i].y;
            }
            s1 = lanes_sum(s1, lanes);
            s2 = lanes_sum(s2, lanes);
            if (lane == 0 && g < p.g_count) sum[g] = make_float2(s1 * inv, s2 * inv);
        }
        __syncthreads();
    }
    if (!p.in) return;
    each_group<V>(t, p.c0, [&](int e, int g) {
        const float2 st = stats[p.n * t.groups + g], su = sum[g - p.g_begin];
        mean[e] = st.x;
        r[e] = st.y;
        s1[e] = su.x;
        s2[e] = su.y;
    });
    for (long l = p.l0; l < p.l1; l += kTurn * t.lanes) {
        Raw<IO, V> cx[kTurn], cd[kTurn], cg[kTurn];
#pragma unroll
        for (int i = 0; i < kTurn; ++i) {
            cx[i] = rx[i];
            cd[i] = rd[i];
            if (kGate) cg[i] = rg[i];
        }
        fetch(l + kTurn * t.lanes);
#pragma unroll
        for (int i = 0; i < kTurn; ++i) {
            const long at = l + i * t.lanes;
            if (at >= p.l1) break;
            float v[V], d[V], gt[V];
            convert(cx[i], v);
            convert(cd[i], d);
            if (kGate) convert(cg[i], gt);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float h = (v[e] - mean[e]) * r[e];
                const float dz = d[e] * (kGate ? act<IO>(gt[e], kSilu)
                                              : act_grad<IO>(fmaf(h, ga[e], be[e]), kSilu).y);
                d[e] = r[e] * (dz * ga[e] - s1[e] - h * s2[e]);
            }
            store<V>(dx + base + (size_t)at * t.C, d);
        }
    }
}

// ------------------------------------------------------------------ host
constexpr int kSms = 148;

// Registers hold up to 4 vectors of 8 a lane (groups of up to 1024 channels; 2 in the backward),
// or 8 single values (groups of up to 256).  Sets of lanes for `ctas` CTAs an SM, and no more
// streams than rows.
RowShape row_shape(long N, int C, int groups, int ctas) {
    RowShape s{N, C, groups, C / groups, 0, 1, 1};
    const int V = s.per % 8 == 0 ? 8 : 1;
    s.units = s.per / V;
    while (s.lanes < s.units && s.lanes < 32) s.lanes *= 2;
    const long sets = (long)kSms * ctas * (kThreads / s.lanes);
    const long n = (sets + groups - 1) / groups;
    s.streams = n < 1 ? 1 : n > N ? N : n;
    return s;
}
constexpr int kFwdCtas = 8, kBwdCtas = 3;
unsigned row_ctas(const RowShape& s) {
    const int per_cta = kThreads / s.lanes;
    return (unsigned)((s.streams * s.groups + per_cta - 1) / per_cta);
}
int row_units(const RowShape& s) {   // the U of the kernels
    const int need = (s.units + s.lanes - 1) / s.lanes;
    const bool vec = s.per % 8 == 0;
    if (need <= 1) return 1;
    if (need <= 2) return 2;
    if (need <= 4) return 4;
    return !vec && need <= 8 ? 8 : 0;
}

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

Tiling tiling(long N, long L, int C, int groups) {
    Tiling t{};
    t.N = N;
    t.L = L;
    t.C = C;
    t.groups = groups;
    t.per = C / groups;
    // vectors of 8 where rows keep them aligned and a tile's bounds can be group bounds too
    const long unit = (long)t.per * 8 / gcd(t.per, 8);
    t.V = C % 8 == 0 && (unit <= 8 * kThreads || t.per % 8 == 0) ? 8 : 1;
    const int most = t.V * kThreads, whole = t.V == 8 ? (int)(unit < most ? unit : most) : t.per;
    if (t.per <= most) {
        t.parts = 1;
        t.width = most / whole * whole;
        if (t.width > C) t.width = C;
        t.tiles = (C + t.width - 1) / t.width;
    } else {
        t.width = most;
        t.parts = (t.per + most - 1) / most;
        t.tiles = groups * t.parts;
    }
    t.vecs = (t.width + t.V - 1) / t.V;
    t.lanes = kThreads / t.vecs;
    // splits: two CTAs an SM (each pays a few hundred instructions a thread to join its groups:
    // [8, 4093, 320] 17 us, with one 24, with three or four 23), but at least 4 positions a lane
    const long ctas = N * t.tiles;
    long want = (2L * kSms + ctas - 1) / ctas;
    const long limit = (L + 4L * t.lanes - 1) / (4L * t.lanes);
    if (want > limit) want = limit;
    if (want < 1) want = 1;
    t.span = (L + want - 1) / want;
    t.splits = (int)((L + t.span - 1) / t.span);
    return t;
}
unsigned tile_ctas(const Tiling& t) { return (unsigned)(t.N * t.splits * t.tiles); }

size_t r256(size_t x) { return (x + 255) & ~size_t(255); }
size_t stats_bytes(const Tiling& t) { return r256((size_t)t.N * t.groups * sizeof(float2)); }
size_t partial_bytes(const Tiling& t) {
    return r256((size_t)t.N * t.groups * t.splits * t.parts * sizeof(float2));
}

template <typename IO, int V, int U>
cudaError_t rows_fwd(const GroupNorm& a, void* y, const RowShape& s, cudaStream_t st) {
    auto run = [&](auto kernel) {
        kernel<<<row_ctas(s), kThreads, 0, st>>>((const IO*)a.x, (const IO*)a.gate, a.gamma, a.beta, a.eps,
                                                 (IO*)y, s);
    };
    if (a.gate) a.silu ? run(group_norm_rows_kernel<IO, V, U, true, true>) : run(group_norm_rows_kernel<IO, V, U, true, false>);
    else a.silu ? run(group_norm_rows_kernel<IO, V, U, false, true>) : run(group_norm_rows_kernel<IO, V, U, false, false>);
    return cudaGetLastError();
}
template <typename IO, int V, int U>
cudaError_t rows_bwd(const GroupNorm& a, const void* dy, void* dx, void* dgate, float* part,
                     const RowShape& s, cudaStream_t st) {
    auto run = [&](auto kernel) {
        kernel<<<row_ctas(s), kThreads, 0, st>>>((const IO*)a.x, (const IO*)a.gate, a.gamma, a.beta, a.eps,
                                                 (const IO*)dy, (IO*)dx, (IO*)dgate, part, s);
    };
    if (a.gate) a.silu ? run(group_norm_rows_bwd_kernel<IO, V, U, true, true>) : run(group_norm_rows_bwd_kernel<IO, V, U, true, false>);
    else a.silu ? run(group_norm_rows_bwd_kernel<IO, V, U, false, true>) : run(group_norm_rows_bwd_kernel<IO, V, U, false, false>);
    return cudaGetLastError();
}

template <typename IO, int V, bool kGate, bool kSilu>
cudaError_t positions_fwd(const GroupNorm& a, void* y, void* ws, const Tiling& t, cudaStream_t st) {
    float2* part = static_cast<float2*>(ws);
    const IO* x = (const IO*)a.x;
    group_norm_stats_kernel<IO, V><<<tile_ctas(t), kThreads, 0, st>>>(x, part, t);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_next(group_norm_apply_kernel<IO, V, kGate, kSilu>, tile_ctas(t), kThreads, 0, st, x,
                       (const IO*)a.gate, a.gamma, a.beta, a.eps, part, (IO*)y, t);
}
template <typename IO, int V, bool kGate, bool kSilu>
cudaError_t positions_bwd(const GroupNorm& a, const void* dy, void* dx, float* dgamma, float* dbeta,
                          void* dgate, void* ws, const Tiling& t, cudaStream_t st) {
    uint8_t* w = static_cast<uint8_t*>(ws);
    float2* stats = reinterpret_cast<float2*>(w);
    float2* part = reinterpret_cast<float2*>(w += stats_bytes(t));
    float2* sums = reinterpret_cast<float2*>(w += partial_bytes(t));
    float* rows = reinterpret_cast<float*>(w += partial_bytes(t));
    const IO *x = (const IO*)a.x, *gate = (const IO*)a.gate, *d = (const IO*)dy;
    const unsigned grid = tile_ctas(t), params = (unsigned)((2 * t.C + 31) / 32);
    group_norm_stats_kernel<IO, V><<<grid, kThreads, 0, st>>>(x, part, t);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    e = launch_next(group_norm_bwd_sums_kernel<IO, V, kGate, kSilu>, grid, kThreads, 0, st, x, gate, a.gamma, a.beta,
                    a.eps, part, d, (IO*)dgate, stats, rows, sums, t);
    if (e != cudaSuccess) return e;
    return launch_next(group_norm_bwd_apply_kernel<IO, V, kGate, kSilu>, grid + params, kThreads, 0, st, x, gate,
                       a.gamma, a.beta, stats, sums, d, (IO*)dx, rows, dgamma, dbeta, grid, t);
}
// f(vector width, gate, silu), the three as compile-time constants
template <typename F>
cudaError_t with_constants(const GroupNorm& a, const Tiling& t, F f) {
    using std::integral_constant;
    auto act = [&](auto v, auto gate) {
        return a.silu ? f(v, gate, std::true_type{}) : f(v, gate, std::false_type{});
    };
    auto gated = [&](auto v) { return a.gate ? act(v, std::true_type{}) : act(v, std::false_type{}); };
    return t.V == 8 ? gated(integral_constant<int, 8>{}) : gated(integral_constant<int, 1>{});
}

// f(lanes of a set, gate, silu) as compile-time constants, where a group is exactly a power of two
// of vectors of 8, up to 32; false otherwise.
template <typename F>
bool full_rows(const GroupNorm& a, const RowShape& s, F f) {
    using std::integral_constant;
    if (s.per % 8 != 0 || s.units != s.lanes) return false;
    auto act = [&](auto l, auto gate) { a.silu ? f(l, gate, std::true_type{}) : f(l, gate, std::false_type{}); };
    auto run = [&](auto l) { a.gate ? act(l, std::true_type{}) : act(l, std::false_type{}); };
    switch (s.lanes) {
    case 1: run(integral_constant<int, 1>{}); break;
    case 2: run(integral_constant<int, 2>{}); break;
    case 4: run(integral_constant<int, 4>{}); break;
    case 8: run(integral_constant<int, 8>{}); break;
    case 16: run(integral_constant<int, 16>{}); break;
    default: run(integral_constant<int, 32>{}); break;
    }
    return true;
}

template <typename IO>
cudaError_t forward_io(const GroupNorm& a, void* y, void* ws, cudaStream_t st) {
    if (a.L == 1) {
        const RowShape s = row_shape(a.N, a.C, a.groups, kFwdCtas);
        const int u = row_units(s);
        if (full_rows(a, s, [&](auto l, auto gate, auto silu) {
                group_norm_full_rows_kernel<IO, l(), gate(), silu()><<<row_ctas(s), kThreads, 0, st>>>(
                    (const IO*)a.x, (const IO*)a.gate, a.gamma, a.beta, a.eps, (IO*)y, s);
            }))
            return cudaGetLastError();
        if (s.per % 8 == 0)
            return u == 1 ? rows_fwd<IO, 8, 1>(a, y, s, st) : u == 2 ? rows_fwd<IO, 8, 2>(a, y, s, st)
                 : u == 4 ? rows_fwd<IO, 8, 4>(a, y, s, st) : rows_fwd<IO, 8, 0>(a, y, s, st);
        return u == 1 ? rows_fwd<IO, 1, 1>(a, y, s, st) : u == 2 ? rows_fwd<IO, 1, 2>(a, y, s, st)
             : u == 4 ? rows_fwd<IO, 1, 4>(a, y, s, st) : u == 8 ? rows_fwd<IO, 1, 8>(a, y, s, st)
             : rows_fwd<IO, 1, 0>(a, y, s, st);
    }
    const Tiling t = tiling(a.N, a.L, a.C, a.groups);
    return with_constants(a, t, [&](auto v, auto gate, auto silu) {
        return positions_fwd<IO, v(), gate(), silu()>(a, y, ws, t, st);
    });
}

template <typename IO>
cudaError_t backward_io(const GroupNorm& a, const void* dy, void* dx, float* dgamma, float* dbeta,
                        void* dgate, void* ws, cudaStream_t st) {
    if (a.L == 1) {
        const RowShape s = row_shape(a.N, a.C, a.groups, kBwdCtas);
        const int u = row_units(s);
        float* part = static_cast<float*>(ws);
        cudaError_t e;
        if (full_rows(a, s, [&](auto l, auto gate, auto silu) {
                group_norm_full_rows_bwd_kernel<IO, l(), gate(), silu()><<<row_ctas(s), kThreads, 0, st>>>(
                    (const IO*)a.x, (const IO*)a.gate, a.gamma, a.beta, a.eps, (const IO*)dy, (IO*)dx, (IO*)dgate,
                    part, s);
            }))
            e = cudaGetLastError();
        else if (s.per % 8 == 0)
            e = u == 1 ? rows_bwd<IO, 8, 1>(a, dy, dx, dgate, part, s, st)
              : u == 2 ? rows_bwd<IO, 8, 2>(a, dy, dx, dgate, part, s, st)
                       : rows_bwd<IO, 8, 0>(a, dy, dx, dgate, part, s, st);   // 4 would spill
        else
            e = u == 1 ? rows_bwd<IO, 1, 1>(a, dy, dx, dgate, part, s, st)
              : u == 2 ? rows_bwd<IO, 1, 2>(a, dy, dx, dgate, part, s, st)
              : u == 4 ? rows_bwd<IO, 1, 4>(a, dy, dx, dgate, part, s, st)
              : u == 8 ? rows_bwd<IO, 1, 8>(a, dy, dx, dgate, part, s, st)
                       : rows_bwd<IO, 1, 0>(a, dy, dx, dgate, part, s, st);
        if (e != cudaSuccess) return e;
        return launch_next(group_norm_param_kernel, (unsigned)((2 * a.C + 31) / 32), 32 * kParamWarps, 0, st, part,
                           s.streams, a.C, dgamma, dbeta);
    }
    const Tiling t = tiling(a.N, a.L, a.C, a.groups);
    return with_constants(a, t, [&](auto v, auto gate, auto silu) {
        return positions_bwd<IO, v(), gate(), silu()>(a, dy, dx, dgamma, dbeta, dgate, ws, t, st);
    });
}

}  // namespace

size_t group_norm_bytes(long N, long L, int C, int groups) {
    return L == 1 ? 0 : partial_bytes(tiling(N, L, C, groups));
}

size_t group_norm_backward_bytes(long N, long L, int C, int groups) {
    if (L == 1) return r256((size_t)row_shape(N, C, groups, kBwdCtas).streams * 2 * C * sizeof(float));
    const Tiling t = tiling(N, L, C, groups);
    return stats_bytes(t) + 2 * partial_bytes(t) + r256((size_t)N * t.splits * 2 * C * sizeof(float));
}

cudaError_t launch_group_norm(const GroupNorm& a, void* y, void* ws, bool bf16, cudaStream_t st) {
    return bf16 ? forward_io<__nv_bfloat16>(a, y, ws, st) : forward_io<float>(a, y, ws, st);
}

cudaError_t launch_group_norm_backward(const GroupNorm& a, const void* dy, void* dx, float* dgamma,
                                       float* dbeta, void* dgate, void* ws, bool bf16,
                                       cudaStream_t st) {
    return bf16 ? backward_io<__nv_bfloat16>(a, dy, dx, dgamma, dbeta, dgate, ws, st)
                : backward_io<float>(a, dy, dx, dgamma, dbeta, dgate, ws, st);
}

}  // namespace goldwkv
