// Group norm over channels-last tensors with an activation, forward and backward (sm_100a).
//
// x [N][L][C]; for each n and group of per = C / groups channels, over its L positions:
//     h = (x - mean) / sqrt(var + eps),   z = h gamma + beta,   y = act(z), or z act(gate).
// Backward, with dz = dy act'(z) (or dy act(gate), and then dgate = dy z act'(gate)):
//     dbeta = sum dz,   dgamma = sum dz h   (over n and positions),
//     dh = dz gamma,    dx = (dh - mean(dh) - h mean(dh h)) / sqrt(var + eps).
// Every pass is bound by memory; sums are fp32, of differences from a value of the data, so
// that a mean far from zero costs no digits.
//
// One position (L = 1, each token's heads): a group is a contiguous run of `per` values held
// in the registers of a few adjacent lanes, read once and written once in one launch.
//
// Several positions: a thread owns 8 adjacent channels (one, where C is no multiple of 8) and
// walks positions, so that accesses are whole rows whatever the group's width; it keeps sums
// per channel, which a small second launch joins into groups, before a third pass applies
// them.  The positions of one n are cut into as many splits as fill the device.
#include "common.cuh"
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

// sigmoid: the fast exponential and division where the result is rounded to bf16 (relative
// error about 2^-21), the accurate ones for fp32.
template <typename IO> __device__ __forceinline__ float sigmoid(float x);
template <> __device__ __forceinline__ float sigmoid<float>(float x) { return 1.f / (1.f + expf(-x)); }
template <> __device__ __forceinline__ float sigmoid<__nv_bfloat16>(float x) {
    return __fdividef(1.f, 1.f + __expf(-x));
}
template <typename IO>
__device__ __forceinline__ float act(float x, bool silu) { return silu ? x * sigmoid<IO>(x) : x; }
// act(x) and act'(x)
template <typename IO>
__device__ __forceinline__ float2 act_grad(float x, bool silu) {
    if (!silu) return make_float2(x, 1.f);
    const float s = sigmoid<IO>(x);
    return make_float2(x * s, s * fmaf(x, 1.f - s, 1.f));
}

// sum over the `lanes` (a power of two) adjacent lanes of a group
__device__ __forceinline__ float lanes_sum(float x, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// ------------------------------------------------------------------ one position
// A group's `units` (of V values) lie on `lanes` adjacent lanes, U a lane (unit = lane +
// lanes * i), in registers.  U = 0: more than the registers hold, read again for each pass.
struct RowShape {
    long rows;       // N
    int C, groups, per, units, lanes;
};

// lanes_sum over everything of group g of row n that this lane holds or reads
template <typename IO, int V, int U>
__global__ void __launch_bounds__(kThreads)
group_norm_rows_kernel(const IO* __restrict__ x, const IO* __restrict__ gate,
                       const float* __restrict__ gamma, const float* __restrict__ beta, float eps,
                       bool silu, IO* __restrict__ y, RowShape s) {
    const int per_cta = kThreads / s.lanes;                 // groups a CTA takes
    const long item = (long)blockIdx.x * per_cta + threadIdx.x / s.lanes;
    const int l = threadIdx.x & (s.lanes - 1);
    const bool in = item < s.rows * s.groups;
    const long n = in ? item / s.groups : 0;
    const int g = in ? (int)(item - n * s.groups) : 0;
    const size_t base = (size_t)n * s.C + (size_t)g * s.per;
    const float inv_n = 1.f / (float)s.per;
    if (U > 0) {
        constexpr int K = U > 0 ? U : 1;
        float v[K][V], gt[K][V];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int u = l + s.lanes * i;
            if (in && u < s.units) {
                load<V>(x + base + (size_t)u * V, v[i]);
                if (gate) load<V>(gate + base + (size_t)u * V, gt[i]);
#pragma unroll
                for (int e = 0; e < V; ++e) sum += v[i][e];
            }
        }
        const float mean = lanes_sum(sum, s.lanes) * inv_n;
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < K; ++i)
            if (in && l + s.lanes * i < s.units) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    v[i][e] -= mean;
                    sq = fmaf(v[i][e], v[i][e], sq);
                }
            }
        const float r = rsqrtf(lanes_sum(sq, s.lanes) * inv_n + eps);
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int u = l + s.lanes * i;
            if (in && u < s.units) {
                float ga[V], be[V];
                load<V>(gamma + g * s.per + u * V, ga);
                load<V>(beta + g * s.per + u * V, be);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float z = fmaf(v[i][e] * r, ga[e], be[e]);
                    v[i][e] = gate ? z * act<IO>(gt[i][e], silu) : act<IO>(z, silu);
                }
                store<V>(y + base + (size_t)u * V, v[i]);
            }
        }
    } else {
        float v[V], gt[V], sum = 0.f, sq = 0.f;
        if (in)
            for (int u = l; u < s.units; u += s.lanes) {
                load<V>(x + base + (size_t)u * V, v);
#pragma unroll
                for (int e = 0; e < V; ++e) sum += v[e];
            }
        const float mean = lanes_sum(sum, s.lanes) * inv_n;
        if (in)
            for (int u = l; u < s.units; u += s.lanes) {
                load<V>(x + base + (size_t)u * V, v);
#pragma unroll
                for (int e = 0; e < V; ++e) sq = fmaf(v[e] - mean, v[e] - mean, sq);
            }
        const float r = rsqrtf(lanes_sum(sq, s.lanes) * inv_n + eps);
        if (in)
            for (int u = l; u < s.units; u += s.lanes) {
                float ga[V], be[V];
                load<V>(x + base + (size_t)u * V, v);
                if (gate) load<V>(gate + base + (size_t)u * V, gt);
                load<V>(gamma + g * s.per + u * V, ga);
                load<V>(beta + g * s.per + u * V, be);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float z = fmaf((v[e] - mean) * r, ga[e], be[e]);
                    v[e] = gate ? z * act<IO>(gt[e], silu) : act<IO>(z, silu);
                }
                store<V>(y + base + (size_t)u * V, v);
            }
    }
}

// Backward over rows: a set of `lanes` lanes keeps one group g and walks rows n = stream,
// stream + streams, ..., so that its channels' dgamma and dbeta sums stay in registers
// (U > 0); they leave as one row of partial sums a stream.  U = 0 (wide groups): the sums are
// kept in the partial row itself, which no one else touches.
template <typename IO, int V, int U>
__global__ void __launch_bounds__(kThreads)
group_norm_rows_bwd_kernel(const IO* __restrict__ x, const IO* __restrict__ gate,
                           const float* __restrict__ gamma, const float* __restrict__ beta,
                           float eps, bool silu, const IO* __restrict__ dy, IO* __restrict__ dx,
                           IO* __restrict__ dgate, float* __restrict__ part, long streams,
                           RowShape s) {
    const int per_cta = kThreads / s.lanes;
    const long set = (long)blockIdx.x * per_cta + threadIdx.x / s.lanes;
    const int l = threadIdx.x & (s.lanes - 1);
    const bool in = set < streams * s.groups;
    const long stream = in ? set / s.groups : 0;
    const int g = in ? (int)(set - stream * s.groups) : 0;
    const int c0 = g * s.per;
    const float inv_n = 1.f / (float)s.per;
    // partial rows: dgamma then dbeta, [streams][2][C]
    float* pg = part + (size_t)stream * 2 * s.C + c0;
    float* pb = pg + s.C;
    constexpr int K = U > 0 ? U : 1;
    float dga[K][V], dbe[K][V], ga[K][V], be[K][V];
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) dga[i][e] = dbe[i][e] = ga[i][e] = be[i][e] = 0.f;
    if (U > 0) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int u = l + s.lanes * i;
            if (in && u < s.units) {
                load<V>(gamma + c0 + u * V, ga[i]);
                load<V>(beta + c0 + u * V, be[i]);
            }
        }
    } else if (in) {
        for (int u = l; u < s.units; u += s.lanes) {
            store<V>(pg + u * V, dga[0]);
            store<V>(pb + u * V, dga[0]);
        }
    }
    // every lane of a warp runs the same number of rows: the shuffles need them all
    const long turns = (s.rows + streams - 1) / streams;
    for (long it = 0; it < turns; ++it) {
        const long n = stream + it * streams;
        const bool row = in && n < s.rows;
        const size_t base = (size_t)(row ? n : 0) * s.C + c0;
        if (U > 0) {
            float v[K][V], d[K][V], gt[K][V];
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const int u = l + s.lanes * i;
                if (row && u < s.units) {
                    load<V>(x + base + (size_t)u * V, v[i]);
                    load<V>(dy + base + (size_t)u * V, d[i]);
                    if (gate) load<V>(gate + base + (size_t)u * V, gt[i]);
#pragma unroll
                    for (int e = 0; e < V; ++e) sum += v[i][e];
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) v[i][e] = d[i][e] = gt[i][e] = 0.f;
                }
            }
            const float mean = lanes_sum(sum, s.lanes) * inv_n;
            float sq = 0.f;
#pragma unroll
            for (int i = 0; i < K; ++i)
                if (row && l + s.lanes * i < s.units) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        v[i][e] -= mean;
                        sq = fmaf(v[i][e], v[i][e], sq);
                    }
                }
            const float r = rsqrtf(lanes_sum(sq, s.lanes) * inv_n + eps);
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const int u = l + s.lanes * i;
                const bool has = row && u < s.units;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float h = v[i][e] * r, z = fmaf(h, ga[i][e], be[i][e]);
                    float dz;
                    if (gate) {
                        const float2 a = act_grad<IO>(gt[i][e], silu);
                        gt[i][e] = d[i][e] * z * a.y;
                        dz = d[i][e] * a.x;
                    } else {
                        dz = d[i][e] * act_grad<IO>(z, silu).y;
                    }
                    if (has) {
                        dga[i][e] = fmaf(dz, h, dga[i][e]);
                        dbe[i][e] += dz;
                        const float dh = dz * ga[i][e];
                        s1 += dh;
                        s2 = fmaf(dh, h, s2);
                        d[i][e] = dh;
                        v[i][e] = h;
                    }
                }
                if (gate && has) store<V>(dgate + base + (size_t)u * V, gt[i]);
            }
            s1 = lanes_sum(s1, s.lanes) * inv_n;
            s2 = lanes_sum(s2, s.lanes) * inv_n;
#pragma unroll
            for (int i = 0; i < K; ++i) {
                const int u = l + s.lanes * i;
                if (row && u < s.units) {
#pragma unroll
                    for (int e = 0; e < V; ++e) d[i][e] = r * (d[i][e] - s1 - v[i][e] * s2);
                    store<V>(dx + base + (size_t)u * V, d[i]);
                }
            }
        } else {
            float v[V], d[V], gt[V], gg[V], bb[V];
            float sum = 0.f, sq = 0.f, s1 = 0.f, s2 = 0.f;
            const int units = row ? s.units : 0;
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
                    if (gate) load<V>(gate + base + (size_t)u * V, gt);
                    load<V>(gamma + c0 + u * V, gg);
                    load<V>(beta + c0 + u * V, bb);
                    float a1[V], a2[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float h = (v[e] - mean) * r, z = fmaf(h, gg[e], bb[e]);
                        float dz;
                        if (gate) {
                            const float2 a = act_grad<IO>(gt[e], silu);
                            gt[e] = d[e] * z * a.y;
                            dz = d[e] * a.x;
                        } else {
                            dz = d[e] * act_grad<IO>(z, silu).y;
                        }
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
                        if (gate) store<V>(dgate + base + (size_t)u * V, gt);
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
    if (U > 0) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int u = l + s.lanes * i;
            if (in && u < s.units) {
                store<V>(pg + u * V, dga[i]);
                store<V>(pb + u * V, dbe[i]);
            }
        }
    }
}

// dgamma[c], dbeta[c] = the sums of `rows` partial rows ([rows][2][C]), in a fixed order: 32
// columns a CTA, 8 row lanes each, joined through shared memory.
__global__ void __launch_bounds__(kThreads)
group_norm_param_kernel(const float* __restrict__ part, long rows, int C, float* __restrict__ dgamma,
                        float* __restrict__ dbeta) {
    __shared__ float red[kThreads / 32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int i = blockIdx.x * 32 + lane;   // column of the 2 C
    float acc = 0.f;
    if (i < 2 * C)
        for (long r = warp; r < rows; r += kThreads / 32) acc += part[(size_t)r * 2 * C + i];
    red[warp][lane] = acc;
    __syncthreads();
    if (warp == 0 && i < 2 * C) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) t += red[w][lane];
        if (i < C) dgamma[i] = t;
        else dbeta[i - C] = t;
    }
}

// ------------------------------------------------------------------ several positions
// A CTA covers positions [l0, l1) of one n and a tile of up to kThreads channel vectors;
// thread = (row lane, vector): row lane i walks positions l0 + i, l0 + i + lanes, ...
struct Tiling {
    long N, L;
    int C, groups, per;
    int vecs;        // channel vectors of the tile in use (all of them when C fits one)
    int lanes;       // position lanes of the CTA
    int ctiles;      // channel tiles
    int splits;      // splits of the positions
    long span;       // positions of a split
};
struct Place {
    long n;
    int split, c0;       // first channel of the thread's vector
    long l0, l1;         // its positions: l0, l0 + lanes, ... < l1
    bool in;
};
template <int V>
__device__ __forceinline__ Place place(const Tiling& t) {
    Place p;
    long i = blockIdx.x;
    const int ct = (int)(i % t.ctiles);
    i /= t.ctiles;
    p.split = (int)(i % t.splits);
    p.n = i / t.splits;
    const int lane = threadIdx.x / t.vecs, vec = ct * t.vecs + (threadIdx.x - lane * t.vecs);
    p.c0 = vec * V;
    p.l0 = p.split * t.span + lane;
    p.l1 = min(t.L, (p.split + 1) * t.span);
    p.in = lane < t.lanes && p.c0 < t.C;
    return p;
}

// Per channel of a split: mean and the sum of squares about it.  part [N][splits][C] float2.
template <typename IO, int V>
__global__ void __launch_bounds__(kThreads)
group_norm_stats_kernel(const IO* __restrict__ x, float2* __restrict__ part, Tiling t) {
    __shared__ float2 red[kThreads * V];   // (lane, vector, element): mean, M2
    const Place p = place<V>(t);
    const IO* xp = x + ((size_t)p.n * t.L) * t.C + p.c0;
    float k[V], a[V], q[V];
    int cnt = 0;
#pragma unroll
    for (int e = 0; e < V; ++e) k[e] = a[e] = q[e] = 0.f;
    if (p.in && p.l0 < p.l1) {
        load<V>(xp + (size_t)p.l0 * t.C, k);   // differences from the thread's first values
#pragma unroll 4
        for (long l = p.l0; l < p.l1; l += t.lanes) {
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
    }
    const float inv = cnt > 0 ? 1.f / (float)cnt : 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float m = a[e] * inv;
        red[threadIdx.x * V + e] = make_float2(k[e] + m, fmaxf(q[e] - a[e] * m, 0.f));
    }
    __syncthreads();
    // join the position lanes of each channel
    const long first = (long)p.split * t.span, have = max(0L, min(t.L, first + t.span) - first);
    const int ct = (int)(blockIdx.x % t.ctiles), width = t.vecs * V;
    for (int c = threadIdx.x; c < width; c += kThreads) {
        const int ch = ct * width + c;
        if (ch >= t.C) continue;
        float mean = 0.f, m2 = 0.f;
        for (int i = 0; i < t.lanes; ++i) {
            const long n_i = have > i ? (have - i + t.lanes - 1) / t.lanes : 0;
            mean += (float)n_i * red[i * width + c].x;
        }
        mean /= (float)have;
        for (int i = 0; i < t.lanes; ++i) {
            const long n_i = have > i ? (have - i + t.lanes - 1) / t.lanes : 0;
            const float2 r = red[i * width + c];
            const float d = r.x - mean;
            m2 += r.y + (float)n_i * d * d;
        }
        part[((size_t)p.n * t.splits + p.split) * t.C + ch] = make_float2(mean, m2);
    }
}

__device__ __forceinline__ float cta_sum(float x, float* red) {
    x = warp_sum(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    float t = 0.f;
    for (int w = 0; w < (int)(blockDim.x >> 5); ++w) t += red[w];
    return t;
}

// (mean, 1 / sqrt(var + eps)) of each (n, group) from the channels' partial statistics.
__global__ void __launch_bounds__(128)
group_norm_join_stats_kernel(const float2* __restrict__ part, float2* __restrict__ stats, float eps,
                             Tiling t) {
    __shared__ float red[4];
    const long n = blockIdx.x / t.groups;
    const int g = (int)(blockIdx.x - n * t.groups);
    const float2* pp = part + (size_t)n * t.splits * t.C + (size_t)g * t.per;
    const long items = (long)t.splits * t.per;
    float s = 0.f;
    for (long i = threadIdx.x; i < items; i += blockDim.x) {
        const int sp = (int)(i / t.per), c = (int)(i - (long)sp * t.per);
        const float cnt = (float)(min(t.L, (sp + 1) * t.span) - sp * t.span);
        s = fmaf(cnt, pp[(size_t)sp * t.C + c].x, s);
    }
    const float inv = 1.f / ((float)t.L * (float)t.per);
    const float mean = cta_sum(s, red) * inv;
    float q = 0.f;
    for (long i = threadIdx.x; i < items; i += blockDim.x) {
        const int sp = (int)(i / t.per), c = (int)(i - (long)sp * t.per);
        const float cnt = (float)(min(t.L, (sp + 1) * t.span) - sp * t.span);
        const float2 r = pp[(size_t)sp * t.C + c];
        const float d = r.x - mean;
        q += fmaf(cnt * d, d, r.y);
    }
    const float var = cta_sum(q, red) * inv;
    if (threadIdx.x == 0) stats[blockIdx.x] = make_float2(mean, rsqrtf(var + eps));
}

template <typename IO, int V>
__global__ void __launch_bounds__(kThreads)
group_norm_apply_kernel(const IO* __restrict__ x, const IO* __restrict__ gate,
                        const float* __restrict__ gamma, const float* __restrict__ beta, bool silu,
                        const float2* __restrict__ stats, IO* __restrict__ y, Tiling t) {
    const Place p = place<V>(t);
    if (!p.in) return;
    float mean[V], r[V], be[V];
    load<V>(gamma + p.c0, r);
    load<V>(beta + p.c0, be);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float2 st = stats[p.n * t.groups + (p.c0 + e) / t.per];
        mean[e] = st.x;
        r[e] *= st.y;
    }
    const size_t base = ((size_t)p.n * t.L) * t.C + p.c0;
#pragma unroll 2
    for (long l = p.l0; l < p.l1; l += t.lanes) {
        const size_t o = base + (size_t)l * t.C;
        float v[V], gt[V];
        load<V>(x + o, v);
        if (gate) load<V>(gate + o, gt);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float z = fmaf(v[e] - mean[e], r[e], be[e]);
            v[e] = gate ? z * act<IO>(gt[e], silu) : act<IO>(z, silu);
        }
        store<V>(y + o, v);
    }
}

// Per channel of a split: sums of dz h and of dz; dgate.  part [N][splits][2][C].
template <typename IO, int V>
__global__ void __launch_bounds__(kThreads)
group_norm_bwd_sums_kernel(const IO* __restrict__ x, const IO* __restrict__ gate,
                           const float* __restrict__ gamma, const float* __restrict__ beta,
                           bool silu, const float2* __restrict__ stats, const IO* __restrict__ dy,
                           IO* __restrict__ dgate, float* __restrict__ part, Tiling t) {
    __shared__ float2 red[kThreads * V];
    const Place p = place<V>(t);
    float sg[V], sb[V];
#pragma unroll
    for (int e = 0; e < V; ++e) sg[e] = sb[e] = 0.f;
    if (p.in) {
        float mean[V], r[V], ga[V], be[V];
        load<V>(gamma + p.c0, ga);
        load<V>(beta + p.c0, be);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float2 st = stats[p.n * t.groups + (p.c0 + e) / t.per];
            mean[e] = st.x;
            r[e] = st.y;
        }
        const size_t base = ((size_t)p.n * t.L) * t.C + p.c0;
        for (long l = p.l0; l < p.l1; l += t.lanes) {
            const size_t o = base + (size_t)l * t.C;
            float v[V], d[V], gt[V];
            load<V>(x + o, v);
            load<V>(dy + o, d);
            if (gate) load<V>(gate + o, gt);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float h = (v[e] - mean[e]) * r[e], z = fmaf(h, ga[e], be[e]);
                float dz;
                if (gate) {
                    const float2 a = act_grad<IO>(gt[e], silu);
                    gt[e] = d[e] * z * a.y;
                    dz = d[e] * a.x;
                } else {
                    dz = d[e] * act_grad<IO>(z, silu).y;
                }
                sg[e] = fmaf(dz, h, sg[e]);
                sb[e] += dz;
            }
            if (gate) store<V>(dgate + o, gt);
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) red[threadIdx.x * V + e] = make_float2(sg[e], sb[e]);
    __syncthreads();
    const int ct = (int)(blockIdx.x % t.ctiles), width = t.vecs * V;
    float* row = part + ((size_t)p.n * t.splits + p.split) * 2 * t.C;
    for (int c = threadIdx.x; c < width; c += kThreads) {
        const int ch = ct * width + c;
        if (ch >= t.C) continue;
        float a = 0.f, b = 0.f;
        for (int i = 0; i < t.lanes; ++i) {
            a += red[i * width + c].x;
            b += red[i * width + c].y;
        }
        row[ch] = a;
        row[t.C + ch] = b;
    }
}

// (mean(dh), mean(dh h)) of each (n, group).
__global__ void __launch_bounds__(128)
group_norm_join_sums_kernel(const float* __restrict__ part, const float* __restrict__ gamma,
                            float2* __restrict__ sums, Tiling t) {
    __shared__ float red[4];
    const long n = blockIdx.x / t.groups;
    const int g = (int)(blockIdx.x - n * t.groups);
    const float* pp = part + (size_t)n * t.splits * 2 * t.C + (size_t)g * t.per;
    const long items = (long)t.splits * t.per;
    float s1 = 0.f, s2 = 0.f;
    for (long i = threadIdx.x; i < items; i += blockDim.x) {
        const int sp = (int)(i / t.per), c = (int)(i - (long)sp * t.per);
        const float ga = gamma[g * t.per + c];
        s2 = fmaf(ga, pp[(size_t)sp * 2 * t.C + c], s2);
        s1 = fmaf(ga, pp[(size_t)sp * 2 * t.C + t.C + c], s1);
    }
    s1 = cta_sum(s1, red);
    s2 = cta_sum(s2, red);
    const float inv = 1.f / ((float)t.L * (float)t.per);
    if (threadIdx.x == 0) sums[blockIdx.x] = make_float2(s1 * inv, s2 * inv);
}

template <typename IO, int V>
__global__ void __launch_bounds__(kThreads)
group_norm_bwd_apply_kernel(const IO* __restrict__ x, const IO* __restrict__ gate,
                            const float* __restrict__ gamma, const float* __restrict__ beta,
                            bool silu, const float2* __restrict__ stats,
                            const float2* __restrict__ sums, const IO* __restrict__ dy,
                            IO* __restrict__ dx, Tiling t) {
    const Place p = place<V>(t);
    if (!p.in) return;
    float mean[V], r[V], ga[V], be[V], s1[V], s2[V];
    load<V>(gamma + p.c0, ga);
    load<V>(beta + p.c0, be);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const long i = p.n * t.groups + (p.c0 + e) / t.per;
        const float2 st = stats[i], su = sums[i];
        mean[e] = st.x;
        r[e] = st.y;
        s1[e] = su.x;
        s2[e] = su.y;
    }
    const size_t base = ((size_t)p.n * t.L) * t.C + p.c0;
    for (long l = p.l0; l < p.l1; l += t.lanes) {
        const size_t o = base + (size_t)l * t.C;
        float v[V], d[V], gt[V];
        load<V>(x + o, v);
        load<V>(dy + o, d);
        if (gate) load<V>(gate + o, gt);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float h = (v[e] - mean[e]) * r[e];
            const float dz = d[e] * (gate ? act<IO>(gt[e], silu)
                                          : act_grad<IO>(fmaf(h, ga[e], be[e]), silu).y);
            d[e] = r[e] * (dz * ga[e] - s1[e] - h * s2[e]);
        }
        store<V>(dx + o, d);
    }
}

// ------------------------------------------------------------------ host
constexpr int kSms = 148;

// Registers hold up to 4 vectors of 8 a lane (groups of up to 1024 channels; 2 in the backward),
// or 8 single values (groups of up to 256).
RowShape row_shape(long N, int C, int groups) {
    RowShape s{N, C, groups, C / groups, 0, 1};
    const int V = s.per % 8 == 0 ? 8 : 1;
    s.units = s.per / V;
    while (s.lanes < s.units && s.lanes < 32) s.lanes *= 2;
    return s;
}
int row_units(const RowShape& s) {   // the U of the kernels
    const int need = (s.units + s.lanes - 1) / s.lanes;
    const bool vec = s.per % 8 == 0;
    if (need <= 1) return 1;
    if (need <= 2) return 2;
    if (need <= 4) return 4;
    return !vec && need <= 8 ? 8 : 0;
}
// Row streams of the backward: enough sets of lanes for four CTAs an SM, and no more than rows.
long row_streams(const RowShape& s) {
    const long sets = (long)kSms * 4 * (kThreads / s.lanes);
    const long n = (sets + s.groups - 1) / s.groups;
    return n < 1 ? 1 : n > s.rows ? s.rows : n;
}

Tiling tiling(long N, long L, int C, int groups) {
    Tiling t{N, L, C, groups, C / groups, 0, 0, 0, 0, 0};
    const int V = C % 8 == 0 ? 8 : 1, vecs = C / V;
    t.vecs = vecs < kThreads ? vecs : kThreads;
    t.lanes = kThreads / t.vecs;
    t.ctiles = (vecs + t.vecs - 1) / t.vecs;
    // splits: four CTAs an SM, but at least 8 positions a lane
    const long ctas = N * t.ctiles;
    long want = (4L * kSms + ctas - 1) / ctas;
    const long most = (L + 8L * t.lanes - 1) / (8L * t.lanes);
    if (want > most) want = most;
    if (want < 1) want = 1;
    t.span = (L + want - 1) / want;
    t.splits = (int)((L + t.span - 1) / t.span);
    return t;
}
unsigned tile_ctas(const Tiling& t) { return (unsigned)(t.N * t.splits * t.ctiles); }

size_t r256(size_t x) { return (x + 255) & ~size_t(255); }

template <typename IO, int V, int U>
cudaError_t rows_fwd(const GroupNorm& a, void* y, const RowShape& s, cudaStream_t st) {
    const int per_cta = kThreads / s.lanes;
    const long items = s.rows * s.groups;
    group_norm_rows_kernel<IO, V, U><<<(unsigned)((items + per_cta - 1) / per_cta), kThreads, 0, st>>>(
        (const IO*)a.x, (const IO*)a.gate, a.gamma, a.beta, a.eps, a.silu, (IO*)y, s);
    return cudaGetLastError();
}
template <typename IO, int V, int U>
cudaError_t rows_bwd(const GroupNorm& a, const void* dy, void* dx, void* dgate, float* part,
                     const RowShape& s, cudaStream_t st) {
    const int per_cta = kThreads / s.lanes;
    const long streams = row_streams(s), sets = streams * s.groups;
    group_norm_rows_bwd_kernel<IO, V, U><<<(unsigned)((sets + per_cta - 1) / per_cta), kThreads, 0, st>>>(
        (const IO*)a.x, (const IO*)a.gate, a.gamma, a.beta, a.eps, a.silu, (const IO*)dy, (IO*)dx,
        (IO*)dgate, part, streams, s);
    return cudaGetLastError();
}

template <typename IO>
cudaError_t forward_io(const GroupNorm& a, void* y, void* ws, cudaStream_t st) {
    if (a.L == 1) {
        const RowShape s = row_shape(a.N, a.C, a.groups);
        const int u = row_units(s);
        if (s.per % 8 == 0)
            return u == 1 ? rows_fwd<IO, 8, 1>(a, y, s, st) : u == 2 ? rows_fwd<IO, 8, 2>(a, y, s, st)
                 : u == 4 ? rows_fwd<IO, 8, 4>(a, y, s, st) : rows_fwd<IO, 8, 0>(a, y, s, st);
        return u == 1 ? rows_fwd<IO, 1, 1>(a, y, s, st) : u == 2 ? rows_fwd<IO, 1, 2>(a, y, s, st)
             : u == 4 ? rows_fwd<IO, 1, 4>(a, y, s, st) : u == 8 ? rows_fwd<IO, 1, 8>(a, y, s, st)
             : rows_fwd<IO, 1, 0>(a, y, s, st);
    }
    const Tiling t = tiling(a.N, a.L, a.C, a.groups);
    float2* stats = static_cast<float2*>(ws);
    float2* part = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + r256((size_t)a.N * a.groups * sizeof(float2)));
    const IO* x = (const IO*)a.x;
    if (a.C % 8 == 0) group_norm_stats_kernel<IO, 8><<<tile_ctas(t), kThreads, 0, st>>>(x, part, t);
    else group_norm_stats_kernel<IO, 1><<<tile_ctas(t), kThreads, 0, st>>>(x, part, t);
    group_norm_join_stats_kernel<<<(unsigned)(a.N * a.groups), 128, 0, st>>>(part, stats, a.eps, t);
    if (a.C % 8 == 0)
        group_norm_apply_kernel<IO, 8><<<tile_ctas(t), kThreads, 0, st>>>(
            x, (const IO*)a.gate, a.gamma, a.beta, a.silu, stats, (IO*)y, t);
    else
        group_norm_apply_kernel<IO, 1><<<tile_ctas(t), kThreads, 0, st>>>(
            x, (const IO*)a.gate, a.gamma, a.beta, a.silu, stats, (IO*)y, t);
    return cudaGetLastError();
}

cudaError_t params(const float* part, long rows, int C, float* dgamma, float* dbeta, cudaStream_t st) {
    group_norm_param_kernel<<<(unsigned)((2 * C + 31) / 32), kThreads, 0, st>>>(part, rows, C, dgamma, dbeta);
    return cudaGetLastError();
}

template <typename IO>
cudaError_t backward_io(const GroupNorm& a, const void* dy, void* dx, float* dgamma, float* dbeta,
                        void* dgate, void* ws, cudaStream_t st) {
    if (a.L == 1) {
        const RowShape s = row_shape(a.N, a.C, a.groups);
        const int u = row_units(s);
        float* part = static_cast<float*>(ws);
        cudaError_t e;
        if (s.per % 8 == 0)
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
        return params(part, row_streams(s), a.C, dgamma, dbeta, st);
    }
    const Tiling t = tiling(a.N, a.L, a.C, a.groups);
    const size_t sbytes = r256((size_t)a.N * a.groups * sizeof(float2));
    uint8_t* w = static_cast<uint8_t*>(ws);
    float2* stats = reinterpret_cast<float2*>(w);
    float2* sums = reinterpret_cast<float2*>(w + sbytes);
    float* part = reinterpret_cast<float*>(w + 2 * sbytes);   // statistics, then sums
    const IO *x = (const IO*)a.x, *gate = (const IO*)a.gate, *d = (const IO*)dy;
    const unsigned grid = tile_ctas(t), gn = (unsigned)(a.N * a.groups);
    const bool vec = a.C % 8 == 0;
    if (vec) group_norm_stats_kernel<IO, 8><<<grid, kThreads, 0, st>>>(x, (float2*)part, t);
    else group_norm_stats_kernel<IO, 1><<<grid, kThreads, 0, st>>>(x, (float2*)part, t);
    group_norm_join_stats_kernel<<<gn, 128, 0, st>>>((float2*)part, stats, a.eps, t);
    if (vec)
        group_norm_bwd_sums_kernel<IO, 8><<<grid, kThreads, 0, st>>>(
            x, gate, a.gamma, a.beta, a.silu, stats, d, (IO*)dgate, part, t);
    else
        group_norm_bwd_sums_kernel<IO, 1><<<grid, kThreads, 0, st>>>(
            x, gate, a.gamma, a.beta, a.silu, stats, d, (IO*)dgate, part, t);
    group_norm_join_sums_kernel<<<gn, 128, 0, st>>>(part, a.gamma, sums, t);
    if (vec)
        group_norm_bwd_apply_kernel<IO, 8><<<grid, kThreads, 0, st>>>(
            x, gate, a.gamma, a.beta, a.silu, stats, sums, d, (IO*)dx, t);
    else
        group_norm_bwd_apply_kernel<IO, 1><<<grid, kThreads, 0, st>>>(
            x, gate, a.gamma, a.beta, a.silu, stats, sums, d, (IO*)dx, t);
    if (cudaError_t e = cudaGetLastError()) return e;
    return params(part, a.N * t.splits, a.C, dgamma, dbeta, st);
}

}  // namespace

size_t group_norm_bytes(long N, long L, int C, int groups, bool) {
    if (L == 1) return 0;
    const Tiling t = tiling(N, L, C, groups);
    return r256((size_t)N * groups * sizeof(float2)) + r256((size_t)N * t.splits * C * sizeof(float2));
}

size_t group_norm_backward_bytes(long N, long L, int C, int groups, bool) {
    if (L == 1) return r256((size_t)row_streams(row_shape(N, C, groups)) * 2 * C * sizeof(float));
    const Tiling t = tiling(N, L, C, groups);
    return 2 * r256((size_t)N * groups * sizeof(float2)) + r256((size_t)N * t.splits * C * sizeof(float2));
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
