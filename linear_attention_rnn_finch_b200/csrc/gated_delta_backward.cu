// Backward of the gated delta rule on CUDA cores in fp32, chunk by chunk (sm_100a).
//
// A chunk of 64 tokens entering with state S, L_t the sum of log w up to t inside it,
// g = e^L, D_ts = e^(L_t - L_s) <= 1 for t >= s, b the write strengths as a diagonal matrix:
//     M = strictly lower (K K^T . D),   T = (I + M b)^-1,   F = V - g (K S),   E = T F,
//     V' = b E,   P = scale lower (Q K^T . D),   Y = scale g (Q S) + P V',
//     S+ = g_C S + Kt^T V',   Kt_s = (g_C / g_s) k_s.
// With G the gradient of S+ and dY that of Y:
//     X = P^T dY + Kt G,   dF = T^T (b X) = dV,
//     G- = g_C G + scale (g Q)^T dY - (g K)^T dF,
//     dQ = scale g (dY S^T) + dP K,              dP = scale lower (dY V'^T . D),
//     dK = dP^T Q + b (g_C / g) (E G^T) - g (dF S^T) + (dM + dM^T) K,
//                                                dM = -strictly lower (dF V'^T . D),
//     db_s = sum_t P_ts dY_t.E_s - sum_t M_ts dF_t.E_s + kt_s . (E G^T)_s
// (every product of db taken with E = V' / b, so that b = 0 needs no division).
// The decay's gradient sums every pair of a reader at t or after it and a source before it,
// whose weight holds w_t; a difference of running sums would cancel where w_t is small:
//     dlog w_t = sum_{tau >= t, s < t} (P . dY V'^T - M . dF V'^T)_{tau s}
//              + sum_{tau >= t} g_tau (scale q_tau . (S dY_tau) - k_tau . (S dF_tau))
//              + sum_{s < t} V'_s . (Kt G)_s + g_C <G, S>,
//     domega_t = -exp(omega_t) dlog w_t.
//
// Four launches: what depends on no state, parallel over chunks (T, P^T dY, scale (g Q)^T dY);
// the states S forward; the gradients G backward, each a chain over a head's chunks of three
// 64 x 64 x 64 products; and dQ, dK, db, domega, parallel over chunks, a CTA per key head
// that adds up its value heads in registers (no atomics: the same bits every time).  All
// products are fp32 FMAs over shared-memory tiles, a thread 4 x 4 of the 64 x 64 results:
// this is the fp32 path, where the CUDA cores bound it.
#include "common.cuh"
#include "gated_delta.h"
#include "gated_delta_math.cuh"

namespace goldwkv {

namespace {

using namespace gdr;

constexpr int kThreads = 256;
constexpr int kLd = C + 4;                    // padded row of a shared-memory tile
constexpr int kTileFloats = C * kLd;
constexpr size_t kMat = (size_t)C * C;        // floats of one 64 x 64 matrix in the workspace

// Results of a product: rows 4 ty + i, columns 4 tx + j, or tx + 16 j where kStr.
template <bool kStr>
__device__ __forceinline__ int col(int tx, int j) { return kStr ? tx + 16 * j : 4 * tx + j; }

// acc += op(A) op(B) over 64 x 64 tiles; B transposed forces the strided columns.
template <bool kTA, bool kTB, bool kStr>
__device__ __forceinline__ void mm(float (&acc)[4][4], const float* A, const float* B, int ty, int tx) {
    static_assert(!kTB || kStr, "a transposed B has strided columns");
    static_assert(!(kTA && kTB), "not needed");
#pragma unroll 2
    for (int k = 0; k < C; k += 4) {
        float4 a[4];
        if (!kTA) {
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (4 * ty + i) * kLd + k);
        }
        if (kTB) {
            float4 b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * kLd + k);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, acc[i][j]))));
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float av[4], bv[4];
                if (kTA) {
                    const float4 x = *reinterpret_cast<const float4*>(A + (k + e) * kLd + 4 * ty);
                    av[0] = x.x; av[1] = x.y; av[2] = x.z; av[3] = x.w;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) av[i] = e == 0 ? a[i].x : e == 1 ? a[i].y : e == 2 ? a[i].z : a[i].w;
                }
                if (kStr) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) bv[j] = B[(k + e) * kLd + tx + 16 * j];
                } else {
                    const float4 x = *reinterpret_cast<const float4*>(B + (k + e) * kLd + 4 * tx);
                    bv[0] = x.x; bv[1] = x.y; bv[2] = x.z; bv[3] = x.w;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
            }
        }
    }
}

__device__ __forceinline__ void clear(float (&acc)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
}

// Rows t0 .. t0 + 63 of a token tensor (row stride `step` elements) into a tile, rows at T or
// beyond as zeros.  A thread moves 16 channels of one row.
template <typename IO>
__device__ __forceinline__ void load_tokens(float* tile, const IO* base, size_t step, int t0, int T) {
    const int r = threadIdx.x >> 2, c = 16 * (threadIdx.x & 3);
    float* dst = tile + r * kLd + c;
    if (t0 + r < T) {
        const IO* src = base + (size_t)(t0 + r) * step + c;
#pragma unroll
        for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4*>(dst + i) = load4(src + i);
    } else {
#pragma unroll
        for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4*>(dst + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
}
// A 64 x 64 fp32 matrix of the workspace into a tile (null: zeros).
__device__ __forceinline__ void load_matrix(float* tile, const float* src) {
    const int r = threadIdx.x >> 2, c = 16 * (threadIdx.x & 3);
#pragma unroll
    for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(tile + r * kLd + c + i) =
            src ? *reinterpret_cast<const float4*>(src + r * C + c + i) : make_float4(0.f, 0.f, 0.f, 0.f);
}
__device__ __forceinline__ void store_matrix(float* dst, const float* tile) {
    const int r = threadIdx.x >> 2, c = 16 * (threadIdx.x & 3);
#pragma unroll
    for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(dst + r * C + c + i) = *reinterpret_cast<const float4*>(tile + r * kLd + c + i);
}
__device__ __forceinline__ void store_acc(float* tile, const float (&acc)[4][4], int ty, int tx) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(tile + (4 * ty + i) * kLd + 4 * tx) =
            make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
}

// T = (I + A)^-1 of the strictly lower triangular tile A: each 16 x 16 diagonal block by
// substitution, a warp a block and a lane a column; then blocks of twice the size from
// T21 = -T22 (A21 T11).  Substitution, not a power series: every entry of T stays bounded
// where keys are alike, while the powers of A grow and cancel.
__device__ void invert(float* T, const float* A, float* tmp) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < kTileFloats; i += kThreads) T[i] = 0.f;
    __syncthreads();
    if (warp < 4 && lane < 16) {
        const int o = 16 * warp;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float v = i == lane ? 1.f : 0.f;
#pragma unroll
            for (int s = 0; s < i; ++s) v = fmaf(-A[(o + i) * kLd + o + s], x[s], v);
            x[i] = v;
            T[(o + i) * kLd + o + lane] = v;
        }
    }
    __syncthreads();
#pragma unroll
    for (int m = 16; m < C; m *= 2) {
        const int blocks = C / (2 * m), n = blocks * m * m;
        for (int i = tid; i < n; i += kThreads) {
            const int blk = i / (m * m), r = (i / m) % m, c = i % m, o = 2 * m * blk;
            float v = 0.f;
            for (int k = 0; k < m; ++k) v = fmaf(A[(o + m + r) * kLd + o + k], T[(o + k) * kLd + o + c], v);
            tmp[i] = v;
        }
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
            const int blk = i / (m * m), r = (i / m) % m, c = i % m, o = 2 * m * blk;
            float v = 0.f;
            for (int k = 0; k < m; ++k) v = fmaf(T[(o + m + r) * kLd + o + m + k], tmp[blk * m * m + k * m + c], v);
            T[(o + m + r) * kLd + o + c] = -v;
        }
        __syncthreads();
    }
}

struct Args {
    GdrIn in;
    const void* dy;
    const float* s_in;
    const float* ds_out;
    float* ds_in;
    void* dq;
    void* dk;
    void* dv;
    void* domega;
    void* dbeta;
    float* wT;   // per (head, chunk), kMat floats each: T
    float* wX;   // P^T dY, then dF
    float* wG;   // scale (g Q)^T dY, then G
    float* wS;   // the state entering the chunk
    float* wE;   // E
    int NC;
};

// ---- 1: T, P^T dY and scale (g Q)^T dY of every chunk
struct LocalSmem {
    float q[kTileFloats], k[kTileFloats], dy[kTileFloats], a[kTileFloats], t[kTileFloats];
    float tmp[32 * 32];
    Gates gates;
};

template <typename IO>
__global__ void __launch_bounds__(kThreads)
gated_delta_bwd_local_kernel(Args p) {
    extern __shared__ __align__(16) uint8_t raw[];
    LocalSmem& s = *reinterpret_cast<LocalSmem*>(raw);
    const int n = blockIdx.x % p.NC, bh = blockIdx.x / p.NC;
    const int H = p.in.H, HK = p.in.HK, T = p.in.T, b = bh / H, h = bh - b * H, hk = h / (H / HK);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, t0 = n * C;
    load_tokens(s.q, (const IO*)p.in.q + ((size_t)b * T * HK + hk) * C, (size_t)HK * C, t0, T);
    load_tokens(s.k, (const IO*)p.in.k + ((size_t)b * T * HK + hk) * C, (size_t)HK * C, t0, T);
    load_tokens(s.dy, (const IO*)p.dy + ((size_t)b * T * H + h) * C, (size_t)H * C, t0, T);
    load_gates(s.gates, (const IO*)p.in.omega, (const IO*)p.in.beta, (size_t)b * T * H + h, H, t0, T);
    __syncthreads();
    float acc[4][4];
    clear(acc);
    mm<false, true, true>(acc, s.k, s.k, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = 4 * ty + i, u = col<true>(tx, j);
            s.a[t * kLd + u] = t > u ? acc[i][j] * s.gates.between(t, u) * s.gates.beta[u] : 0.f;
        }
    __syncthreads();
    invert(s.t, s.a, s.tmp);
    const size_t at = ((size_t)bh * p.NC + n) * kMat;
    store_matrix(p.wT + at, s.t);
    clear(acc);
    mm<false, true, true>(acc, s.q, s.k, ty, tx);
    __syncthreads();   // A's last use was in invert
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = 4 * ty + i, u = col<true>(tx, j);
            s.a[t * kLd + u] = t >= u ? p.in.scale * acc[i][j] * s.gates.between(t, u) : 0.f;
        }
    // q <- scale g q
    {
        const int r = tid >> 2, c = 16 * (tid & 3);
        const float f = p.in.scale * s.gates.g[r];
#pragma unroll
        for (int i = 0; i < 16; ++i) s.q[r * kLd + c + i] *= f;
    }
    __syncthreads();
    clear(acc);
    mm<true, false, false>(acc, s.a, s.dy, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(p.wX + at + (4 * ty + i) * C + 4 * tx) =
            make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
    clear(acc);
    mm<true, false, false>(acc, s.q, s.dy, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(p.wG + at + (4 * ty + i) * C + 4 * tx) =
            make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
}

// ---- 2: the states, forward
struct StateSmem {
    float k[kTileFloats], s[kTileFloats], f[kTileFloats], t[kTileFloats];
    Gates gates;
};

template <typename IO>
__global__ void __launch_bounds__(kThreads)
gated_delta_bwd_states_kernel(Args p) {
    extern __shared__ __align__(16) uint8_t raw[];
    StateSmem& s = *reinterpret_cast<StateSmem*>(raw);
    const int bh = blockIdx.x;
    const int H = p.in.H, HK = p.in.HK, T = p.in.T, b = bh / H, h = bh - b * H, hk = h / (H / HK);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    load_matrix(s.s, p.s_in ? p.s_in + (size_t)bh * kMat : nullptr);
    for (int n = 0; n < p.NC; ++n) {
        const size_t at = ((size_t)bh * p.NC + n) * kMat;
        load_tokens(s.k, (const IO*)p.in.k + ((size_t)b * T * HK + hk) * C, (size_t)HK * C, n * C, T);
        load_tokens(s.f, (const IO*)p.in.v + ((size_t)b * T * H + h) * C, (size_t)H * C, n * C, T);
        load_matrix(s.t, p.wT + at);
        load_gates(s.gates, (const IO*)p.in.omega, (const IO*)p.in.beta, (size_t)b * T * H + h, H, n * C, T);
        __syncthreads();
        store_matrix(p.wS + at, s.s);
        float acc[4][4];
        clear(acc);
        mm<false, false, false>(acc, s.k, s.s, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {   // F = V - g (K S), each element its own thread's
                float* f = &s.f[(4 * ty + i) * kLd + 4 * tx + j];
                *f = fmaf(-s.gates.g[4 * ty + i], acc[i][j], *f);
            }
        __syncthreads();
        clear(acc);
        mm<false, false, false>(acc, s.t, s.f, ty, tx);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * ty + i;
            *reinterpret_cast<float4*>(p.wE + at + t * C + 4 * tx) =
                make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
            const float f = s.gates.beta[t] * s.gates.to_end[t];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] *= f;
        }
        store_acc(s.f, acc, ty, tx);
        __syncthreads();
        const float gc = s.gates.g[C - 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(&s.s[(4 * ty + i) * kLd + 4 * tx]);
            acc[i][0] = gc * x.x;
            acc[i][1] = gc * x.y;
            acc[i][2] = gc * x.z;
            acc[i][3] = gc * x.w;
        }
        mm<true, false, false>(acc, s.k, s.f, ty, tx);
        store_acc(s.s, acc, ty, tx);
        __syncthreads();
    }
}

// ---- 3: the state gradients, backward; dV
struct GradStateSmem {
    float k[kTileFloats], g[kTileFloats], x[kTileFloats], t[kTileFloats];
    Gates gates;
};

template <typename IO>
__global__ void __launch_bounds__(kThreads)
gated_delta_bwd_state_grads_kernel(Args p) {
    extern __shared__ __align__(16) uint8_t raw[];
    GradStateSmem& s = *reinterpret_cast<GradStateSmem*>(raw);
    const int bh = blockIdx.x;
    const int H = p.in.H, HK = p.in.HK, T = p.in.T, b = bh / H, h = bh - b * H, hk = h / (H / HK);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    IO* dv = (IO*)p.dv + ((size_t)b * T * H + h) * C;
    load_matrix(s.g, p.ds_out ? p.ds_out + (size_t)bh * kMat : nullptr);
    for (int n = p.NC - 1; n >= 0; --n) {
        const size_t at = ((size_t)bh * p.NC + n) * kMat;
        load_tokens(s.k, (const IO*)p.in.k + ((size_t)b * T * HK + hk) * C, (size_t)HK * C, n * C, T);
        load_matrix(s.t, p.wT + at);
        load_gates(s.gates, (const IO*)p.in.omega, (const IO*)p.in.beta, (size_t)b * T * H + h, H, n * C, T);
        __syncthreads();
        float acc[4][4], into[4][4];
        clear(acc);
        mm<false, false, false>(acc, s.k, s.g, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // b X = b (P^T dY + Kt G)
            const int t = 4 * ty + i;
            const float4 x = *reinterpret_cast<const float4*>(p.wX + at + t * C + 4 * tx);
            const float e = s.gates.to_end[t], bt = s.gates.beta[t];
            acc[i][0] = bt * fmaf(e, acc[i][0], x.x);
            acc[i][1] = bt * fmaf(e, acc[i][1], x.y);
            acc[i][2] = bt * fmaf(e, acc[i][2], x.z);
            acc[i][3] = bt * fmaf(e, acc[i][3], x.w);
            // scale (g Q)^T dY, whose place G takes
            float4* gp = reinterpret_cast<float4*>(p.wG + at + t * C + 4 * tx);
            const float4 y = *gp;
            const float4 G = *reinterpret_cast<const float4*>(&s.g[t * kLd + 4 * tx]);
            *gp = G;
            const float gc = s.gates.g[C - 1];
            into[i][0] = fmaf(gc, G.x, y.x);
            into[i][1] = fmaf(gc, G.y, y.y);
            into[i][2] = fmaf(gc, G.z, y.z);
            into[i][3] = fmaf(gc, G.w, y.w);
        }
        store_acc(s.x, acc, ty, tx);
        __syncthreads();
        clear(acc);
        mm<true, false, false>(acc, s.t, s.x, ty, tx);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * ty + i;
            *reinterpret_cast<float4*>(p.wX + at + t * C + 4 * tx) =
                make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
            if (n * C + t < T) store4(dv + (size_t)(n * C + t) * H * C + 4 * tx, acc[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] *= -s.gates.g[t];
        }
        store_acc(s.x, acc, ty, tx);
        __syncthreads();
        mm<true, false, false>(into, s.k, s.x, ty, tx);
        store_acc(s.g, into, ty, tx);
        __syncthreads();
    }
    if (p.ds_in) store_matrix(p.ds_in + (size_t)bh * kMat, s.g);
}

// ---- 4: dQ, dK, dbeta, domega
struct OutSmem {
    float q[kTileFloats], k[kTileFloats], dy[kTileFloats], e[kTileFloats], df[kTileFloats];
    float s[kTileFloats], g[kTileFloats], dp[kTileFloats], dm[kTileFloats], w[kTileFloats];
    float cols[16][C];
    float reads[C], kt_eg[C];
    float red[kThreads / 32];
    Gates gates;
};

template <typename IO>
__global__ void __launch_bounds__(kThreads)
gated_delta_bwd_out_kernel(Args p) {
    extern __shared__ __align__(16) uint8_t raw[];
    OutSmem& s = *reinterpret_cast<OutSmem*>(raw);
    const int n = blockIdx.x % p.NC, bk = blockIdx.x / p.NC;
    const int H = p.in.H, HK = p.in.HK, T = p.in.T, b = bk / HK, hk = bk - b * HK, per = H / HK;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ty = tid >> 4, tx = tid & 15;
    const int t0 = n * C;
    load_tokens(s.q, (const IO*)p.in.q + ((size_t)b * T * HK + hk) * C, (size_t)HK * C, t0, T);
    load_tokens(s.k, (const IO*)p.in.k + ((size_t)b * T * HK + hk) * C, (size_t)HK * C, t0, T);
    float dq[4][4], dk[4][4];
    clear(dq);
    clear(dk);
    for (int h = hk * per; h < (hk + 1) * per; ++h) {
        const size_t at = ((size_t)(b * H + h) * p.NC + n) * kMat;
        load_tokens(s.dy, (const IO*)p.dy + ((size_t)b * T * H + h) * C, (size_t)H * C, t0, T);
        load_matrix(s.e, p.wE + at);
        load_matrix(s.df, p.wX + at);
        load_matrix(s.s, p.wS + at);
        load_matrix(s.g, p.wG + at);
        load_gates(s.gates, (const IO*)p.in.omega, (const IO*)p.in.beta, (size_t)b * T * H + h, H, t0, T);
        __syncthreads();
        float acc[4][4], bcc[4][4], w[4][4], cs[4] = {0.f, 0.f, 0.f, 0.f};
        clear(acc);
        clear(bcc);
        mm<false, true, true>(acc, s.q, s.k, ty, tx);
        mm<false, true, true>(bcc, s.dy, s.e, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 4 * ty + i, u = col<true>(tx, j);
                const float d = t >= u ? p.in.scale * s.gates.between(t, u) : 0.f;
                const float x = t >= u ? bcc[i][j] * d * acc[i][j] : 0.f;   // P_ts dY_t . E_s
                cs[j] += x;
                w[i][j] = t > u ? s.gates.beta[u] * x : 0.f;
                s.dp[t * kLd + u] = t >= u ? d * s.gates.beta[u] * bcc[i][j] : 0.f;
            }
        clear(acc);
        clear(bcc);
        mm<false, true, true>(acc, s.k, s.k, ty, tx);
        mm<false, true, true>(bcc, s.df, s.e, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = 4 * ty + i, u = col<true>(tx, j);
                const float d = t > u ? s.gates.between(t, u) : 0.f;
                const float x = t > u ? bcc[i][j] * d * acc[i][j] : 0.f;    // M_ts dF_t . E_s
                cs[j] -= x;
                s.w[t * kLd + u] = t > u ? fmaf(-s.gates.beta[u], x, w[i][j]) : 0.f;
                const float m = t > u ? -d * s.gates.beta[u] * bcc[i][j] : 0.f;
                if (t >= u) s.dm[t * kLd + u] = m;   // dM + dM^T, symmetric
                if (t > u) s.dm[u * kLd + t] = m;
            }
#pragma unroll
        for (int j = 0; j < 4; ++j) s.cols[ty][col<true>(tx, j)] = cs[j];
        // <G, S>
        float gs = 0.f;
        for (int i = tid; i < C * C; i += kThreads) {
            const int o = (i >> 6) * kLd + (i & 63);
            gs = fmaf(s.g[o], s.s[o], gs);
        }
        gs = warp_sum(gs);
        if (lane == 0) s.red[warp] = gs;
        __syncthreads();
        mm<false, false, true>(dq, s.dp, s.k, ty, tx);
        mm<true, false, true>(dk, s.dp, s.q, ty, tx);
        mm<false, false, true>(dk, s.dm, s.k, ty, tx);
        clear(acc);
        mm<false, true, true>(acc, s.dy, s.s, ty, tx);
        float rd[4], ke[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * ty + i;
            const float f = p.in.scale * s.gates.g[t];
            rd[i] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = f * acc[i][j];
                dq[i][j] += x;
                rd[i] = fmaf(s.q[t * kLd + col<true>(tx, j)], x, rd[i]);
            }
        }
        clear(acc);
        mm<false, true, true>(acc, s.df, s.s, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * ty + i;
            const float f = s.gates.g[t];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = f * acc[i][j];
                dk[i][j] -= x;
                rd[i] = fmaf(-s.k[t * kLd + col<true>(tx, j)], x, rd[i]);
            }
        }
        clear(acc);
        mm<false, true, true>(acc, s.e, s.g, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * ty + i;
            const float f = s.gates.to_end[t];
            ke[i] = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = f * acc[i][j];
                dk[i][j] = fmaf(s.gates.beta[t], x, dk[i][j]);
                ke[i] = fmaf(s.k[t * kLd + col<true>(tx, j)], x, ke[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) {
                rd[i] += __shfl_xor_sync(0xffffffffu, rd[i], o);
                ke[i] += __shfl_xor_sync(0xffffffffu, ke[i], o);
            }
            if (tx == 0) {
                s.reads[4 * ty + i] = rd[i];
                s.kt_eg[4 * ty + i] = ke[i];
            }
        }
        // column sums of W from each row down
        if (tid < C) {
            float c = 0.f;
            for (int t = C - 1; t > tid; --t) s.w[t * kLd + tid] = c += s.w[t * kLd + tid];
        }
        __syncthreads();
        if (tid < C && t0 + tid < T) {
            const int t = tid;
            float db = s.kt_eg[t];
#pragma unroll
            for (int i = 0; i < 16; ++i) db += s.cols[i][t];
            float pairs = 0.f, rs = 0.f, src = 0.f, gsum = 0.f;
            for (int u = 0; u < t; ++u) {
                pairs += s.w[t * kLd + u];
                src = fmaf(s.gates.beta[u], s.kt_eg[u], src);
            }
            for (int u = C - 1; u >= t; --u) rs += s.reads[u];
            for (int i = 0; i < kThreads / 32; ++i) gsum += s.red[i];
            const float dl = ((pairs + rs) + src) + s.gates.g[C - 1] * gsum;
            const size_t o = (size_t)b * T * H + h + (size_t)(t0 + t) * H;
            ((IO*)p.domega)[o] = from_f32<IO>(-s.gates.rate[t] * dl);
            ((IO*)p.dbeta)[o] = from_f32<IO>(db);
        }
        __syncthreads();
    }
    IO* oq = (IO*)p.dq + ((size_t)b * T * HK + hk) * C;
    IO* ok = (IO*)p.dk + ((size_t)b * T * HK + hk) * C;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + 4 * ty + i;
        if (t >= T) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            oq[(size_t)t * HK * C + col<true>(tx, j)] = from_f32<IO>(dq[i][j]);
            ok[(size_t)t * HK * C + col<true>(tx, j)] = from_f32<IO>(dk[i][j]);
        }
    }
}

template <typename Kernel>
cudaError_t run(Kernel kernel, unsigned grid, size_t smem, const Args& a, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename IO>
cudaError_t backward_io(const Args& a, cudaStream_t st) {
    const unsigned heads = (unsigned)(a.in.B * a.in.H), chunks = heads * (unsigned)a.NC;
    cudaError_t e = run(gated_delta_bwd_local_kernel<IO>, chunks, sizeof(LocalSmem), a, st);
    if (e == cudaSuccess) e = run(gated_delta_bwd_states_kernel<IO>, heads, sizeof(StateSmem), a, st);
    if (e == cudaSuccess) e = run(gated_delta_bwd_state_grads_kernel<IO>, heads, sizeof(GradStateSmem), a, st);
    if (e == cudaSuccess)
        e = run(gated_delta_bwd_out_kernel<IO>, (unsigned)(a.in.B * a.in.HK) * (unsigned)a.NC, sizeof(OutSmem), a, st);
    return e;
}

}  // namespace

size_t gdr_backward_simt_bytes(int B, int T, int H) {
    return 5 * (size_t)B * H * ((T + C - 1) / C) * kMat * sizeof(float);
}

cudaError_t launch_gdr_backward_simt(const GdrIn& in, const float* s_in, const GdrGrads& g,
                                     void* ws, bool bf16, cudaStream_t st) {
    const int NC = (in.T + C - 1) / C;
    const size_t each = (size_t)in.B * in.H * NC * kMat;
    float* w = static_cast<float*>(ws);
    const Args a{in, g.dy, s_in, g.ds_out, g.ds_in, g.dq, g.dk, g.dv, g.domega, g.dbeta,
                 w, w + each, w + 2 * each, w + 3 * each, w + 4 * each, NC};
    return bf16 ? backward_io<__nv_bfloat16>(a, st) : backward_io<float>(a, st);
}

}  // namespace goldwkv
