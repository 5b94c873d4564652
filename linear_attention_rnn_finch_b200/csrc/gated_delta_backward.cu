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
// The fp32 path, where the CUDA cores bound it.  Three launches: what depends on no state,
// parallel over chunks (T, P^T dY, scale (g Q)^T dY); the states S forward and the gradients G
// backward, chains over a head's chunks of three 64 x 64 x 64 products each that need nothing
// of each other, in CTAs of their own; and dQ, dK, db, domega, parallel over chunks.  There a CTA
// has a key head and adds up its value heads in registers; where that would leave SMs without
// one, it has a value head, and a fourth launch adds up dQ and dK of those that share a key head,
// in their order.  No atomics: the same bits every time.
// All products are fp32 FMAs over shared-memory tiles.
#include "common.cuh"
#include "dependent_launch.cuh"
#include "gated_delta.h"
#include "gated_delta_math.cuh"
#include "warp_mma.cuh"

namespace goldwkv {

namespace {

using namespace gdr;

constexpr int kThreads = 256;
constexpr int kLd = C + 4;                    // padded row of a shared-memory tile
constexpr int kTileFloats = C * kLd;
constexpr size_t kMat = (size_t)C * C;        // floats of one 64 x 64 matrix in the workspace

// A thread's results of a product: rows 4 ty + i, columns 4 tx + j, or tx + 16 j where kStr.
template <bool kStr>
__device__ __forceinline__ int col(int tx, int j) { return kStr ? tx + 16 * j : 4 * tx + j; }

template <int kJ>
__device__ __forceinline__ void load_cols(float (&v)[kJ], const float* p) {
    if (kJ == 2) {
        const float2 x = *reinterpret_cast<const float2*>(p);
        v[0] = x.x;
        v[1] = x.y;
    } else {
        const float4 x = *reinterpret_cast<const float4*>(p);
        v[0] = x.x;
        v[1] = x.y;
        v[2 % kJ] = x.z;
        v[3 % kJ] = x.w;
    }
}
template <int kJ>
__device__ __forceinline__ void store_cols(float* p, const float (&v)[kJ]) {
    if (kJ == 2) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    else *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2 % kJ], v[3 % kJ]);
}

// acc += op(A) op(B) over 64 x 64 tiles; B transposed forces the strided columns.  Four k at a time,
// the next four's operands read before these are used: with two warps a scheduler nothing else
// hides shared memory's latency.  Its reads bound a product, 4096 of its cycles for 2048 of FMAs.
template <bool kTA, bool kTB, bool kStr>
__device__ __forceinline__ void mm(float (&acc)[4][4], const float* A, const float* B, int ty, int tx) {
    static_assert(!kTB || kStr, "a transposed B has strided columns");
    static_assert(!(kTA && kTB), "not needed");
    // a[i][e], b[j][e]: k + e
    auto load = [&](int k, float (&a)[4][4], float (&b)[4][4]) {
        if (kTA) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v[4];
                load_cols<4>(v, A + (k + e) * kLd + 4 * ty);
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i][e] = v[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) load_cols<4>(a[i], A + (4 * ty + i) * kLd + k);
        }
        if (kTB) {
#pragma unroll
            for (int j = 0; j < 4; ++j) load_cols<4>(b[j], B + (tx + 16 * j) * kLd + k);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v[4];
                if (kStr) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] = B[(k + e) * kLd + tx + 16 * j];
                } else {
                    load_cols<4>(v, B + (k + e) * kLd + 4 * tx);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j][e] = v[j];
            }
        }
    };
    auto use = [&](const float (&a)[4][4], const float (&b)[4][4]) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i][e], b[j][e], acc[i][j]);
    };
    float a0[4][4], b0[4][4], a1[4][4], b1[4][4];
    load(0, a0, b0);
#pragma unroll 1
    for (int k = 0; k < C; k += 8) {
        load(k + 4, a1, b1);
        use(a0, b0);
        if (k + 8 < C) load(k + 8, a0, b0);
        use(a1, b1);
    }
}

__device__ __forceinline__ void clear(float (&acc)[4][4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
}

// Rows t0 .. t0 + 63 of a token tensor (row stride `step` values) on their way into a tile, rows at
// T or beyond as zeros; landed() waits.  A thread moves 16 channels of one row.
__device__ __forceinline__ void load_tokens(float* tile, const float* base, size_t step, int t0, int T) {
    const int r = threadIdx.x >> 2, c = 16 * (threadIdx.x & 3);
    const bool in = t0 + r < T;
    const uint32_t dst = ptx::smem_addr(tile + r * kLd + c);
    const float* src = base + (in ? (size_t)(t0 + r) * step : 0) + c;
#pragma unroll
    for (int i = 0; i < 16; i += 4) wm::cp_async16(dst + 4 * i, src + i, in);
}
// A 64 x 64 fp32 matrix of the workspace on its way into a tile.
__device__ __forceinline__ void load_matrix(float* tile, const float* src) {
    const int r = threadIdx.x >> 2, c = 16 * (threadIdx.x & 3);
    const uint32_t dst = ptx::smem_addr(tile + r * kLd + c);
#pragma unroll
    for (int i = 0; i < 16; i += 4) wm::cp_async16(dst + 4 * i, src + r * C + c + i, true);
}
__device__ __forceinline__ void landed() {
    wm::cp_async_commit();
    wm::cp_async_wait<0>();
    __syncthreads();
}
__device__ __forceinline__ void store_matrix(float* dst, const float* tile) {
    const int r = threadIdx.x >> 2, c = 16 * (threadIdx.x & 3);
#pragma unroll
    for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(dst + r * C + c + i) = *reinterpret_cast<const float4*>(tile + r * kLd + c + i);
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
    // two results of two rows a thread, four k at a time
    auto product = [&](const float* X, int ldx, const float* Y, int ldy, int m, int r, int c, float (&v)[2][2]) {
        v[0][0] = v[0][1] = v[1][0] = v[1][1] = 0.f;
#pragma unroll 2
        for (int k = 0; k < m; k += 4) {
            float x0[4], x1[4];
            load_cols<4>(x0, X + r * ldx + k);
            load_cols<4>(x1, X + (r + 1) * ldx + k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float y[2];
                load_cols<2>(y, Y + (k + e) * ldy + c);
                v[0][0] = fmaf(x0[e], y[0], v[0][0]);
                v[0][1] = fmaf(x0[e], y[1], v[0][1]);
                v[1][0] = fmaf(x1[e], y[0], v[1][0]);
                v[1][1] = fmaf(x1[e], y[1], v[1][1]);
            }
        }
    };
#pragma unroll
    for (int m = 16; m < C; m *= 2) {
        const int quads = m * m / 4, blk = tid / quads, q = tid - blk * quads, o = 2 * m * blk;
        const int r = 2 * (q / (m / 2)), c = 2 * (q % (m / 2));
        const bool on = blk < C / (2 * m);
        float v[2][2];
        float* t = tmp + blk * m * m;
        if (on) {
            product(A + (o + m) * kLd + o, kLd, T + o * kLd + o, kLd, m, r, c, v);
            store_cols<2>(t + r * m + c, v[0]);
            store_cols<2>(t + (r + 1) * m + c, v[1]);
        }
        __syncthreads();
        if (on) {
            product(T + (o + m) * kLd + o + m, kLd, t, m, m, r, c, v);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float w[2] = {-v[i][0], -v[i][1]};
                store_cols<2>(T + (o + m + r + i) * kLd + o + c, w);
            }
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

// ---- 1: of every chunk T, and (in a CTA of its own) P^T dY and scale (g Q)^T dY
struct LocalSmem {
    float q[kTileFloats], k[kTileFloats], dy[kTileFloats], a[kTileFloats];
    float tmp[32 * 32];
    Gates gates;
};

__global__ void __launch_bounds__(kThreads)
gated_delta_bwd_local_kernel(Args p) {
    extern __shared__ __align__(16) uint8_t raw[];
    LocalSmem& s = *reinterpret_cast<LocalSmem*>(raw);
    const bool inverse = blockIdx.x & 1;
    const int i0 = blockIdx.x >> 1, n = i0 % p.NC, bh = i0 / p.NC;
    const int H = p.in.H, HK = p.in.HK, T = p.in.T, b = bh / H, h = bh - b * H, hk = h / (H / HK);
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15, t0 = n * C;
    const auto gates = fetch_gates((const float*)p.in.omega, (const float*)p.in.beta, (size_t)b * T * H + h, H, t0, T);
    load_tokens(s.k, (const float*)p.in.k + ((size_t)b * T * HK + hk) * C, (size_t)HK * C, t0, T);
    if (!inverse) {
        load_tokens(s.q, (const float*)p.in.q + ((size_t)b * T * HK + hk) * C, (size_t)HK * C, t0, T);
        load_tokens(s.dy, (const float*)p.dy + ((size_t)b * T * H + h) * C, (size_t)H * C, t0, T);
    }
    put_gates(s.gates, gates, t0, T);
    landed();
    const size_t at = ((size_t)bh * p.NC + n) * kMat;
    float acc[4][4];
    clear(acc);
    mm<false, true, true>(acc, inverse ? s.k : s.q, s.k, ty, tx);
    // M b, or P
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = 4 * ty + i, u = col<true>(tx, j);
            const float f = inverse ? s.gates.beta[u] : p.in.scale;
            s.a[t * kLd + u] = t > u || (t == u && !inverse) ? f * acc[i][j] * s.gates.between(t, u) : 0.f;
        }
    if (inverse) {
        __syncthreads();
        invert(s.dy, s.a, s.tmp);
        store_matrix(p.wT + at, s.dy);
        return;
    }
    __syncthreads();   // K Q^T is formed: q <- scale g q
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
    for (int i = 0; i < 4; ++i) store_cols<4>(p.wX + at + (4 * ty + i) * C + 4 * tx, acc[i]);
    clear(acc);
    mm<true, false, false>(acc, s.q, s.dy, ty, tx);
#pragma unroll
    for (int i = 0; i < 4; ++i) store_cols<4>(p.wG + at + (4 * ty + i) * C + 4 * tx, acc[i]);
}

// ---- 2: the states forward, the state gradients backward and dV
// Value columns are independent.  A CTA takes all 64 of a head, 256 threads with 4 x 4 results each,
// or 8 where the CTAs then still have an SM each (up to 9 heads: narrow_chain).  One warp more
// forms the decays a chunk ahead, and the next chunk's operands are on their way in registers
// while one is worked on.  Reads of shared memory bound both: a 16-byte read takes four of its
// cycles even where lanes share addresses.
constexpr int kWork = 256, kChainThreads = kWork + 32;
struct ChainSmem {
    float k[kTileFloats], t[kTileFloats];
    float m[kTileFloats], f[kTileFloats];   // S or G; F, then b to_end E, or b X, then -g dF
    Gates gates[2];
};

// The decays' warp of a chain: `syncs` barriers a chunk, the first of them publishes a chunk's.
template <bool kBack, typename Smem>
__device__ __forceinline__ void chain_gates(Smem& sm, const Args& p, int bh, int syncs, int lane) {
    const int H = p.in.H, T = p.in.T, b = bh / H, h = bh - b * H;
    auto gates = [&](int step) {
        const int t0 = (kBack ? p.NC - 1 - step : step) * C;
        put_gates(sm.gates[step & 1], fetch_gates((const float*)p.in.omega, (const float*)p.in.beta,
                                                  (size_t)b * T * H + h, H, t0, T, lane), t0, T, lane);
    };
    gates(0);
    for (int step = 0; step < p.NC; ++step) {
        __syncthreads();
        if (step + 1 < p.NC) gates(step + 1);
        for (int i = 1; i < syncs; ++i) __syncthreads();
    }
}

template <bool kBack>
__device__ __forceinline__ void chain(ChainSmem& sm, const Args& p, int bh) {
    const int H = p.in.H, HK = p.in.HK, T = p.in.T, b = bh / H, h = bh - b * H, hk = h / (H / HK);
    const int tid = threadIdx.x;
    auto chunk = [&](int step) { return kBack ? p.NC - 1 - step : step; };
    if (tid >= kWork) {
        chain_gates<kBack>(sm, p, bh, 5, tid - kWork);
        return;
    }
    const int ty = tid >> 4, tx = tid & 15, c0 = 4 * tx;
    const float* k = (const float*)p.in.k + ((size_t)b * T * HK + hk) * C;
    const float* v = (const float*)p.in.v + ((size_t)b * T * H + h) * C + c0;
    float* dv = (float*)p.dv + ((size_t)b * T * H + h) * C + c0;
    const size_t head = (size_t)bh * p.NC * kMat;

    // 16 values of a row of K and of T; the thread's own values of V
    constexpr int kLoads = 4;
    const int lr = tid >> 2, lc = 16 * (tid & 3);
    float4 rk[kLoads], rt[kLoads];
    float rv[4][4];
    auto fetch = [&](int n) {
        const int t = n * C + lr;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            rk[i] = t < T ? load4(k + (size_t)t * HK * C + lc + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
            rt[i] = load4(p.wT + head + n * kMat + lr * C + lc + 4 * i);
        }
        if (!kBack) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tv = n * C + 4 * ty + i;
                if (tv < T) {
                    load_cols<4>(rv[i], v + (size_t)tv * H * C);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) rv[i][j] = 0.f;
                }
            }
        }
    };
    float m[4][4];   // rows 4 ty + i of S or G
    const float* from = kBack ? p.ds_out : p.s_in;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (from) {
            load_cols<4>(m[i], from + (size_t)bh * kMat + (4 * ty + i) * C + c0);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) m[i][j] = 0.f;
        }
    }
    fetch(chunk(0));
    for (int step = 0; step < p.NC; ++step) {
        const int n = chunk(step);
        const size_t at = head + n * kMat;
        const Gates& gates = sm.gates[step & 1];
        float x[4][4], y[4][4];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            *reinterpret_cast<float4*>(sm.k + lr * kLd + lc + 4 * i) = rk[i];
            *reinterpret_cast<float4*>(sm.t + lr * kLd + lc + 4 * i) = rt[i];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            store_cols<4>(sm.m + (4 * ty + i) * kLd + 4 * tx, m[i]);
            const size_t o = at + (4 * ty + i) * C + c0;
            if (kBack) {
                load_cols<4>(x[i], p.wX + o);   // P^T dY
                load_cols<4>(y[i], p.wG + o);   // scale (g Q)^T dY, whose place G takes
                store_cols<4>(p.wG + o, m[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) x[i][j] = rv[i][j];
                store_cols<4>(p.wS + o, m[i]);
            }
        }
        __syncthreads();
        if (step + 1 < p.NC) fetch(chunk(step + 1));
        float acc[4][4];
        clear(acc);
        mm<false, false, false>(acc, sm.k, sm.m, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * ty + i;
#pragma unroll
            for (int j = 0; j < 4; ++j)   // F = V - g (K S), or b X = b (P^T dY + Kt G)
                acc[i][j] = kBack ? gates.beta[t] * fmaf(gates.to_end[t], acc[i][j], x[i][j])
                                  : fmaf(-gates.g[t], acc[i][j], x[i][j]);
            store_cols<4>(sm.f + t * kLd + 4 * tx, acc[i]);
        }
        __syncthreads();
        clear(acc);
        mm<kBack, false, false>(acc, sm.t, sm.f, ty, tx);   // E = T F, or dF = T^T (b X)
        __syncthreads();
        const float gc = gates.g[C - 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = 4 * ty + i;
            store_cols<4>((kBack ? p.wX : p.wE) + at + t * C + c0, acc[i]);
            if (kBack && n * C + t < T) store_cols<4>(dv + (size_t)(n * C + t) * H * C, acc[i]);
            const float f = kBack ? -gates.g[t] : gates.beta[t] * gates.to_end[t];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                acc[i][j] *= f;
                m[i][j] = kBack ? fmaf(gc, m[i][j], y[i][j]) : gc * m[i][j];
            }
            store_cols<4>(sm.f + t * kLd + 4 * tx, acc[i]);
        }
        __syncthreads();
        mm<true, false, false>(m, sm.k, sm.f, ty, tx);
        __syncthreads();
    }
    if (kBack && p.ds_in)
#pragma unroll
        for (int i = 0; i < 4; ++i) store_cols<4>(p.ds_in + (size_t)bh * kMat + (4 * ty + i) * C + c0, m[i]);
}

__global__ void __launch_bounds__(kChainThreads)
gated_delta_bwd_chains_f32_kernel(Args p) {
    extern __shared__ __align__(16) uint8_t raw[];
    ChainSmem& s = *reinterpret_cast<ChainSmem*>(raw);
    previous_ended();
    if (blockIdx.x & 1) chain<false>(s, p, blockIdx.x >> 1);
    else chain<true>(s, p, blockIdx.x >> 1);
}

// Eight value columns in a CTA of 512 threads: a chunk takes 4.9 us instead of 9.7, for about four
// times the reads in all.  Four adjacent lanes share four rows of a column, each contracting every
// fourth group of four k, and each is left with one of the rows.
constexpr int kNarrow = 8, kNarrowWork = 512, kNarrowThreads = kNarrowWork + 32;
constexpr int kNarrowLd = 10;   // the four lanes' rows of B, 4 apart, lie 8 banks apart
struct NarrowSmem {
    float k[kTileFloats], t[kTileFloats];
    float m[C * kNarrowLd], f[C * kNarrowLd];
    Gates gates[2];
};

// Row 4 ty + kg of column tx of op(A) B.
template <bool kTA>
__device__ __forceinline__ float narrow_product(const float* A, const float* B, int ty, int tx, int kg) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k0 = 0; k0 < C; k0 += 16) {
        const int k = k0 + 4 * kg;
        float a[4][4];   // [row][k], or [k][row]
#pragma unroll
        for (int i = 0; i < 4; ++i) load_cols<4>(a[i], kTA ? A + (k + i) * kLd + 4 * ty : A + (4 * ty + i) * kLd + k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = B[(k + e) * kNarrowLd + tx];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = fmaf(kTA ? a[e][i] : a[i][e], x, acc[i]);
        }
    }
    // sums over the four lanes, each step handing half of the rows over
    const bool odd = kg & 1, high = kg & 2;
    const float x = (odd ? acc[1] : acc[0]) + __shfl_xor_sync(0xffffffffu, odd ? acc[0] : acc[1], 1);
    const float y = (odd ? acc[3] : acc[2]) + __shfl_xor_sync(0xffffffffu, odd ? acc[2] : acc[3], 1);
    return (high ? y : x) + __shfl_xor_sync(0xffffffffu, high ? x : y, 2);
}

template <bool kBack>
__device__ __forceinline__ void narrow_chain(NarrowSmem& sm, const Args& p, int bh, int cols) {
    const int H = p.in.H, HK = p.in.HK, T = p.in.T, b = bh / H, h = bh - b * H, hk = h / (H / HK);
    const int tid = threadIdx.x;
    auto chunk = [&](int step) { return kBack ? p.NC - 1 - step : step; };
    if (tid >= kNarrowWork) {
        chain_gates<kBack>(sm, p, bh, 5, tid - kNarrowWork);
        return;
    }
    const int kg = tid & 3, tx = (tid >> 2) & 7, ty = tid >> 5, t = 4 * ty + kg;   // its row and column
    const float* k = (const float*)p.in.k + ((size_t)b * T * HK + hk) * C;
    const float* v = (const float*)p.in.v + ((size_t)b * T * H + h) * C + cols + tx;
    float* dv = (float*)p.dv + ((size_t)b * T * H + h) * C + cols + tx;
    const size_t head = (size_t)bh * p.NC * kMat, own = (size_t)t * C + cols + tx;
    const int lr = tid >> 3, lc = 8 * (tid & 7);
    float4 rk[2], rt[2];
    float x, y = 0.f;   // V, or P^T dY and scale (g Q)^T dY
    auto fetch = [&](int n) {
        const size_t at = head + n * kMat;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            rk[i] = n * C + lr < T ? load4(k + (size_t)(n * C + lr) * HK * C + lc + 4 * i) : make_float4(0.f, 0.f, 0.f, 0.f);
            rt[i] = load4(p.wT + at + lr * C + lc + 4 * i);
        }
        if (kBack) {
            x = p.wX[at + own];
            y = p.wG[at + own];
        } else {
            x = n * C + t < T ? v[(size_t)(n * C + t) * H * C] : 0.f;
        }
    };
    const float* from = kBack ? p.ds_out : p.s_in;
    float m = from ? from[(size_t)bh * kMat + own] : 0.f;   // S or G
    fetch(chunk(0));
    for (int step = 0; step < p.NC; ++step) {
        const int n = chunk(step);
        const size_t at = head + n * kMat + own;
        const Gates& gates = sm.gates[step & 1];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            *reinterpret_cast<float4*>(sm.k + lr * kLd + lc + 4 * i) = rk[i];
            *reinterpret_cast<float4*>(sm.t + lr * kLd + lc + 4 * i) = rt[i];
        }
        sm.m[t * kNarrowLd + tx] = m;
        (kBack ? p.wG : p.wS)[at] = m;
        const float xn = x, yn = y;
        __syncthreads();
        if (step + 1 < p.NC) fetch(chunk(step + 1));
        float r = narrow_product<false>(sm.k, sm.m, ty, tx, kg);
        // F = V - g (K S), or b X = b (P^T dY + Kt G)
        sm.f[t * kNarrowLd + tx] = kBack ? gates.beta[t] * fmaf(gates.to_end[t], r, xn) : fmaf(-gates.g[t], r, xn);
        __syncthreads();
        r = narrow_product<kBack>(sm.t, sm.f, ty, tx, kg);   // E = T F, or dF = T^T (b X)
        __syncthreads();
        (kBack ? p.wX : p.wE)[at] = r;
        if (kBack && n * C + t < T) dv[(size_t)(n * C + t) * H * C] = r;
        sm.f[t * kNarrowLd + tx] = r * (kBack ? -gates.g[t] : gates.beta[t] * gates.to_end[t]);
        __syncthreads();
        r = narrow_product<true>(sm.k, sm.f, ty, tx, kg);
        m = fmaf(gates.g[C - 1], m, kBack ? yn + r : r);
        __syncthreads();
    }
    if (kBack && p.ds_in) p.ds_in[(size_t)bh * kMat + own] = m;
}

__global__ void __launch_bounds__(kNarrowThreads)
gated_delta_bwd_narrow_chains_kernel(Args p) {
    __shared__ __align__(16) NarrowSmem s;
    previous_ended();
    constexpr int kParts = C / kNarrow;
    const int i = blockIdx.x >> 1, bh = i / kParts, cols = kNarrow * (i - bh * kParts);
    if (blockIdx.x & 1) narrow_chain<false>(s, p, bh, cols);
    else narrow_chain<true>(s, p, bh, cols);
}

// ---- 3: dQ, dK, dbeta, domega
// Where key heads and chunks do not fill the device, each value head of a shared key head has a CTA
// of its own (`apart`), which leaves its dQ and dK over T and E, and one more launch adds them up:
// B2 T333 H4 over 2 key heads 32 + 6 us instead of 59.
struct OutSmem {
    float q[kTileFloats], k[kTileFloats], dy[kTileFloats], e[kTileFloats], df[kTileFloats];
    float s[kTileFloats], g[kTileFloats], dp[kTileFloats], dm[kTileFloats], w[kTileFloats];
    float cols[16][C];
    float reads[C], kt_eg[C];
    float red[kThreads / 32];
    Gates gates;
};

__global__ void __launch_bounds__(kThreads)
gated_delta_bwd_out_kernel(Args p, bool apart) {
    extern __shared__ __align__(16) uint8_t raw[];
    OutSmem& s = *reinterpret_cast<OutSmem*>(raw);
    const int H = p.in.H, HK = p.in.HK, T = p.in.T, per = H / HK;
    const int n = blockIdx.x % p.NC, i0 = blockIdx.x / p.NC, b = i0 / (apart ? H : HK), j0 = i0 - b * (apart ? H : HK);
    const int h0 = apart ? j0 : j0 * per, h1 = apart ? h0 + 1 : h0 + per, hk = h0 / per;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ty = tid >> 4, tx = tid & 15;
    const int t0 = n * C;
    load_tokens(s.q, (const float*)p.in.q + ((size_t)b * T * HK + hk) * C, (size_t)HK * C, t0, T);
    load_tokens(s.k, (const float*)p.in.k + ((size_t)b * T * HK + hk) * C, (size_t)HK * C, t0, T);
    previous_ended();
    float dq[4][4], dk[4][4];
    clear(dq);
    clear(dk);
    for (int h = h0; h < h1; ++h) {
        const size_t at = ((size_t)(b * H + h) * p.NC + n) * kMat;
        load_tokens(s.dy, (const float*)p.dy + ((size_t)b * T * H + h) * C, (size_t)H * C, t0, T);
        load_matrix(s.e, p.wE + at);
        load_matrix(s.df, p.wX + at);
        load_matrix(s.s, p.wS + at);
        load_matrix(s.g, p.wG + at);
        load_gates(s.gates, (const float*)p.in.omega, (const float*)p.in.beta, (size_t)b * T * H + h, H, t0, T);
        landed();
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
        // column sums of W from each row down: four lanes a column, 16 rows each
        const int x = tid >> 2, part = tid & 3, first = 16 * part;
        {
            float c = 0.f;
#pragma unroll
            for (int i = 15; i >= 0; --i) c += s.w[(first + i) * kLd + x];
            float below = 0.f;   // the lanes' after this one
#pragma unroll
            for (int o = 1; o < 4; ++o) {
                const float y = __shfl_down_sync(0xffffffffu, c, o, 4);
                if (part + o < 4) below += y;
            }
#pragma unroll
            for (int i = 15; i >= 0; --i) s.w[(first + i) * kLd + x] = below += s.w[(first + i) * kLd + x];
        }
        __syncthreads();
        {   // four lanes a token: the columns before it, the sources before it, the reads from it on
            float sum = 0.f, db = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int u = first + i;
                sum += u < x ? s.w[x * kLd + u] : 0.f;
                sum = u < x ? fmaf(s.gates.beta[u], s.kt_eg[u], sum) : sum + s.reads[u];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) db += s.cols[4 * part + i][x];
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
                db += __shfl_xor_sync(0xffffffffu, db, o);
            }
            if (part == 0 && t0 + x < T) {
                float gsum = 0.f;
                for (int i = 0; i < kThreads / 32; ++i) gsum += s.red[i];
                const float dl = sum + s.gates.g[C - 1] * gsum;
                const size_t o = (size_t)b * T * H + h + (size_t)(t0 + x) * H;
                ((float*)p.domega)[o] = -s.gates.rate[x] * dl;
                ((float*)p.dbeta)[o] = s.kt_eg[x] + db;
            }
        }
        __syncthreads();
    }
    if (apart) {
        const size_t at = ((size_t)(b * H + h0) * p.NC + n) * kMat;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                p.wT[at + (4 * ty + i) * C + col<true>(tx, j)] = dq[i][j];
                p.wE[at + (4 * ty + i) * C + col<true>(tx, j)] = dk[i][j];
            }
        return;
    }
    float* oq = (float*)p.dq + ((size_t)b * T * HK + hk) * C;
    float* ok = (float*)p.dk + ((size_t)b * T * HK + hk) * C;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int t = t0 + 4 * ty + i;
        if (t >= T) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            oq[(size_t)t * HK * C + col<true>(tx, j)] = dq[i][j];
            ok[(size_t)t * HK * C + col<true>(tx, j)] = dk[i][j];
        }
    }
}

__global__ void __launch_bounds__(kThreads)
gated_delta_bwd_heads_kernel(Args p) {   // four values a thread, four CTAs a chunk
    const int H = p.in.H, HK = p.in.HK, T = p.in.T, per = H / HK, i = 4 * ((blockIdx.x & 3) * kThreads + threadIdx.x);
    const int i0 = blockIdx.x >> 2, n = i0 % p.NC, bk = i0 / p.NC, b = bk / HK, hk = bk - b * HK, t = n * C + (i >> 6);
    previous_ended();
    if (t >= T) return;
    const size_t first = ((size_t)(b * H + hk * per) * p.NC + n) * kMat + i, step = (size_t)p.NC * kMat;
    float q[4] = {0.f, 0.f, 0.f, 0.f}, k[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int h = 0; h < per; ++h) {
        float x[4], y[4];
        load_cols<4>(x, p.wT + first + h * step);
        load_cols<4>(y, p.wE + first + h * step);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            q[e] += x[e];
            k[e] += y[e];
        }
    }
    const size_t o = (((size_t)b * T + t) * HK + hk) * C + (i & 63);
    store_cols<4>((float*)p.dq + o, q);
    store_cols<4>((float*)p.dk + o, k);
}

template <typename Kernel, typename... More>
cudaError_t run(bool first, Kernel kernel, unsigned grid, int threads, size_t smem, const Args& a, cudaStream_t st,
                More... more) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (!first) return launch_next(kernel, grid, threads, smem, st, a, more...);
    kernel<<<grid, threads, smem, st>>>(a, more...);
    return cudaGetLastError();
}

constexpr int kSms = 148;

}  // namespace

size_t gdr_backward_f32_bytes(int B, int T, int H) {
    return 5 * (size_t)B * H * ((T + C - 1) / C) * kMat * sizeof(float);
}

cudaError_t launch_gdr_backward_f32(const GdrIn& in, const float* s_in, const GdrGrads& g,
                                    void* ws, cudaStream_t st) {
    const int NC = (in.T + C - 1) / C;
    const size_t each = (size_t)in.B * in.H * NC * kMat;
    float* w = static_cast<float*>(ws);
    const Args a{in, g.dy, s_in, g.ds_out, g.ds_in, g.dq, g.dk, g.dv, g.domega, g.dbeta,
                 w, w + each, w + 2 * each, w + 3 * each, w + 4 * each, NC};
    const unsigned heads = (unsigned)(in.B * in.H);
    cudaError_t e = run(true, gated_delta_bwd_local_kernel, 2 * heads * NC, kThreads, sizeof(LocalSmem), a, st);
    if (e != cudaSuccess) return e;
    if (2 * heads * (C / kNarrow) <= (unsigned)kSms)
        e = run(false, gated_delta_bwd_narrow_chains_kernel, 2 * heads * (C / kNarrow), kNarrowThreads, 0, a, st);
    else
        e = run(false, gated_delta_bwd_chains_f32_kernel, 2 * heads, kChainThreads, sizeof(ChainSmem), a, st);
    if (e != cudaSuccess) return e;
    const unsigned groups = (unsigned)(in.B * in.HK) * (unsigned)NC;
    const bool apart = in.H > in.HK && groups < (unsigned)kSms;
    e = run(false, gated_delta_bwd_out_kernel, apart ? heads * NC : groups, kThreads, sizeof(OutSmem), a, st, apart);
    if (e != cudaSuccess || !apart) return e;
    return run(false, gated_delta_bwd_heads_kernel, 4 * groups, kThreads, 0, a, st);
}

}  // namespace goldwkv
