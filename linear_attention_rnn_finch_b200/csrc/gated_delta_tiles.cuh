// What the tensor-core kernels of the gated delta rule share: loading blocks of 64 tokens and
// preparing what depends on no state.
//
// A block is cut into sub-chunks of 16 tokens.  Inside one, with L_t the sum of log w up to t,
// g = e^L, D_ts = e^(L_t - L_s) <= 1 for t >= s, and the entering state S (64 x 64):
//     M = strictly lower (K K^T . D),  T = (I + M b)^-1,  P = scale lower (Q K^T . D),
//     F = V - g (K S),  E = T F,  Y = scale g (Q S) + P (b E),
//     S+ = g_16 S + K^T (b to_end E),   to_end_t = e^(L_16 - L_t).
// 16, not 64: the products with S, Q S, K^T E cost the same per token whatever the length of a
// sub-chunk, while those with T and P and the inverse grow with it (per 64 tokens and 16 value
// columns and in two parts 240 matrix instructions instead of 312, an inverse without block
// products).
//
// Four warps (the chain) own 16 value columns each and keep S^T in registers as accumulators
// (rows value columns, columns key channels; two warps of 32 columns issue less in all, but leave
// schedulers idle: B8 T4096 H32 423 us against 289).  Everything transposed (F^T = V^T - g S^T K^T,
// E^T = F^T T^T, ...), each result has the layout of the next product's A operand, so a block
// passes through them without shared memory or barriers between its products.  Four more warps
// (the preparation) work one block ahead: they issue the copies of the block after it, and
// form decays, T and P of one sub-chunk each.  The two halves meet once a block.
//
// Operands that are not the caller's bf16 values are kept as sums of bf16 parts.  Three (2^-25 of
// the value) for what comes back in the fp32 state: S against K, T, F and the terms added to S,
// whose products are summed on their own and added to S by FMAs.  The state is then as exact as
// fp32 sums make it: off by 1e-7 to 3e-7 of its norm for strengths up to one and any decay.  (Two
// parts of S against K: 2e-6 where little is forgotten; of F and the terms: 3e-6; of T, with keys
// alike and strengths near two: 1e-4 after 150 tokens.)  Strength two without decay forgets nothing
// ever: 8e-6 after 4096 tokens, where fp32 token by token is off by 1.4e-6, since the tensor cores
// cut sums off rather than rounding them (two parts of S against K: 3e-5).
// Two parts (2^-17) where a value only leads to bf16 results: S against Q, P and b E in the readout.
// Outputs then differ from those of fp32 sums by 1.3e-4 of their norm, single steps of bf16 where
// a value lies at the edge of a rounding; their error against 64 bits is that of the rounding either
// way, 1.7e-3.  Three parts there take B8 T4096 H32 a tenth longer.
// B8 T4096 H32 takes 353 us so, with two parts against K 322, with two throughout 287.
//
// mma.sync: the chain's products are 16 x 16 x 64 and smaller and each needs the one before it, 21
// cycles from registers to registers, one every 8 a scheduler.  tcgen05 would take the 64-token form:
// three groups of products a block (K S, T F, K^T E), each a round through shared memory, a barrier, a
// commit and TMEM loads, about 1000 cycles in the backward's second launch, against 5500 for the
// four sub-chunks of a block here; that form has not been built.  What bounds a chain here is its
// schedulers: an mma.sync keeps the FP32 pipe's dispatch for about 6 of its 8
// cycles, so the 82 of a sub-chunk and the 400 instructions beside them hardly overlap (1370 cycles
// a sub-chunk where the tensor pipe needs 660; a second CTA on the SM adds a twentieth).
#pragma once

#include "gated_delta.h"
#include "gated_delta_math.cuh"
#include "warp_mma.cuh"

namespace goldwkv {
namespace gdr {

using namespace wm;

constexpr int kSub = 16;                    // tokens of a sub-chunk
constexpr int kSubs = C / kSub;
constexpr int kChainWarps = 4;
constexpr int kPrepThreads = 128;
constexpr int kTcThreads = 256;             // chain warps, then as many of preparation
constexpr uint32_t kTileBytes = C * C * 2;  // 64 rows of 128 bytes
constexpr int kTile16 = kSub * 32;          // a 16 x 16 bf16 tile
// Its row of 32 bytes, two 16-byte chunks that trade places every four rows: eight rows then lie
// in different banks.
__device__ __forceinline__ uint32_t off16(int row, int chunk) {
    return (uint32_t)(row * 32 + ((chunk ^ ((row >> 2) & 1)) << 4));
}

// What the preparation hands to the chain for one block.
struct Prep {
    uint8_t t[3][kSubs][kTile16];    // T in three parts, [t][s]
    uint8_t p[3][kSubs][kTile16];    // P in two, or three
    float g[C];                      // e^L inside the sub-chunk
    float to_end[C];
    float beta[C];
    float g_end[kSubs];
};

// ldmatrix address of a 16 x 16 tile: both n halves of a B operand from [n][k] rows ...
__device__ __forceinline__ uint32_t addr16_b(uint32_t tile, int lane) {
    return tile + off16(((lane >> 4) << 3) + (lane & 7), (lane >> 3) & 1);
}
// ... and from [k][n] rows (.trans)
__device__ __forceinline__ uint32_t addr16_bt(uint32_t tile, int lane) { return tile + off16(lane & 15, lane >> 4); }

// Rows t0 .. t0 + 63 of a token tensor (row stride `step` values) into a tile by `threads`
// threads; rows at T or beyond as zeros.
template <int kThreads>
__device__ __forceinline__ void copy_block(uint32_t tile, const __nv_bfloat16* base, size_t step, int t0,
                                           int T, int tid) {
#pragma unroll
    for (int i = 0; i < C * 8 / kThreads; ++i) {
        const int row = (tid >> 3) + i * (kThreads / 8), chunk = tid & 7;
        const bool in = t0 + row < T;
        cp_async16(tile + sw_off(row, chunk), base + (in ? (size_t)(t0 + row) * step : 0) + chunk * 8, in);
    }
}

// Decay rate and write strength of a lane's token (lanes 16-31 as lanes 0-15); tokens at T or
// beyond neither decay nor write.
struct Gate {
    __nv_bfloat16 omega, beta;   // as stored: converted at their use, a block later
    bool in;
};
__device__ __forceinline__ Gate load_gate(const __nv_bfloat16* omega, const __nv_bfloat16* beta, int stride, int t, int T) {
    Gate g;
    g.in = t < T;
    g.omega = g.in ? omega[(size_t)t * stride] : __nv_bfloat16(0.f);
    g.beta = g.in ? beta[(size_t)t * stride] : __nv_bfloat16(0.f);
    return g;
}

// One warp prepares sub-chunk j of a block, P in kP parts (0: none).  at: 16 x 20 floats of the
// warp's own.
template <int kP>
__device__ __forceinline__ void prepare_sub(Prep& out, float* at, uint32_t kt, uint32_t qt, int j, Gate gate,
                                            float scale, int lane) {
    const int r = lane >> 2, c = 2 * (lane & 3);
    const uint32_t ka = addr_a(kt, kSub * j, 0, lane), kb = addr_b(kt, kSub * j, 0, lane), qa = ka + (qt - kt);
    // running sums of log2 w in 64 bits, kept as two floats: a difference then carries its own
    // rounding only, not that of a sum that one strong decay has made large
    const float beta = to_f32(gate.beta);
    double l = gate.in ? -1.4426950408889634 * (double)decay_rate(to_f32(gate.omega)) : 0.0;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, l, o, 16);
        if ((lane & 15) >= o) l += x;
    }
    const double total = __shfl_sync(0xffffffffu, l, 15, 16);
    const float hi = (float)l, lo = (float)(l - (double)hi);
    if (lane < 16) {
        out.g[kSub * j + lane] = exp2f(hi);
        out.to_end[kSub * j + lane] = exp2f((float)(total - l));
        out.beta[kSub * j + lane] = beta;
        if (lane == 15) out.g_end[j] = exp2f(hi);
    }
    float kk[2][4], qk[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        clear(kk[n]);
        clear(qk[n]);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        uint32_t a[4], b[4];
        ldsm4(b, step(kb, s));
        ldsm4(a, step(ka, s));
        mma(kk[0], a, b[0], b[1]);
        mma(kk[1], a, b[2], b[3]);
        if (kP) {
            ldsm4(a, step(qa, s));
            mma(qk[0], a, b[0], b[1]);
            mma(qk[1], a, b[2], b[3]);
        }
    }
    const float h0 = __shfl_sync(0xffffffffu, hi, r), l0 = __shfl_sync(0xffffffffu, lo, r);
    const float h1 = __shfl_sync(0xffffffffu, hi, r + 8), l1 = __shfl_sync(0xffffffffu, lo, r + 8);
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int u = 8 * n + c + e;
            const float hu = __shfl_sync(0xffffffffu, hi, u), lu = __shfl_sync(0xffffffffu, lo, u);
            const float bu = __shfl_sync(0xffffffffu, beta, u);
            // above the diagonal the difference is positive and may overflow: not taken there
            const float d0 = r >= u ? tiles::fast_exp2((h0 - hu) + (l0 - lu)) : 0.f;
            const float d1 = r + 8 >= u ? tiles::fast_exp2((h1 - hu) + (l1 - lu)) : 0.f;
            at[u * 20 + r] = r > u ? kk[n][e] * d0 * bu : 0.f;        // (M b)^T
            at[u * 20 + r + 8] = r + 8 > u ? kk[n][2 + e] * d1 * bu : 0.f;
            if (kP) {
                qk[n][e] = r >= u ? scale * qk[n][e] * d0 : 0.f;
                qk[n][2 + e] = r + 8 >= u ? scale * qk[n][2 + e] * d1 : 0.f;
            }
        }
    __syncwarp();
    // (I + M b)^-1 by substitution, a lane a column.  Not a power series: every entry of the
    // inverse stays bounded where keys are alike, while the powers of M b grow and cancel.
    float x[kSub];
#pragma unroll
    for (int i = 0; i < kSub; ++i) x[i] = i == (lane & 15) ? 1.f : 0.f;
#pragma unroll
    for (int s = 0; s < kSub - 1; ++s)
#pragma unroll
        for (int i = (s + 1) & ~3; i < kSub; i += 4) {
            const float4 m = *reinterpret_cast<const float4*>(at + s * 20 + i);   // zero up to i == s
            x[i] = fmaf(-m.x, x[s], x[i]);
            x[i + 1] = fmaf(-m.y, x[s], x[i + 1]);
            x[i + 2] = fmaf(-m.z, x[s], x[i + 2]);
            x[i + 3] = fmaf(-m.w, x[s], x[i + 3]);
        }
    // lanes 0-15 store the first part of their column and the third, lanes 16-31 the second
    uint8_t* dst = out.t[lane >> 4][j];
    const int ch = (lane >> 3) & 1, by = 2 * (lane & 7);
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
        const __nv_bfloat16 h = __float2bfloat16_rn(x[i]);
        const float rest = x[i] - __bfloat162float(h);
        const __nv_bfloat16 m = __float2bfloat16_rn(rest);
        *reinterpret_cast<__nv_bfloat16*>(dst + off16(i, ch) + by) = lane < 16 ? h : m;
        if (lane < 16)
            *reinterpret_cast<__nv_bfloat16*>(out.t[2][j] + off16(i, ch) + by) =
                __float2bfloat16_rn(rest - __bfloat162float(m));
    }
    if (kP) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t a, b, e = 0;
                const float2 x = make_float2(qk[n][2 * h], qk[n][2 * h + 1]);
                if (kP == 3) split3(x, a, b, e);
                else split2(x, a, b);
                const uint32_t o = off16(r + 8 * h, n) + 2 * c;
                *reinterpret_cast<uint32_t*>(out.p[0][j] + o) = a;
                *reinterpret_cast<uint32_t*>(out.p[1][j] + o) = b;
                if (kP == 3) *reinterpret_cast<uint32_t*>(out.p[2][j] + o) = e;
            }
    }
    __syncwarp();
}

// E^T = F^T T^T (kTrans: F^T T) for a chain warp: F^T as accumulators, taken in three parts (kExact)
// or two; `t` the sub-chunk's tile of T's first part.  The smallest terms first, in two chains of
// sums.
template <bool kExact, bool kTrans = false>
__device__ __forceinline__ void times_t(float (&e)[2][4], const float (&x)[2][4], uint32_t t, int lane) {
    uint32_t b0[4], b1[4], b2[4], a0[4], a1[4], a2[4];
    const uint32_t at = kTrans ? addr16_bt(t, lane) : addr16_b(t, lane);
    if (kTrans) {
        ldsm4t(b0, at);
        ldsm4t(b1, at + kSubs * kTile16);
        ldsm4t(b2, at + 2 * kSubs * kTile16);
    } else {
        ldsm4(b0, at);
        ldsm4(b1, at + kSubs * kTile16);
        ldsm4(b2, at + 2 * kSubs * kTile16);
    }
    float f[2][4];
    if (kExact) split_a3(a0, a1, a2, x[0], x[1]);
    else split_a(a0, a1, x[0], x[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        mma0(e[i], a0, b2[2 * i], b2[2 * i + 1]);
        if (kExact) mma0(f[i], a2, b0[2 * i], b0[2 * i + 1]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        mma(e[i], a1, b1[2 * i], b1[2 * i + 1]);
        if (kExact) mma(f[i], a1, b0[2 * i], b0[2 * i + 1]);
        else mma0(f[i], a1, b0[2 * i], b0[2 * i + 1]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        mma(e[i], a0, b1[2 * i], b1[2 * i + 1]);
        mma(f[i], a0, b0[2 * i], b0[2 * i + 1]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) e[i][k] += f[i][k];
}

// A state-shaped matrix [key][value] fp32 (null: zeros) to and from a chain warp's accumulators:
// S[i]: value columns 16 cw + r, + 8; keys 8 i + c, c + 1.
__device__ __forceinline__ void load_state(float (&S)[8][4], const float* src, int cw, int lane) {
    const int r = lane >> 2, c = 2 * (lane & 3);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            S[i][e] = src ? src[(8 * i + c + (e & 1)) * C + 16 * cw + r + 8 * (e >> 1)] : 0.f;
}
__device__ __forceinline__ void unit_state(float (&S)[8][4], int cw, int lane) {
    const int r = lane >> 2, c = 2 * (lane & 3);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[i][e] = 8 * i + c + (e & 1) == 16 * cw + r + 8 * (e >> 1) ? 1.f : 0.f;
}
__device__ __forceinline__ void store_state(float* dst, const float (&S)[8][4], int cw, int lane) {
    const int r = lane >> 2, c = 2 * (lane & 3);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[(8 * i + c + (e & 1)) * C + 16 * cw + r + 8 * (e >> 1)] = S[i][e];
}

// The same, [value][key].
__device__ __forceinline__ void store_state_t(float* dst, const float (&S)[8][4], int cw, int lane) {
    const int r = lane >> 2, c = 2 * (lane & 3);
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float2*>(dst + (16 * cw + r + 8 * h) * C + 8 * i + c) = make_float2(S[i][2 * h], S[i][2 * h + 1]);
}

// S^T = factor S^T + X^T K (+ Z^T Q with kTwo): X^T, Z^T as accumulators, taken in three parts
// (kExact) or two; kt, qt: addr_bt of K's and Q's 16 rows at chunk 0.  The products are summed on
// their own and added to S by FMAs, which round to nearest: an mma.sync cuts its sum off, so that
// S as its accumulator lost a little of its size in every one of three.
template <bool kExact, bool kTwo = false>
__device__ __forceinline__ void update_state(float (&S)[8][4], float factor, const float (&x)[2][4], uint32_t kt,
                                             const float (*z)[4] = nullptr, uint32_t qt = 0) {
    uint32_t a[3][4], c[3][4];
    if (kExact) split_a3(a[0], a[1], a[2], x[0], x[1]);
    else split_a(a[0], a[1], x[0], x[1]);
    if (kTwo) {
        if (kExact) split_a3(c[0], c[1], c[2], z[0], z[1]);
        else split_a(c[0], c[1], z[0], z[1]);
    }
    constexpr int kLast = kExact ? 2 : 1;   // the smallest terms first
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t kb[4], qb[4];
        ldsm4t(kb, step(kt, i));
        if (kTwo) ldsm4t(qb, step(qt, i));
        float d[2][4];
#pragma unroll
        for (int n = kLast; n >= 0; --n) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (n == kLast) mma0(d[u], a[n], kb[2 * u], kb[2 * u + 1]);
                else mma(d[u], a[n], kb[2 * u], kb[2 * u + 1]);
            }
            if (kTwo)
#pragma unroll
                for (int u = 0; u < 2; ++u) mma(d[u], c[n], qb[2 * u], qb[2 * u + 1]);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[2 * i + u][e] = fmaf(S[2 * i + u][e], factor, d[u][e]);
    }
}

// A chain warp's 16 tokens x 16 value columns, as transposed accumulators, rounded to bf16 and
// put to out (token 0, first column of the warp; row stride `step`), tokens at `count` or beyond
// not written.  tile: kTile16 bytes of the warp's own, through which they are turned.
__device__ __forceinline__ void store_tokens(__nv_bfloat16* out, size_t step, int count, const float (&y)[2][4],
                                             uint8_t* tile, int lane) {
    __syncwarp();
    stsm4t(ptx::smem_addr(tile) + off16(((lane >> 4) << 3) + (lane & 7), (lane >> 3) & 1),
           pack2(y[0][0], y[0][1]), pack2(y[0][2], y[0][3]), pack2(y[1][0], y[1][1]), pack2(y[1][2], y[1][3]));
    __syncwarp();
    const int t = lane >> 1;
    if (t < count)
        *reinterpret_cast<uint4*>(out + (size_t)t * step + 8 * (lane & 1)) =
            *reinterpret_cast<const uint4*>(tile + off16(t, lane & 1));
}

}  // namespace gdr
}  // namespace goldwkv
