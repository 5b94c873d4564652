// Device helpers shared by the gated delta rule's kernels: vector loads and stores of four
// values, and a chunk's decays.
#pragma once

#include "common.cuh"

namespace goldwkv {
namespace gdr {

constexpr int C = 64;   // tokens a chunk, and the head size

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                       __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    uint2 w;
    w.x = *reinterpret_cast<const uint32_t*>(&a);
    w.y = *reinterpret_cast<const uint32_t*>(&b);
    *reinterpret_cast<uint2*>(p) = w;
}

// exp(omega), at most 1e4: w = exp(-1e4) is 0 in fp32 as any smaller one is, and a finite rate
// keeps the sums below and rate * w free of inf - inf and inf * 0.  A NaN stays one.
__device__ __forceinline__ float decay_rate(float omega) {
    const float r = expf(omega);
    return r > 1e4f ? 1e4f : r;
}

// w = exp(-exp(omega)) of one token.  Near 1, where a state is multiplied by many of them, expf's
// error of a unit or two does not average out (2e-6 of a state that remembers 90 tokens).  There the
// Taylor series about 0, whose next term is below 4e-10, rounded once as it is taken from 1.
__device__ __forceinline__ float decay(float omega) {
    const float r = expf(omega);
    float p = fmaf(r, 1.f / 5040.f, -1.f / 720.f);
    p = fmaf(r, p, 1.f / 120.f);
    p = fmaf(r, p, -1.f / 24.f);
    p = fmaf(r, p, 1.f / 6.f);
    p = fmaf(r, p, -0.5f);
    p = fmaf(r, p, 1.f);
    const float far = expf(-r);
    return r < 0.25f ? fmaf(-r, p, 1.f) : far;
}

// The decays of one chunk.  The sums of log2 w are taken in 64 bits and kept as two floats:
// a difference of two of them then carries its own rounding only, not that of a running sum
// that one strong decay has made large.
struct Gates {
    float hi[C], lo[C];        // sum of log2 w up to and with t
    float g[C];                // 2^that
    float to_end[C];           // 2^(sum over the tokens after t)
    float beta[C], rate[C];
    __device__ __forceinline__ float between(int t, int s) const {   // s <= t
        float y;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((hi[t] - hi[s]) + (lo[t] - lo[s])));
        return y;
    }
};

// Tokens at T or beyond neither decay nor write (log w = 0, beta = 0).  One warp does it (the first,
// or that whose threads pass 0 .. 31 as tid), two tokens a lane: the loads (fetch) ahead of the
// rest; the caller's barrier publishes it.
template <typename IO>
struct RawGates {
    IO omega[2], beta[2];
};
template <typename IO>
__device__ __forceinline__ RawGates<IO> fetch_gates(const IO* omega, const IO* beta, size_t base, int stride,
                                                    int t0, int T, int tid = threadIdx.x) {
    RawGates<IO> r{};
    if (tid < 32)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * tid + i;
            if (t0 + t < T) {
                r.omega[i] = omega[base + (size_t)(t0 + t) * stride];
                r.beta[i] = beta[base + (size_t)(t0 + t) * stride];
            }
        }
    return r;
}
template <typename IO>
__device__ __forceinline__ void put_gates(Gates& s, const RawGates<IO>& raw, int t0, int T, int tid = threadIdx.x) {
    if (tid >= 32) return;
    const int lane = tid;
    double l[2], run = 0.0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        const bool in = t0 + t < T;
        const float r = in ? decay_rate(to_f32(raw.omega[i])) : 0.f;
        s.rate[t] = r;
        s.beta[t] = in ? to_f32(raw.beta[i]) : 0.f;
        run += -1.4426950408889634 * (double)r;
        l[i] = run;
    }
    double before = run;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += x;
    }
    const double total = __shfl_sync(0xffffffffu, before, 31);
    before -= run;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = 2 * lane + i;
        const double x = before + l[i];
        const float hi = (float)x;
        s.hi[t] = hi;
        s.lo[t] = (float)(x - (double)hi);
        s.g[t] = exp2f((float)x);
        s.to_end[t] = exp2f((float)(total - x));
    }
}
template <typename IO>
__device__ __forceinline__ void load_gates(Gates& s, const IO* omega, const IO* beta, size_t base,
                                           int stride, int t0, int T) {
    put_gates(s, fetch_gates(omega, beta, base, stride, t0, T), t0, T);
}

}  // namespace gdr
}  // namespace goldwkv
