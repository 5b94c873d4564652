// The gated delta rule token by token: the fp32 prefill and the decode step (sm_100a).
//
// Per (b, h), state S (64 key rows x 64 value columns, fp32), w = exp(-exp(omega)):
//     e_t = v_t - w_t S_{t-1}^T k_t,   S_t = w_t S_{t-1} + b_t k_t e_t^T,   y_t = scale S_t^T q_t.
// Both kernels read the state once per token: with a = S_{t-1}^T k_t and c = S_{t-1}^T q_t taken
// together, e_t = v_t - w_t a and y_t = scale (w_t c + b_t (k_t . q_t) e_t), so the readout
// waits for no second pass over the updated state.
#include "common.cuh"
#include "gated_delta.h"
#include "gated_delta_math.cuh"

namespace goldwkv {

namespace {

using gdr::load4;

constexpr int D = kHeadSize;

__device__ __forceinline__ float dot4(float4 a, float4 b, float c) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}

// ------------------------------------------------------------------ prefill
// Value columns are independent.  Four adjacent lanes share kJ columns, 16 state rows each in
// registers; two xor-shuffles finish the sums over rows.  A CTA of 128 threads owns 32 kJ columns
// of a head: 32, grid B*H x 2, when there are few heads, where the chain from one token to the next
// bounds the call (the sums, e and one FMA per state entry, 300 cycles with a warp a scheduler);
// 64, grid B*H, from one CTA an SM on, where reading q and k from shared memory bounds it and two
// columns a thread read them once (B8 T1024 H32: 332 us against 409; B4 T2048 H16 433 against 326).  Tokens come through shared
// memory in tiles of 16, the next tile's loads issued before the present one is walked.
constexpr int kTile = 16;
constexpr int kThreads = 128;
constexpr int kRow = D + 4;   // padded token row: the k . q sums read a column of rows

template <int kJ>
struct Stage {
    float q[kTile][kRow];
    float k[kTile][kRow];
    float v[kTile][32 * kJ];
    float w[kTile], b[kTile], kq[kTile];
};

template <int kJ>
__global__ void __launch_bounds__(kThreads)
gated_delta_recurrent_kernel(const float* __restrict__ q, const float* __restrict__ k,
                             const float* __restrict__ v, const float* __restrict__ omega,
                             const float* __restrict__ beta, float scale, const float* s_in,
                             float* s_out, float* __restrict__ y, int T, int H, int HK) {
    __shared__ __align__(16) Stage<kJ> stage[2];
    const int bh = blockIdx.x, b = bh / H, h = bh - b * H, hk = h / (H / HK);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int part = lane & 3;                    // rows 4 (4 m + part) + {0..3}, m = 0..3
    const int jl = kJ * (warp * 8 + (lane >> 2)); // first column within the CTA
    const int j0 = blockIdx.y * 32 * kJ;

    const float* qp = q + ((size_t)b * T * HK + hk) * D;     // token t: + t * HK * D
    const float* kp = k + ((size_t)b * T * HK + hk) * D;
    const float* vp = v + ((size_t)b * T * H + h) * D + j0;  // token t: + t * H * D
    const float* op = omega + (size_t)b * T * H + h;
    const float* bp = beta + (size_t)b * T * H + h;
    float* yp = y + ((size_t)b * T * H + h) * D + j0 + jl;
    const size_t kstep = (size_t)HK * D, vstep = (size_t)H * D;

    float S[kJ][16];
    const float* s0 = s_in ? s_in + (size_t)bh * D * D + j0 + jl : nullptr;
#pragma unroll
    for (int m = 0; m < 16; ++m)
#pragma unroll
        for (int j = 0; j < kJ; ++j)
            S[j][m] = s0 ? s0[(size_t)(16 * (m >> 2) + 4 * part + (m & 3)) * D + j] : 0.f;

    // a thread stages 4 channels of tokens tid/16 and tid/16 + 8 of q and k, 4 kJ of token tid/8 of v
    const int tq = tid >> 4, cq = 4 * (tid & 15), tv = tid >> 3, cv = 4 * (tid & 7);
    float4 rq[2], rk[2], rv[kJ];
    float rw = 0.f, rb = 0.f;
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = t0 + tq + 8 * i;
            rq[i] = t < T ? load4(qp + t * kstep + cq) : zero;
            rk[i] = t < T ? load4(kp + t * kstep + cq) : zero;
        }
#pragma unroll
        for (int j = 0; j < kJ; ++j) rv[j] = t0 + tv < T ? load4(vp + (t0 + tv) * vstep + cv + 32 * j) : zero;
        if (tid < kTile && t0 + tid < T) {
            rw = op[(size_t)(t0 + tid) * H];
            rb = bp[(size_t)(t0 + tid) * H];
        }
    };
    fetch(0);
    const int tiles = (T + kTile - 1) / kTile;
    for (int n = 0; n < tiles; ++n) {
        Stage<kJ>& s = stage[n & 1];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            *reinterpret_cast<float4*>(&s.q[tq + 8 * i][cq]) = rq[i];
            *reinterpret_cast<float4*>(&s.k[tq + 8 * i][cq]) = rk[i];
            // k . q of the token, over the 16 lanes that hold it
            float d = dot4(rq[i], rk[i], 0.f);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
            if ((lane & 15) == 0) s.kq[tq + 8 * i] = d;
        }
#pragma unroll
        for (int j = 0; j < kJ; ++j) *reinterpret_cast<float4*>(&s.v[tv][cv + 32 * j]) = rv[j];
        if (tid < kTile) {
            s.w[tid] = gdr::decay(rw);
            s.b[tid] = rb;
        }
        __syncthreads();   // the buffer's last readers passed the barrier of tile n - 1
        if (n + 1 < tiles) fetch((n + 1) * kTile);
        const int cnt = min(kTile, T - n * kTile);
        for (int t = 0; t < cnt; ++t) {
            float4 kk[4];
            float a[kJ][4], c[kJ][4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                kk[m] = *reinterpret_cast<const float4*>(&s.k[t][16 * m + 4 * part]);
                const float4 qq = *reinterpret_cast<const float4*>(&s.q[t][16 * m + 4 * part]);
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    const float4 x = make_float4(S[j][4 * m], S[j][4 * m + 1], S[j][4 * m + 2], S[j][4 * m + 3]);
                    a[j][m] = dot4(kk[m], x, 0.f);
                    c[j][m] = dot4(qq, x, 0.f);
                }
            }
            const float w = s.w[t];
            float be[kJ], out[kJ];
#pragma unroll
            for (int j = 0; j < kJ; ++j) {
                float as = (a[j][0] + a[j][1]) + (a[j][2] + a[j][3]), cs = (c[j][0] + c[j][1]) + (c[j][2] + c[j][3]);
                as += __shfl_xor_sync(0xffffffffu, as, 1);
                cs += __shfl_xor_sync(0xffffffffu, cs, 1);
                as += __shfl_xor_sync(0xffffffffu, as, 2);
                cs += __shfl_xor_sync(0xffffffffu, cs, 2);
                be[j] = s.b[t] * fmaf(-w, as, s.v[t][jl + j]);
                out[j] = scale * fmaf(s.kq[t], be[j], w * cs);
            }
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int j = 0; j < kJ; ++j) {
                    S[j][4 * m] = fmaf(kk[m].x, be[j], w * S[j][4 * m]);
                    S[j][4 * m + 1] = fmaf(kk[m].y, be[j], w * S[j][4 * m + 1]);
                    S[j][4 * m + 2] = fmaf(kk[m].z, be[j], w * S[j][4 * m + 2]);
                    S[j][4 * m + 3] = fmaf(kk[m].w, be[j], w * S[j][4 * m + 3]);
                }
            if (part == 0)
#pragma unroll
                for (int j = 0; j < kJ; ++j) yp[(size_t)(n * kTile + t) * vstep + j] = out[j];
        }
    }
    if (s_out) {
        float* so = s_out + (size_t)bh * D * D + j0 + jl;
#pragma unroll
        for (int m = 0; m < 16; ++m)
#pragma unroll
            for (int j = 0; j < kJ; ++j) so[(size_t)(16 * (m >> 2) + 4 * part + (m & 3)) * D + j] = S[j][m];
    }
}

// ------------------------------------------------------------------ decode
// A pure stream over the 16 KB state of each head, as wkv6_decode_kernel: 256 threads a head,
// four 16-byte loads of the state each, all in flight before the small operands are staged.
// The one difference is that e needs the column sums before the state can be written: one
// barrier between the loads and the stores, hidden by the other CTAs of the SM.
constexpr int kDecThreads = 256;

template <typename IO>
__global__ void __launch_bounds__(kDecThreads)
gated_delta_decode_kernel(const IO* __restrict__ q, const IO* __restrict__ k,
                          const IO* __restrict__ v, const IO* __restrict__ omega,
                          const IO* __restrict__ beta, float scale, float* __restrict__ state,
                          IO* __restrict__ y, int H, int HK) {
    __shared__ float sq[D], sk[D];
    __shared__ __align__(16) float sv[D];
    __shared__ float4 reda[kDecThreads / 32][D / 4], redc[kDecThreads / 32][D / 4];
    __shared__ float skq[2];
    const int bh = blockIdx.x, b = bh / H, h = bh - b * H;
    const size_t kh = ((size_t)b * HK + h / (H / HK)) * D;
    const int tid = threadIdx.x;
    const int c = tid & 15;            // columns 4c .. 4c + 3
    const int r0 = tid >> 4;           // rows r0 + 16 m
    float4* S = reinterpret_cast<float4*>(state + (size_t)bh * D * D);

    float4 s[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) s[m] = __ldcs(&S[(r0 + 16 * m) * (D / 4) + c]);
    const float w = gdr::decay(to_f32(omega[bh])), bt = to_f32(beta[bh]);
    if (tid < D) {
        const float qv = to_f32(q[kh + tid]), kv = to_f32(k[kh + tid]);
        sq[tid] = qv;
        sk[tid] = kv;
        sv[tid] = to_f32(v[(size_t)bh * D + tid]);
        const float p = warp_sum(qv * kv);
        if ((tid & 31) == 0) skq[tid >> 5] = p;
    }
    __syncthreads();

    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), cq = a;
    float ki[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const float qi = sq[r0 + 16 * m];
        ki[m] = sk[r0 + 16 * m];
        a.x = fmaf(ki[m], s[m].x, a.x);
        a.y = fmaf(ki[m], s[m].y, a.y);
        a.z = fmaf(ki[m], s[m].z, a.z);
        a.w = fmaf(ki[m], s[m].w, a.w);
        cq.x = fmaf(qi, s[m].x, cq.x);
        cq.y = fmaf(qi, s[m].y, cq.y);
        cq.z = fmaf(qi, s[m].z, cq.z);
        cq.w = fmaf(qi, s[m].w, cq.w);
    }
    a.x += __shfl_xor_sync(0xffffffffu, a.x, 16);
    a.y += __shfl_xor_sync(0xffffffffu, a.y, 16);
    a.z += __shfl_xor_sync(0xffffffffu, a.z, 16);
    a.w += __shfl_xor_sync(0xffffffffu, a.w, 16);
    cq.x += __shfl_xor_sync(0xffffffffu, cq.x, 16);
    cq.y += __shfl_xor_sync(0xffffffffu, cq.y, 16);
    cq.z += __shfl_xor_sync(0xffffffffu, cq.z, 16);
    cq.w += __shfl_xor_sync(0xffffffffu, cq.w, 16);
    if ((tid & 31) < 16) {
        reda[tid >> 5][c] = a;
        redc[tid >> 5][c] = cq;
    }
    __syncthreads();
    a = reda[0][c];
#pragma unroll
    for (int i = 1; i < kDecThreads / 32; ++i) {
        const float4 x = reda[i][c];
        a.x += x.x;
        a.y += x.y;
        a.z += x.z;
        a.w += x.w;
    }
    const float4 vj = reinterpret_cast<const float4*>(sv)[c];
    const float4 be = make_float4(bt * fmaf(-w, a.x, vj.x), bt * fmaf(-w, a.y, vj.y),
                                  bt * fmaf(-w, a.z, vj.z), bt * fmaf(-w, a.w, vj.w));
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        float4 x = s[m];
        x.x = fmaf(ki[m], be.x, w * x.x);
        x.y = fmaf(ki[m], be.y, w * x.y);
        x.z = fmaf(ki[m], be.z, w * x.z);
        x.w = fmaf(ki[m], be.w, w * x.w);
        __stcs(&S[(r0 + 16 * m) * (D / 4) + c], x);
    }
    if (tid < D / 4) {   // c == tid
        cq = redc[0][c];
#pragma unroll
        for (int i = 1; i < kDecThreads / 32; ++i) {
            const float4 x = redc[i][c];
            cq.x += x.x;
            cq.y += x.y;
            cq.z += x.z;
            cq.w += x.w;
        }
        const float kq = skq[0] + skq[1];
        IO* yp = y + (size_t)bh * D + 4 * c;
        yp[0] = from_f32<IO>(scale * fmaf(kq, be.x, w * cq.x));
        yp[1] = from_f32<IO>(scale * fmaf(kq, be.y, w * cq.y));
        yp[2] = from_f32<IO>(scale * fmaf(kq, be.z, w * cq.z));
        yp[3] = from_f32<IO>(scale * fmaf(kq, be.w, w * cq.w));
    }
}

template <typename IO>
cudaError_t decode_io(const GdrIn& in, float* state, void* y, cudaStream_t st) {
    gated_delta_decode_kernel<IO><<<(unsigned)(in.B * in.H), kDecThreads, 0, st>>>(
        (const IO*)in.q, (const IO*)in.k, (const IO*)in.v, (const IO*)in.omega, (const IO*)in.beta,
        in.scale, state, (IO*)y, in.H, in.HK);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_recurrent(const GdrIn& in, const float* s_in, float* s_out, void* y, cudaStream_t st) {
    const unsigned heads = (unsigned)(in.B * in.H);
    auto run = [&](auto kernel, unsigned parts) {
        kernel<<<dim3(heads, parts), kThreads, 0, st>>>(
            (const float*)in.q, (const float*)in.k, (const float*)in.v, (const float*)in.omega,
            (const float*)in.beta, in.scale, s_in, s_out, (float*)y, in.T, in.H, in.HK);
    };
    if (heads >= 148) run(gated_delta_recurrent_kernel<2>, 1);   // a CTA an SM
    else run(gated_delta_recurrent_kernel<1>, 2);
    return cudaGetLastError();
}

cudaError_t launch_gdr_decode(const GdrIn& in, float* state, void* y, bool bf16, cudaStream_t st) {
    return bf16 ? decode_io<__nv_bfloat16>(in, state, y, st) : decode_io<float>(in, state, y, st);
}

}  // namespace goldwkv
