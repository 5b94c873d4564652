// Chunked prefill of the gated delta rule, bf16 inputs, on tensor cores (sm_100a).  The algebra
// and the division of labour are in gated_delta_tiles.cuh.
#include "common.cuh"
#include "gated_delta.h"
#include "gated_delta_tiles.cuh"

namespace goldwkv {

namespace {

using namespace gdr;
using bf16 = __nv_bfloat16;

constexpr int kStages = 3;   // a block in the chain, one in preparation, one on its way

struct Smem {
    uint8_t k[kStages][kTileBytes];
    uint8_t v[kStages][kTileBytes];
    uint8_t q[kStages][kTileBytes];
    Prep prep[2];
    float at[kSubs][kSub * 20];
    uint8_t y[kSubs][kTile16];
};

struct Args {
    GdrIn in;
    const float* s_in;
    float* s_out;
    bf16* y;
};

__global__ void __launch_bounds__(kTcThreads, 2)
gated_delta_chunked_kernel(const __grid_constant__ Args p) {
    extern __shared__ __align__(16) uint8_t raw[];
    Smem& s = tiles::smem_aligned<Smem>(raw);
    const int H = p.in.H, HK = p.in.HK, T = p.in.T, bh = blockIdx.x, b = bh / H, h = bh - b * H, hk = h / (H / HK);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int blocks = (T + C - 1) / C;
    const size_t ko = ((size_t)b * T * HK + hk) * C, vo = ((size_t)b * T * H + h) * C, go = (size_t)b * T * H + h;
    const bf16 *q = (const bf16*)p.in.q + ko, *k = (const bf16*)p.in.k + ko, *v = (const bf16*)p.in.v + vo;
    const uint32_t sk = ptx::smem_addr(s.k), sv = ptx::smem_addr(s.v), sq = ptx::smem_addr(s.q);
    const int r = lane >> 2, c = 2 * (lane & 3);

    if (warp >= kSubs) {   // ---- preparation
        const int j = warp - kSubs, pt = tid - 32 * kSubs;
        const bf16 *omega = (const bf16*)p.in.omega + go, *beta = (const bf16*)p.in.beta + go;
        auto copy = [&](int n) {
            const uint32_t o = (uint32_t)(n % kStages) * kTileBytes;
            copy_block<128>(sk + o, k, (size_t)HK * C, n * C, T, pt);
            copy_block<128>(sv + o, v, (size_t)H * C, n * C, T, pt);
            copy_block<128>(sq + o, q, (size_t)HK * C, n * C, T, pt);
            cp_async_commit();
        };
        copy(0);
        const int t = kSub * j + (lane & 15);
        Gate gate = load_gate(omega, beta, H, t, T);
        cp_async_wait<0>();
        __syncthreads();
        for (int n = -1; n < blocks; ++n) {
            if (n + 2 < blocks) copy(n + 2);
            if (n + 1 < blocks) {
                const Gate next = load_gate(omega, beta, H, (n + 2) * C + t, T);
                const uint32_t o = (uint32_t)((n + 1) % kStages) * kTileBytes;
                if ((n + 1) * C + kSub * j < T)
                    prepare_sub<true>(s.prep[(n + 1) & 1], s.at[j], sk + o, sq + o, j, gate, p.in.scale, lane);
                gate = next;
            }
            cp_async_wait<0>();
            __syncthreads();
        }
        return;
    }

    // ---- chain: value columns 16 warp .. 16 warp + 15
    float S[8][4];   // [key tile]: value columns r, r + 8; keys 8 tile + c, c + 1
    {
        const float* src = p.s_in ? p.s_in + (size_t)bh * C * C + 16 * warp + r : nullptr;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[i][e] = src ? src[(size_t)(8 * i + c + (e & 1)) * C + 8 * (e >> 1)] : 0.f;
    }
    const uint32_t sy = ptx::smem_addr(s.y[warp]);
    // where this lane puts 16 bytes of the block's outputs: token lane / 2, half lane % 2
    bf16* yp = p.y + vo + 16 * warp + 8 * (lane & 1);
    __syncthreads();
    __syncthreads();   // the preparation's first turn, n = -1
    for (int n = 0; n < blocks; ++n) {
        const uint32_t o = (uint32_t)(n % kStages) * kTileBytes, kt = sk + o, vt = sv + o, qt = sq + o;
        const Prep& pr = s.prep[n & 1];
        const uint32_t pt = ptx::smem_addr(pr.t);
        const uint32_t pp0 = ptx::smem_addr(pr.p[0]), pp1 = ptx::smem_addr(pr.p[1]);
        const int subs = min(kSubs, (T - n * C + kSub - 1) / kSub);
        for (int j = 0; j < subs; ++j) {
            float f[2][4], y[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                clear(f[i]);
                clear(y[i]);
            }
            // S^T K^T and S^T Q^T
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t hi[4], lo[4], kb[4], qb[4];
                ldsm4(kb, addr_b(kt, kSub * j, 2 * i, lane));
                ldsm4(qb, addr_b(qt, kSub * j, 2 * i, lane));
                split_a(hi, lo, S[2 * i], S[2 * i + 1]);
                mma(f[0], hi, kb[0], kb[1]);
                mma(f[1], hi, kb[2], kb[3]);
                mma(y[0], hi, qb[0], qb[1]);
                mma(y[1], hi, qb[2], qb[3]);
                mma(f[0], lo, kb[0], kb[1]);
                mma(f[1], lo, kb[2], kb[3]);
                mma(y[0], lo, qb[0], qb[1]);
                mma(y[1], lo, qb[2], qb[3]);
            }
            uint32_t hi[4], lo[4], b0[4], b1[4], vv[4];
            ldsm4t(vv, addr_ct(vt, kSub * j, 2 * warp, lane));
            float2 gt[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                gt[i] = *reinterpret_cast<const float2*>(&pr.g[kSub * j + 8 * i + c]);
                const float2 v0 = tiles::unpack2(vv[2 * i]), v1 = tiles::unpack2(vv[2 * i + 1]);
                f[i][0] = fmaf(-gt[i].x, f[i][0], v0.x);
                f[i][1] = fmaf(-gt[i].y, f[i][1], v0.y);
                f[i][2] = fmaf(-gt[i].x, f[i][2], v1.x);
                f[i][3] = fmaf(-gt[i].y, f[i][3], v1.y);
            }
            // E^T = F^T T^T
            split_a(hi, lo, f[0], f[1]);
            float e[2][4];
            times_t(e, hi, lo, pt + j * kTile16, lane);
            float ke[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 bt = *reinterpret_cast<const float2*>(&pr.beta[kSub * j + 8 * i + c]);
                const float2 te = *reinterpret_cast<const float2*>(&pr.to_end[kSub * j + 8 * i + c]);
                e[i][0] *= bt.x;
                e[i][1] *= bt.y;
                e[i][2] *= bt.x;
                e[i][3] *= bt.y;
                ke[i][0] = e[i][0] * te.x;
                ke[i][1] = e[i][1] * te.y;
                ke[i][2] = e[i][2] * te.x;
                ke[i][3] = e[i][3] * te.y;
            }
            // S+^T = g S^T + (b to_end E)^T K
            split_a(hi, lo, ke[0], ke[1]);
            const float ge = pr.g_end[j];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t kb[4];
                ldsm4t(kb, addr_bt(kt, kSub * j, 2 * i, lane));
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    S[2 * i][m] *= ge;
                    S[2 * i + 1][m] *= ge;
                }
                mma(S[2 * i], lo, kb[0], kb[1]);
                mma(S[2 * i + 1], lo, kb[2], kb[3]);
                mma(S[2 * i], hi, kb[0], kb[1]);
                mma(S[2 * i + 1], hi, kb[2], kb[3]);
            }
            // Y^T = scale g (S^T Q^T) + (b E)^T P^T
            split_a(hi, lo, e[0], e[1]);
            ldsm4(b0, addr16_b(pp0 + j * kTile16, lane));
            ldsm4(b1, addr16_b(pp1 + j * kTile16, lane));
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float gx = p.in.scale * gt[i].x, gy = p.in.scale * gt[i].y;
                y[i][0] *= gx;
                y[i][1] *= gy;
                y[i][2] *= gx;
                y[i][3] *= gy;
                mma(y[i], lo, b0[2 * i], b0[2 * i + 1]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) mma(y[i], hi, b1[2 * i], b1[2 * i + 1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) mma(y[i], hi, b0[2 * i], b0[2 * i + 1]);
            // turned to [token][value] through the warp's own 16 x 16 tile
            __syncwarp();
            stsm4t(sy + (uint32_t)((((lane >> 4) << 3) + (lane & 7)) * kRow16 + ((lane >> 3) & 1) * 16),
                   pack2(y[0][0], y[0][1]), pack2(y[0][2], y[0][3]), pack2(y[1][0], y[1][1]), pack2(y[1][2], y[1][3]));
            __syncwarp();
            const int t = n * C + kSub * j + (lane >> 1);
            if (t < T)
                *reinterpret_cast<uint4*>(yp + (size_t)t * H * C) =
                    *reinterpret_cast<const uint4*>(s.y[warp] + (lane >> 1) * kRow16 + (lane & 1) * 16);
        }
        __syncthreads();
    }
    if (p.s_out) {
        float* dst = p.s_out + (size_t)bh * C * C + 16 * warp + r;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[(size_t)(8 * i + c + (e & 1)) * C + 8 * (e >> 1)] = S[i][e];
    }
}

}  // namespace

cudaError_t launch_gdr_chunked(const GdrIn& in, const float* s_in, float* s_out, void* y, cudaStream_t st) {
    const size_t smem = sizeof(Smem) + 1024;
    cudaError_t e = cudaFuncSetAttribute(gated_delta_chunked_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    gated_delta_chunked_kernel<<<(unsigned)(in.B * in.H), kTcThreads, smem, st>>>(Args{in, s_in, s_out, (bf16*)y});
    return cudaGetLastError();
}

}  // namespace goldwkv
