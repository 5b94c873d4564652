// Chunked prefill of the gated delta rule, bf16 inputs, on tensor cores (sm_100a).  The algebra,
// the division of labour and what bounds it are in gated_delta_tiles.cuh.
//
// B8 T4096 H32: 353 us for 540 MB that it has to move (82 us at the memory's rate), token by token
// on CUDA cores 1771; B1 T65531 H64 over 16 key heads, in two segments: 2.69 ms.
#include "common.cuh"
#include "dependent_launch.cuh"
#include "gated_delta.h"
#include "gated_delta_tiles.cuh"

namespace goldwkv {

namespace {

using namespace gdr;
using bf16 = __nv_bfloat16;

constexpr int kStages = 3;   // a block in the chain, one in preparation, one on its way

// Segments of the sequence (gated_delta_segments.cu); count 1: none.
struct Segments {
    int count, blocks;
    float* a;            // [head][count - 1][64][64]: A^T (its first place: the given state, which the
                         // call's last CTA may already be writing over when the first reads it)
    float* s;            // the same: B, then the state entering segment i + 1
};

struct Smem {
    uint8_t k[kStages][kTileBytes];
    uint8_t v[kStages][kTileBytes];
    uint8_t q[kStages][kTileBytes];
    Prep prep[2];
    float at[kChainWarps][kSub * 20];
    uint8_t y[kChainWarps][kTile16];
};

struct Args {
    GdrIn in;
    const float* s_in;
    float* s_out;
    bf16* y;
    Segments seg;
};

// One CTA's blocks: those of segment `seg` of head bh.  kOut: with outputs; otherwise only the
// state is left, and `unit` leaves A^T instead of B.
template <bool kOut>
__device__ __forceinline__ void walk(const Args& p, int bh, int seg, bool unit, const float* s_in, float* s_out) {
    extern __shared__ __align__(16) uint8_t raw[];
    Smem& s = tiles::smem_aligned<Smem>(raw);
    const int H = p.in.H, HK = p.in.HK, b = bh / H, h = bh - b * H, hk = h / (H / HK);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int first = seg * p.seg.blocks * C, T = p.in.T - first;   // tokens from the segment's first on
    const int blocks = min(p.seg.blocks, (T + C - 1) / C);
    const size_t t0 = (size_t)b * p.in.T + first;
    const size_t ko = (t0 * HK + hk) * C, vo = (t0 * H + h) * C, go = t0 * H + h;
    const bf16 *q = (const bf16*)p.in.q + ko, *k = (const bf16*)p.in.k + ko, *v = (const bf16*)p.in.v + vo;
    const uint32_t sk = ptx::smem_addr(s.k), sv = ptx::smem_addr(s.v), sq = ptx::smem_addr(s.q);

    if (warp >= kChainWarps) {   // ---- preparation
        const int w = warp - kChainWarps, pt = tid - kPrepThreads;
        const bf16 *omega = (const bf16*)p.in.omega + go, *beta = (const bf16*)p.in.beta + go;
        auto copy = [&](int n) {
            const uint32_t o = (uint32_t)(n % kStages) * kTileBytes;
            copy_block<kPrepThreads>(sk + o, k, (size_t)HK * C, n * C, T, pt);
            copy_block<kPrepThreads>(sv + o, v, (size_t)H * C, n * C, unit ? 0 : T, pt);
            if (kOut) copy_block<kPrepThreads>(sq + o, q, (size_t)HK * C, n * C, T, pt);
            cp_async_commit();
        };
        copy(0);
        const int t = kSub * w + (lane & 15);
        Gate gate = load_gate(omega, beta, H, t, T);
        cp_async_wait<0>();
        __syncthreads();
        for (int n = -1; n < blocks; ++n) {
            if (n + 2 < blocks) copy(n + 2);
            if (n + 1 < blocks) {
                const uint32_t o = (uint32_t)((n + 1) % kStages) * kTileBytes;
                const Gate next = load_gate(omega, beta, H, (n + 2) * C + t, T);
                if ((n + 1) * C + kSub * w < T)
                    prepare_sub<kOut ? 2 : 0>(s.prep[(n + 1) & 1], s.at[w], sk + o, sq + o, w, gate, p.in.scale, lane);
                gate = next;
            }
            cp_async_wait<0>();
            __syncthreads();
        }
        return;
    }

    // ---- chain: value columns 16 warp .. 16 warp + 15
    const int c = 2 * (lane & 3);
    float S[8][4];
    if (unit) {
        unit_state(S, warp, lane);
    } else {
        load_state(S, s_in, warp, lane);
        if (!kOut && seg == 0 && s_in) store_state(p.seg.a + (size_t)bh * (p.seg.count - 1) * C * C, S, warp, lane);
    }
    bf16* yp = kOut ? p.y + vo + 16 * warp : nullptr;
    const uint32_t ab = addr_b(0, 0, 0, lane), abt = addr_bt(0, 0, 0, lane), act = addr_ct(0, 0, 2 * warp, lane);
    __syncthreads();
    __syncthreads();   // the preparation's first turn, n = -1
    for (int n = 0; n < blocks; ++n) {
        const uint32_t o = (uint32_t)(n % kStages) * kTileBytes;
        const Prep& pr = s.prep[n & 1];
        const uint32_t pt = ptx::smem_addr(pr.t), pp = ptx::smem_addr(pr.p);
        const int subs = min(kSubs, (T - n * C + kSub - 1) / kSub);
#pragma unroll 2
        for (int j = 0; j < subs; ++j) {
            const int row = kSub * j;
            const uint32_t kt = sk + o + row * 128;
            // S^T K^T, all three parts of S, and S^T Q^T; the smaller parts' terms in sums of their own
            float f[2][4], e[2][4], y[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t a0[4], a1[4], a2[4], kb[4], qb[4];
                ldsm4(kb, step(kt + ab, i));
                if (kOut) ldsm4(qb, step(kt + ab, i) + (sq - sk));
                split_a3(a0, a1, a2, S[2 * i], S[2 * i + 1]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (i == 0) {
                        mma0(e[u], a2, kb[2 * u], kb[2 * u + 1]);
                        mma0(f[u], a0, kb[2 * u], kb[2 * u + 1]);
                        if (kOut) mma0(y[u], a1, qb[2 * u], qb[2 * u + 1]);
                    } else {
                        mma(e[u], a2, kb[2 * u], kb[2 * u + 1]);
                        mma(f[u], a0, kb[2 * u], kb[2 * u + 1]);
                        if (kOut) mma(y[u], a1, qb[2 * u], qb[2 * u + 1]);
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    mma(e[u], a1, kb[2 * u], kb[2 * u + 1]);
                    if (kOut) mma(y[u], a0, qb[2 * u], qb[2 * u + 1]);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x) f[u][x] += e[u][x];
            // F^T = V^T - g S^T K^T
            float2 g[2];
            uint32_t vv[4];
            ldsm4t(vv, sv + o + row * 128 + act);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                g[u] = *reinterpret_cast<const float2*>(&pr.g[row + 8 * u + c]);
                value_minus(f[u], g[u], vv[2 * u], vv[2 * u + 1]);
            }
            times_t<true>(e, f, pt + j * kTile16, lane);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                scale_cols(e[u], *reinterpret_cast<const float2*>(&pr.beta[row + 8 * u + c]));
#pragma unroll
                for (int x = 0; x < 4; ++x) f[u][x] = e[u][x];
                scale_cols(f[u], *reinterpret_cast<const float2*>(&pr.to_end[row + 8 * u + c]));
            }
            if (kOut) {
                // Y^T = scale g (S^T Q^T) + (b E)^T P^T
                uint32_t p0[4], p1[4], hi[4], lo[4];
                ldsm4(p0, addr16_b(pp + j * kTile16, lane));
                ldsm4(p1, addr16_b(pp + (kSubs + j) * kTile16, lane));
                split_a(hi, lo, e[0], e[1]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    scale_cols(y[u], make_float2(p.in.scale * g[u].x, p.in.scale * g[u].y));
                    mma(y[u], lo, p0[2 * u], p0[2 * u + 1]);
                    mma(y[u], hi, p1[2 * u], p1[2 * u + 1]);
                    mma(y[u], hi, p0[2 * u], p0[2 * u + 1]);
                }
            }
            update_state<true>(S, pr.g_end[j], f, kt + abt);
            if (kOut) {
                const int tr = n * C + row;
                store_tokens(yp + (size_t)tr * H * C, (size_t)H * C, T - tr, y, s.y[warp], lane);
            }
        }
        __syncthreads();
    }
    if (s_out) unit ? store_state_t(s_out, S, warp, lane) : store_state(s_out, S, warp, lane);
}

__global__ void __launch_bounds__(kTcThreads, 2)
gated_delta_chunked_kernel(const __grid_constant__ Args p) {
    previous_ended();
    const int bh = blockIdx.x / p.seg.count, seg = blockIdx.x - bh * p.seg.count, last = p.seg.count - 1;
    const float* s_in = p.s_in ? p.s_in + (size_t)bh * C * C : nullptr;
    if (seg > 0) s_in = p.seg.s + ((size_t)bh * last + seg - 1) * C * C;
    else if (last > 0 && s_in) s_in = p.seg.a + (size_t)bh * last * C * C;
    walk<true>(p, bh, seg, false, s_in, seg == last && p.s_out ? p.s_out + (size_t)bh * C * C : nullptr);
}

// B of the segments 0 .. count - 2 of a head (the first from the given state: its final state),
// then A of the segments 1 .. count - 2.
__global__ void __launch_bounds__(kTcThreads, 2)
gated_delta_maps_kernel(const __grid_constant__ Args p) {
    const int last = p.seg.count - 1, each = 2 * last - 1, bh = blockIdx.x / each, i = blockIdx.x - bh * each;
    const bool unit = i >= last;
    const int seg = unit ? i - last + 1 : i;
    float* out = (unit ? p.seg.a : p.seg.s) + ((size_t)bh * last + seg) * C * C;
    walk<false>(p, bh, seg, unit, seg == 0 && p.s_in ? p.s_in + (size_t)bh * C * C : nullptr, out);
}

Segments segments(int B, int T, int H) {
    const GdrSegments g = gdr_segments(B, T, H, 1, 2, 2.9f, 2.3f);
    return Segments{g.count, g.blocks, nullptr, nullptr};
}

template <typename Kernel>
cudaError_t run(bool first, Kernel kernel, unsigned grid, const Args& a, cudaStream_t st) {
    const size_t smem = sizeof(Smem) + 1024;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (!first) return launch_next(kernel, grid, kTcThreads, smem, st, a);
    kernel<<<grid, kTcThreads, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t gdr_chunked_bytes(int B, int T, int H) {
    return 2 * sizeof(float) * (size_t)B * H * (segments(B, T, H).count - 1) * C * C;
}

cudaError_t launch_gdr_chunked(const GdrIn& in, const float* s_in, float* s_out, void* y, void* ws, cudaStream_t st) {
    Args a{in, s_in, s_out, (bf16*)y, segments(in.B, in.T, in.H)};
    const unsigned heads = (unsigned)(in.B * in.H), last = a.seg.count - 1;
    if (last > 0) {
        a.seg.a = static_cast<float*>(ws);
        a.seg.s = a.seg.a + (size_t)heads * last * C * C;
        cudaError_t e = run(true, gated_delta_maps_kernel, heads * (2 * last - 1), a, st);
        if (e != cudaSuccess) return e;
        e = launch_gdr_join(a.seg.a, nullptr, a.seg.s, nullptr, (int)heads, (int)last, st);
        if (e != cudaSuccess) return e;
    }
    return run(last == 0, gated_delta_chunked_kernel, heads * a.seg.count, a, st);
}

}  // namespace goldwkv
