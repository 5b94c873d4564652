// Backward of the gated delta rule, bf16 inputs, on tensor cores (sm_100a).  Formulas: the head of
// gated_delta_backward.cu; division of labour inside a chain: gated_delta_tiles.cuh.
//
// Two launches.  The first runs both chains over a head's blocks of 64 tokens, which need nothing
// of each other, in CTAs of their own:
//   forward:  S as in the prefill, without outputs; leaves the state entering each block and E;
//   backward: with G the gradient of a sub-chunk's final state,
//                 X = P^T dY + to_end K G,   dF = T^T (b X) = dV,
//                 G- = g_16 G + (scale g Q)^T dY - (g K)^T dF,
//             transposed like the forward one; leaves dV, each block's G and dF.
// The second, parallel over blocks, forms dQ, dK, dbeta and domega from those with the 64-token
// forms of the formulas (E and dF are the same values however tokens are grouped).  Its warps own
// tokens: products with S and G contract value columns, which the chains keep on different warps.
//
// S, G, E and dF pass between the launches as two bf16 parts (2^-17 of the value, what the
// products take anyway), transposed ([value][key] and [value][token], as the chains hold them)
// and in the 128-byte-swizzled layout of a tcgen05.mma operand.  64 KB a head and block.
#include "common.cuh"
#include "dependent_launch.cuh"
#include "gated_delta.h"
#include "gated_delta_tiles.cuh"

namespace goldwkv {

namespace {

using namespace gdr;
using bf16 = __nv_bfloat16;

constexpr int kStages = 3;
constexpr size_t kPart = kTileBytes;        // one part of a 64 x 64 matrix
constexpr size_t kMat = 2 * kPart;          // both
constexpr size_t kBlockBytes = 4 * kMat;    // S, E, G, dF of a block

struct Args {
    GdrIn in;
    GdrGrads g;
    const float* s_in;
    uint8_t* ws;     // [head][block][S, E, G, dF]: hi, then lo part of each
    int blocks;
    // segments of the sequence (gated_delta_segments.cu): A^T, A, then the states and the gradients at
    // the borders, each [head][count - 1][64][64] fp32
    GdrSegments seg;
    float *at, *a, *s, *d;
    long long budget;   // cycles a wait of the second launch may take
};

// Two adjacent accumulators of chain warp `warp` (16 value columns x 16 keys or tokens, from
// chunk 2 i of the row on) into a matrix of the workspace, as two parts, through buf (two 16 x 16
// tiles of the warp's own) so that the stores are whole sectors.
__device__ __forceinline__ void put(uint8_t* dst, const float (&x)[4], const float (&y)[4], int i, int warp, int lane,
                                    uint8_t* buf) {
    uint32_t hi[4], lo[4];
    split_a(hi, lo, x, y);
    const uint32_t at = addr16_bt(ptx::smem_addr(buf), lane);
    __syncwarp();
    stsm4(at, hi);
    stsm4(at + kTile16, lo);
    __syncwarp();
    const int row = lane >> 1;
    const uint8_t* from = buf + off16(row, lane & 1);
    uint8_t* to = dst + sw_off(16 * warp + row, 2 * i + (lane & 1));
    *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
    *reinterpret_cast<uint4*>(to + kPart) = *reinterpret_cast<const uint4*>(from + kTile16);
}

// ------------------------------------------------------------------ the chains
struct ChainSmem {
    uint8_t k[kStages][kTileBytes];
    uint8_t x[kStages][kTileBytes];   // V, or dY
    uint8_t q[kStages][kTileBytes];   // backward chain
    Prep prep[2];
    float at[kChainWarps][kSub * 20];
    uint8_t y[kChainWarps][2 * kTile16];
};

// Segment `seg` of head bh from the state (or gradient) `from` (null: zero; `unit`: the identity,
// with v = 0).  kStore: what the second launch reads, and dV; otherwise only the final matrix.
// kExact: what comes back is kept in three parts; the forward chain's E and S end in bf16 gradients
// and do with two, but for A, which carries the state's fp32 gradient too.
template <bool kBack, bool kStore, bool kExact>
__device__ __forceinline__ void chain(ChainSmem& s, const Args& p, int bh, int seg, bool unit, const float* from,
                                      float* to, float* to_t = nullptr) {
    const int H = p.in.H, HK = p.in.HK, b = bh / H, h = bh - b * H, hk = h / (H / HK);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int first = seg * p.seg.blocks, T = p.in.T - first * C, blocks = min(p.seg.blocks, p.blocks - first);
    const size_t bt = (size_t)b * p.in.T + first * C;
    const size_t ko = (bt * HK + hk) * C, vo = (bt * H + h) * C, go = bt * H + h;
    const bf16 *q = (const bf16*)p.in.q + ko, *k = (const bf16*)p.in.k + ko;
    const bf16* x = (const bf16*)(kBack ? p.g.dy : p.in.v) + vo;
    const uint32_t sk = ptx::smem_addr(s.k), sx = ptx::smem_addr(s.x), sq = ptx::smem_addr(s.q);
    // the m-th block walked
    auto block = [&](int m) { return kBack ? blocks - 1 - m : m; };

    if (warp >= kChainWarps) {   // ---- preparation
        const int w = warp - kChainWarps, pt = tid - kPrepThreads;
        const bf16 *omega = (const bf16*)p.in.omega + go, *beta = (const bf16*)p.in.beta + go;
        auto copy = [&](int m) {
            const uint32_t o = (uint32_t)(m % kStages) * kTileBytes;
            const int t0 = block(m) * C;
            copy_block<kPrepThreads>(sk + o, k, (size_t)HK * C, t0, T, pt);
            copy_block<kPrepThreads>(sx + o, x, (size_t)H * C, t0, unit ? 0 : T, pt);
            if (kBack) copy_block<kPrepThreads>(sq + o, q, (size_t)HK * C, t0, T, pt);
            cp_async_commit();
        };
        auto gate_of = [&](int m) {
            return load_gate(omega, beta, H, m < blocks ? block(m) * C + kSub * w + (lane & 15) : T, T);
        };
        copy(0);
        Gate gate = gate_of(0);
        cp_async_wait<0>();
        __syncthreads();
        for (int m = -1; m < blocks; ++m) {
            if (m + 2 < blocks) copy(m + 2);
            if (m + 1 < blocks) {
                const uint32_t o = (uint32_t)((m + 1) % kStages) * kTileBytes;
                const Gate next = gate_of(m + 2);
                prepare_sub<kBack ? 3 : 0>(s.prep[(m + 1) & 1], s.at[w], sk + o, sq + o, w, gate, p.in.scale, lane);
                gate = next;
            }
            cp_async_wait<0>();
            __syncthreads();
        }
        return;
    }

    const int c = 2 * (lane & 3);
    float S[8][4];
    if (unit) unit_state(S, warp, lane);
    else load_state(S, from, warp, lane);
    bf16* dv = (bf16*)p.g.dv + vo + 16 * warp;
    uint8_t* ws = p.ws + ((size_t)bh * p.blocks + first) * kBlockBytes + (kBack ? 2 * kMat : 0);
    const uint32_t ab = addr_b(0, 0, 0, lane), abt = addr_bt(0, 0, 0, lane), act = addr_ct(0, 0, 2 * warp, lane);
    __syncthreads();
    __syncthreads();   // the preparation's first turn
    for (int m = 0; m < blocks; ++m) {
        const uint32_t o = (uint32_t)(m % kStages) * kTileBytes;
        const int t0 = block(m) * C;
        const Prep& pr = s.prep[m & 1];
        const uint32_t pt = ptx::smem_addr(pr.t), pp = ptx::smem_addr(pr.p);
        uint8_t* wb = ws + (size_t)block(m) * kBlockBytes;
        if (kStore) {
#pragma unroll
            for (int i = 0; i < 4; ++i) put(wb, S[2 * i], S[2 * i + 1], i, warp, lane, s.y[warp]);
        }
#pragma unroll 2
        for (int i0 = 0; i0 < kSubs; ++i0) {
            const int j = kBack ? kSubs - 1 - i0 : i0, row = kSub * j;
            const uint32_t kt = sk + o + row * 128;
            float f[2][4], e[2][4];   // S^T K^T (or G^T K^T)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t a0[4], a1[4], a2[4], kb[4];
                ldsm4(kb, step(kt + ab, i));
                if (kExact) split_a3(a0, a1, a2, S[2 * i], S[2 * i + 1]);
                else split_a(a0, a1, S[2 * i], S[2 * i + 1]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {   // the first part and the smaller ones in sums of their own
                    if (i == 0) {
                        mma0(f[u], a0, kb[2 * u], kb[2 * u + 1]);
                        mma0(e[u], a1, kb[2 * u], kb[2 * u + 1]);
                    } else {
                        mma(f[u], a0, kb[2 * u], kb[2 * u + 1]);
                        mma(e[u], a1, kb[2 * u], kb[2 * u + 1]);
                    }
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    if (kExact) mma(e[u], a2, kb[2 * u], kb[2 * u + 1]);
            }
            uint32_t xv[4];   // V^T or dY^T, as the A operand [value][token]
            ldsm4t(xv, sx + o + row * 128 + act);
            float2 g[2], bt[2], te[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                g[u] = *reinterpret_cast<const float2*>(&pr.g[row + 8 * u + c]);
                bt[u] = *reinterpret_cast<const float2*>(&pr.beta[row + 8 * u + c]);
                te[u] = *reinterpret_cast<const float2*>(&pr.to_end[row + 8 * u + c]);
#pragma unroll
                for (int n = 0; n < 4; ++n) f[u][n] += e[u][n];
            }
            if (!kBack) {
#pragma unroll
                for (int u = 0; u < 2; ++u) value_minus(f[u], g[u], xv[2 * u], xv[2 * u + 1]);
                times_t<kExact>(e, f, pt + j * kTile16, lane);
                if (kStore) put(wb + kMat, e[0], e[1], j, warp, lane, s.y[warp]);
#pragma unroll
                for (int u = 0; u < 2; ++u) scale_cols(e[u], make_float2(bt[u].x * te[u].x, bt[u].y * te[u].y));
                update_state<kExact>(S, pr.g_end[j], e, kt + abt);
            } else {
                // X^T = to_end G^T K^T + dY^T P
                uint32_t p0[4], p1[4], p2[4];
                ldsm4t(p0, addr16_bt(pp + j * kTile16, lane));
                ldsm4t(p1, addr16_bt(pp + (kSubs + j) * kTile16, lane));
                ldsm4t(p2, addr16_bt(pp + (2 * kSubs + j) * kTile16, lane));
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    scale_cols(f[u], te[u]);
                    mma(f[u], xv, p2[2 * u], p2[2 * u + 1]);
                    mma(f[u], xv, p1[2 * u], p1[2 * u + 1]);
                    mma(f[u], xv, p0[2 * u], p0[2 * u + 1]);
                    scale_cols(f[u], bt[u]);
                }
                times_t<kExact, true>(e, f, pt + j * kTile16, lane);
                if (kStore)
                    store_tokens(dv + (size_t)(t0 + row) * H * C, (size_t)H * C, T - t0 - row, e, s.y[warp], lane);
                if (kStore) put(wb + kMat, e[0], e[1], j, warp, lane, s.y[warp]);
                // G^T = g_16 G^T + (scale g dY)^T Q - (g dF)^T K
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const float2 y0 = tiles::unpack2(xv[2 * u]), y1 = tiles::unpack2(xv[2 * u + 1]);
                    f[u][0] = y0.x;
                    f[u][1] = y0.y;
                    f[u][2] = y1.x;
                    f[u][3] = y1.y;
                    scale_cols(f[u], make_float2(p.in.scale * g[u].x, p.in.scale * g[u].y));
                    scale_cols(e[u], make_float2(-g[u].x, -g[u].y));
                }
                update_state<kExact, true>(S, pr.g_end[j], e, kt + abt, f, kt + abt + (sq - sk));
            }
        }
        __syncthreads();
    }
    if (to) store_state(to, S, warp, lane);
    if (unit) store_state_t(to_t, S, warp, lane);
}

// The chains of a head's segments, the longer ones (backward) first.
__global__ void __launch_bounds__(kTcThreads, 2)
gated_delta_bwd_chains_kernel(const __grid_constant__ Args p) {
    extern __shared__ __align__(16) uint8_t raw[];
    ChainSmem& s = tiles::smem_aligned<ChainSmem>(raw);
    previous_ended();
    const int n = p.seg.count, last = n - 1, half = (int)(gridDim.x >> 1);
    const bool back = (int)blockIdx.x < half;
    const int i = back ? blockIdx.x : blockIdx.x - half, bh = i / n, seg = i - bh * n;
    const size_t at = (size_t)bh * C * C, border = (size_t)bh * last;
    if (back)
        chain<true, true, true>(s, p, bh, seg, false,
                          seg < last ? p.d + (border + seg) * C * C : p.g.ds_out ? p.g.ds_out + at : nullptr,
                          seg == 0 && p.g.ds_in ? p.g.ds_in + at : nullptr);
    else
        chain<false, true, false>(s, p, bh, seg, false,
                           seg > 0 ? p.s + (border + seg - 1) * C * C : p.s_in ? p.s_in + at : nullptr, nullptr);
}

// B of the segments 0 .. count - 2 (the first from the given state), A of 1 .. count - 2, and B' of
// 1 .. count - 1 (the last from the given gradient).
__global__ void __launch_bounds__(kTcThreads, 2)
gated_delta_bwd_maps_kernel(const __grid_constant__ Args p) {
    extern __shared__ __align__(16) uint8_t raw[];
    ChainSmem& s = tiles::smem_aligned<ChainSmem>(raw);
    const int last = p.seg.count - 1, each = 3 * last - 1, bh = blockIdx.x / each, i = blockIdx.x - bh * each;
    const size_t at = (size_t)bh * C * C, border = (size_t)bh * last;
    if (i < last) {
        const int seg = i + 1;
        chain<true, false, true>(s, p, bh, seg, false, seg == last && p.g.ds_out ? p.g.ds_out + at : nullptr,
                           p.d + (border + i) * C * C);
    } else if (i < 2 * last) {
        const int seg = i - last;
        chain<false, false, false>(s, p, bh, seg, false, seg == 0 && p.s_in ? p.s_in + at : nullptr,
                            p.s + (border + seg) * C * C);
    } else {
        const int seg = i - 2 * last + 1;
        chain<false, false, true>(s, p, bh, seg, true, nullptr, p.a + (border + seg) * C * C, p.at + (border + seg) * C * C);
    }
}

// ------------------------------------------------------------------ dQ, dK, dbeta, domega
// A CTA per key head and block; 64 x 64 x 64 products on tcgen05 (M = N = 64, fp32 in TMEM), three
// groups a value head, each issued by one thread once the last one's results are read:
//     dY S^T, dF S^T, E G^T and Q K^T;   K K^T, dY E^T and dF E^T;   dP K and dP^T Q + (dM + dM^T) K,
// dP and dM, as two bf16 parts, over S and G's place.  Warp (w, half) reads tokens
// 16 w .. 16 w + 15 and 32 columns of each result, in mma accumulator layout.  256 TMEM columns,
// 94 KB and 128 registers: two CTAs an SM, of which one loads while the other computes.  (The same
// on mma.sync: operand loads kept the shared-memory pipe 60 % busy, at B8 T4096 H32 749 us against
// 530.)
constexpr int kOutThreads = 256;
constexpr uint32_t kTmemCols = 256;
constexpr long long kDrain = 2000000000LL;   // cycles the last wait may take: about a second

struct OutSmem {
    uint8_t q[kTileBytes], k[kTileBytes], dy[kTileBytes];
    union {
        struct {
            uint8_t s[kMat], g[kMat];                       // [value][key]
        };
        struct {
            uint8_t dp[2][kTileBytes], dm[2][kTileBytes];   // [t][s]
        };
    };
    uint8_t e[kMat], df[kMat];                              // [value][token]
    Gates gates;
    float cols[4][C];      // column sums of P dY E - M dF E over each row tile
    float rows[4][C];      // [s tile][t]: row sums of the same, times b_s, left of the diagonal
    float reads[2][C], kte[2][C];
    float gs[8];
    float diag[C];         // the same over a token's own tile: rows from it on, columns before it
    uint64_t done;
    uint32_t tmem;
    int late;              // a wait ran out
};

// D (+)= A B over one 64 x 64 x 64 product.  kA, kB: the operand's rows are the contracted index
// (MN-major: 16 of them are 2048 bytes on), else its own (K-major: 16 k are 32 bytes on).
template <bool kA, bool kB>
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint32_t b, bool add) {
    const uint64_t da = kA ? ptx::desc_mnmajor(a) : ptx::desc_kmajor(a), db = kB ? ptx::desc_mnmajor(b) : ptx::desc_kmajor(b);
    constexpr uint32_t kDesc = ptx::idesc_bf16(64, 64, kA, kB);
#pragma unroll
    for (int k = 0; k < 4; ++k)   // addresses count in 16 bytes
        ptx::mma_bf16(d, da + (kA ? 128 : 2) * k, db + (kB ? 128 : 2) * k, kDesc, add || k > 0);
}

// Sums over the eight lanes that share columns c, c + 1, 8 + c, 9 + c (x[0..3]): each step a lane
// hands half of its columns over and keeps the other.  Lane l < 16 returns column column_of(l)'s.
__device__ __forceinline__ float column_sums(const float (&x)[4], int lane) {
    const bool a = lane & 4, b = lane & 8;
    float k0 = a ? x[2] : x[0], k1 = a ? x[3] : x[1];
    k0 += __shfl_xor_sync(0xffffffffu, a ? x[0] : x[2], 4);
    k1 += __shfl_xor_sync(0xffffffffu, a ? x[1] : x[3], 4);
    float k = b ? k1 : k0;
    k += __shfl_xor_sync(0xffffffffu, b ? k0 : k1, 8);
    return k + __shfl_xor_sync(0xffffffffu, k, 16);
}
__device__ __forceinline__ int column_of(int lane) { return 2 * (lane & 3) + 8 * ((lane >> 2) & 1) + ((lane >> 3) & 1); }

__global__ void __launch_bounds__(kOutThreads, 2)
gated_delta_bwd_out_tc_kernel(const __grid_constant__ Args p) {
    extern __shared__ __align__(16) uint8_t raw[];
    OutSmem& s = tiles::smem_aligned<OutSmem>(raw);
    const int n = blockIdx.x % p.blocks, bk = blockIdx.x / p.blocks;
    const int H = p.in.H, HK = p.in.HK, T = p.in.T, b = bk / HK, hk = bk - b * HK, per = H / HK;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, w = warp & 3, half = warp >> 2;
    const int r = lane >> 2, c = 2 * (lane & 3);
    const int t0 = n * C, row = kSub * w;
    const size_t ko = ((size_t)b * T * HK + hk) * C;
    const uint32_t sq = ptx::smem_addr(s.q), sk = ptx::smem_addr(s.k), sy = ptx::smem_addr(s.dy);
    const uint32_t ss = ptx::smem_addr(s.s), sg = ptx::smem_addr(s.g), se = ptx::smem_addr(s.e), sf = ptx::smem_addr(s.df);
    if (tid == 0) {
        ptx::mbar_init(&s.done, 1);
        ptx::fence_mbar_init();
        s.late = 0;
    }
    if (warp == 0) ptx::tmem_alloc(&s.tmem, kTmemCols);
    copy_block<kOutThreads>(sq, (const bf16*)p.in.q + ko, (size_t)HK * C, t0, T, tid);
    copy_block<kOutThreads>(sk, (const bf16*)p.in.k + ko, (size_t)HK * C, t0, T, tid);
    previous_ended();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tm = s.tmem, tw = tm + ((uint32_t)(32 * w) << 16);   // this warp's lanes
    // one thread issues; the warp's number through a shuffle, so that the branch and with it the
    // descriptors stay in uniform registers
    const bool issuer = __shfl_sync(0xffffffffu, warp, 0) == 0;
    uint32_t phase = 0;
    // all wait for the group last issued; bounded, and once late no more waits and no more products
    auto arrived = [&] {
        if (!s.late && !ptx::mbar_wait(&s.done, phase, p.budget)) s.late = 1;
        phase ^= 1;
        ptx::tc_fence_after();
    };
    // before the next group: TMEM is read, shared memory written
    auto ready = [&] {
        ptx::tc_fence_before();
        ptx::fence_proxy_async_smem();
        return __syncthreads_or(s.late) == 0;
    };
    float dq[4][4], dk[4][4];   // key tiles 4 half .. 4 half + 3
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        clear(dq[i]);
        clear(dk[i]);
    }
    bool good = true;
    for (int h = hk * per; h < (hk + 1) * per && good; ++h) {
        const size_t bh = (size_t)b * H + h;
        const uint8_t* wb = p.ws + (bh * p.blocks + n) * kBlockBytes;   // S, E, G, dF
        const auto raw_gates = fetch_gates((const bf16*)p.in.omega, (const bf16*)p.in.beta, (size_t)b * T * H + h, H, t0, T);
        copy_block<kOutThreads>(sy, (const bf16*)p.g.dy + ((size_t)b * T * H + h) * C, (size_t)H * C, t0, T, tid);
#pragma unroll
        for (int i = 0; i < (int)(kMat / 16 / kOutThreads); ++i) {
            const int o = (i * kOutThreads + tid) * 16;
            cp_async16(ss + o, wb + o, true);
            cp_async16(se + o, wb + kMat + o, true);
            cp_async16(sg + o, wb + 2 * kMat + o, true);
            cp_async16(sf + o, wb + 3 * kMat + o, true);
        }
        cp_async_commit();
        put_gates(s.gates, raw_gates, t0, T);
        cp_async_wait<0>();
        if (!(good = ready())) break;
        if (issuer && ptx::elect_one()) {   // the smallest terms first
            ptx::tc_fence_after();
            product<false, true>(tm, sy, ss + kPart, false);
            product<false, true>(tm, sy, ss, true);
            product<true, true>(tm + 64, sf + kPart, ss, false);
            product<true, true>(tm + 64, sf, ss + kPart, true);
            product<true, true>(tm + 64, sf, ss, true);
            product<true, true>(tm + 128, se + kPart, sg, false);
            product<true, true>(tm + 128, se, sg + kPart, true);
            product<true, true>(tm + 128, se, sg, true);
            ptx::mma_commit(&s.done);
            product<false, false>(tm + 192, sq, sk, false);   // awaited with the next group
        }
        // <G, S>
        {
            float gs = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int o = (i * kOutThreads + tid) * 16;
                const uint4 a = *reinterpret_cast<const uint4*>(s.s + o), al = *reinterpret_cast<const uint4*>(s.s + kPart + o);
                const uint4 d = *reinterpret_cast<const uint4*>(s.g + o), dl = *reinterpret_cast<const uint4*>(s.g + kPart + o);
                const uint32_t av[4] = {a.x, a.y, a.z, a.w}, alv[4] = {al.x, al.y, al.z, al.w};
                const uint32_t dv[4] = {d.x, d.y, d.z, d.w}, dlv[4] = {dl.x, dl.y, dl.z, dl.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 x = tiles::unpack2(av[e]), xl = tiles::unpack2(alv[e]);
                    const float2 y = tiles::unpack2(dv[e]), yl = tiles::unpack2(dlv[e]);
                    gs = fmaf(x.x + xl.x, y.x + yl.x, gs);
                    gs = fmaf(x.y + xl.y, y.y + yl.y, gs);
                }
            }
            gs = warp_sum(gs);
            if (lane == 0) s.gs[warp] = gs;
        }
        arrived();
        // ---- with the states: dK += b to_end (E G^T) - g (dF S^T), dQ += scale g (dY S^T)
        {
            uint32_t x1[16], x2[16], x3[16];
            tiles::tmem_ld16x4(tw + 32 * half, x1);
            tiles::tmem_ld16x4(tw + 64 + 32 * half, x2);
            tiles::tmem_ld16x4(tw + 128 + 32 * half, x3);
            ptx::tmem_wait_ld();
            float ke[2] = {0.f, 0.f}, rd[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int t = row + r + 8 * e;
                const float gt = s.gates.g[t], sgt = p.in.scale * gt, te = s.gates.to_end[t], bt = s.gates.beta[t];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t o = sw_off(t, 4 * half + i) + 2 * c;
                    const float2 qv = tiles::unpack2(tiles::lds32(s.q, o)), kv = tiles::unpack2(tiles::lds32(s.k, o));
                    const float y0 = sgt * __uint_as_float(x1[4 * i + 2 * e]), y1 = sgt * __uint_as_float(x1[4 * i + 2 * e + 1]);
                    const float f0 = gt * __uint_as_float(x2[4 * i + 2 * e]), f1 = gt * __uint_as_float(x2[4 * i + 2 * e + 1]);
                    const float v0 = te * __uint_as_float(x3[4 * i + 2 * e]), v1 = te * __uint_as_float(x3[4 * i + 2 * e + 1]);
                    dq[i][2 * e] += y0;
                    dq[i][2 * e + 1] += y1;
                    dk[i][2 * e] += fmaf(bt, v0, -f0);
                    dk[i][2 * e + 1] += fmaf(bt, v1, -f1);
                    ke[e] = fmaf(kv.x, v0, fmaf(kv.y, v1, ke[e]));
                    rd[e] += (qv.x * y0 - kv.x * f0) + (qv.y * y1 - kv.y * f1);
                }
                ke[e] += __shfl_xor_sync(0xffffffffu, ke[e], 1);
                rd[e] += __shfl_xor_sync(0xffffffffu, rd[e], 1);
                ke[e] += __shfl_xor_sync(0xffffffffu, ke[e], 2);
                rd[e] += __shfl_xor_sync(0xffffffffu, rd[e], 2);
                if ((lane & 3) == 0) {
                    s.kte[half][t] = ke[e];
                    s.reads[half][t] = rd[e];
                }
            }
        }
        if (!(good = ready())) break;
        if (issuer && ptx::elect_one()) {
            ptx::tc_fence_after();
            product<false, false>(tm, sk, sk, false);
            product<false, true>(tm + 64, sy, se + kPart, false);
            product<false, true>(tm + 64, sy, se, true);
            product<true, true>(tm + 128, sf + kPart, se, false);
            product<true, true>(tm + 128, sf, se + kPart, true);
            product<true, true>(tm + 128, sf, se, true);
            ptx::mma_commit(&s.done);
        }
        arrived();
        // ---- the triangles: two tiles of 16 x 16 a warp, those above the diagonal zero
#pragma unroll 1
        for (int v = 2 * half; v < 2 * half + 2; ++v) {
            const int ar = row + r;
            uint32_t ph[4] = {0, 0, 0, 0}, pl[4] = {0, 0, 0, 0}, mh[4] = {0, 0, 0, 0}, ml[4] = {0, 0, 0, 0};
            if (v <= w) {
                uint32_t kk[8], ye[8], fe[8], qk[8];
                tiles::tmem_ld16x2_256(tw + 16 * v, kk);
                tiles::tmem_ld16x2_256(tw + 64 + 16 * v, ye);
                tiles::tmem_ld16x2_256(tw + 128 + 16 * v, fe);
                tiles::tmem_ld16x2_256(tw + 192 + 16 * v, qk);
                ptx::tmem_wait_ld();
                const float hh[2] = {s.gates.hi[ar], s.gates.hi[ar + 8]}, ll[2] = {s.gates.lo[ar], s.gates.lo[ar + 8]};
                float cs[4], rw[2] = {0.f, 0.f}, dp[2][4], dm[2][4], wt[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int cl = 8 * u + c + (x & 1), sc = kSub * v + cl, rl = r + 8 * (x >> 1);
                        const bool on = v < w || rl >= cl;
                        float d = tiles::fast_exp2((hh[x >> 1] - s.gates.hi[sc]) + (ll[x >> 1] - s.gates.lo[sc]));
                        d = on ? d : 0.f;   // above the diagonal it may be infinite
                        const float bs = s.gates.beta[sc], db = d * bs;
                        const float y = on ? p.in.scale * __uint_as_float(ye[4 * u + x]) : 0.f;
                        const float f = v < w || rl > cl ? __uint_as_float(fe[4 * u + x]) : 0.f;
                        const float sum = d * (__uint_as_float(qk[4 * u + x]) * y - __uint_as_float(kk[4 * u + x]) * f);
                        if (x < 2) cs[2 * u + x] = sum;
                        else cs[2 * u + x - 2] += sum;
                        wt[u][x] = v < w || rl > cl ? bs * sum : 0.f;
                        rw[x >> 1] += wt[u][x];
                        dp[u][x] = db * y;
                        dm[u][x] = -db * f;
                    }
                if (v == w) {
                    // inside the diagonal tile: for each column u the sum over rows from u on of
                    // the row's entries before u
                    float before[2][4];
                    const int q = lane & 3;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float left = 0.f;   // the row's first eight columns
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float pair = wt[u][2 * e] + wt[u][2 * e + 1];
                            float x = __shfl_up_sync(0xffffffffu, pair, 1, 4);
                            float run = q > 0 ? x : 0.f;
                            x = __shfl_up_sync(0xffffffffu, run + pair, 2, 4);
                            // run: the pair before; x: the two before that one
                            run += q > 1 ? x : 0.f;
                            before[u][2 * e] = left + run;
                            before[u][2 * e + 1] = left + run + wt[u][2 * e];
                            left = __shfl_sync(0xffffffffu, run + pair, 3, 4);
                        }
                    }
                    float ds[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int u = x >> 1, cl = 8 * u + c + (x & 1);
                        ds[x] = (r >= cl ? before[u][x & 1] : 0.f) + (r + 8 >= cl ? before[u][2 + (x & 1)] : 0.f);
                    }
                    const float dsum = column_sums(ds, lane);
                    if (lane < 16) s.diag[row + column_of(lane)] = dsum;
                }
                // column sums over the tile's rows, row sums over its columns
                const float col = column_sums(cs, lane);
                if (lane < 16) s.cols[w][kSub * v + column_of(lane)] = col;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    rw[e] += __shfl_xor_sync(0xffffffffu, rw[e], 1);
                    rw[e] += __shfl_xor_sync(0xffffffffu, rw[e], 2);
                    if ((lane & 3) == 0) s.rows[v][ar + 8 * e] = rw[e];   // read where v < w
                }
                split_a(ph, pl, dp[0], dp[1]);
                split_a(mh, ml, dm[0], dm[1]);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t o = sw_off(ar + 8 * (x & 1), 2 * v + (x >> 1)) + 2 * c;
                tiles::sts32(s.dp[0], o, ph[x]);
                tiles::sts32(s.dp[1], o, pl[x]);
                tiles::sts32(s.dm[0], o, mh[x]);
                tiles::sts32(s.dm[1], o, ml[x]);
            }
        }
        if (!(good = ready())) break;
        if (issuer && ptx::elect_one()) {
            const uint32_t sp = ptx::smem_addr(s.dp), sm = ptx::smem_addr(s.dm);
            ptx::tc_fence_after();
            product<false, true>(tm, sp + kTileBytes, sk, false);
            product<false, true>(tm, sp, sk, true);
            product<true, true>(tm + 64, sp + kTileBytes, sq, false);
            product<false, true>(tm + 64, sm + kTileBytes, sk, true);
            product<true, true>(tm + 64, sm + kTileBytes, sk, true);
            product<true, true>(tm + 64, sp, sq, true);
            product<false, true>(tm + 64, sm, sk, true);
            product<true, true>(tm + 64, sm, sk, true);
            ptx::mma_commit(&s.done);
        }
        // ---- dbeta and domega of the row tile's 16 tokens, a lane a token (lanes 16-31 repeat them)
        if (half == 1) {   // not the issuing warp
            const int l = lane & 15, t = row + l;
            // rows of this tile from t on, columns of the tiles to the left
            float rs = s.reads[0][t] + s.reads[1][t];
            for (int v = 0; v < w; ++v) rs += s.rows[v][t];
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) {   // from the last token back
                const float x = __shfl_down_sync(0xffffffffu, rs, o, 16);
                if (l + o < 16) rs += x;
            }
            float later = 0.f;                   // reads of the tiles below
            for (int i = row + kSub + lane; i < C; i += 32) later += s.reads[0][i] + s.reads[1][i];
            // columns before t in the rows of the tiles below, and the sources before t
            float before = 0.f;
            for (int i = lane; i < row; i += 32) {
                float x = s.kte[0][i] + s.kte[1][i];
                for (int a = w + 1; a < 4; ++a) x += s.cols[a][i];
                before = fmaf(s.gates.beta[i], x, before);
            }
            later = warp_sum(later);
            before = warp_sum(before);
            const float kte = s.kte[0][t] + s.kte[1][t];
            float own = kte;
            for (int a = w + 1; a < 4; ++a) own += s.cols[a][t];
            const float db = own + s.cols[w][t];
            float pre = s.gates.beta[t] * own;
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) {
                const float x = __shfl_up_sync(0xffffffffu, pre, o, 16);
                if (l >= o) pre += x;
            }
            pre = __shfl_up_sync(0xffffffffu, pre, 1, 16);
            if (l == 0) pre = 0.f;
            float gsum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) gsum += s.gs[i];
            const float dl = ((s.diag[t] + rs) + later) + (before + pre) + s.gates.g[C - 1] * gsum;
            if (lane < 16 && t0 + t < T) {
                const size_t o = ((size_t)b * T + t0 + t) * H + h;
                ((bf16*)p.g.domega)[o] = __float2bfloat16_rn(-s.gates.rate[t] * dl);
                ((bf16*)p.g.dbeta)[o] = __float2bfloat16_rn(db);
            }
        }
        arrived();
        {
            uint32_t x1[16], x2[16];
            tiles::tmem_ld16x4(tw + 32 * half, x1);
            tiles::tmem_ld16x4(tw + 64 + 32 * half, x2);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dq[i][e] += __uint_as_float(x1[4 * i + e]);
                    dk[i][e] += __uint_as_float(x2[4 * i + e]);
                }
        }
        good = ready();   // also: this head's tiles may be overwritten
    }
    // late: NaN results; the products issued may be running still, on tiles and columns that others
    // get next.  They have a second's time: the group last committed, then what went out behind it
    // (Q K^T, behind the first group), for which a commit of its own answers.
    if (!good) {
        (void)ptx::mbar_wait(&s.done, phase ^ 1, kDrain);
        if (issuer && ptx::elect_one()) ptx::mma_commit(&s.done);
        (void)ptx::mbar_wait(&s.done, phase, kDrain);
        const float nan = __int_as_float(0x7fffffff);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) dq[i][e] = dk[i][e] = nan;
        for (int i = tid; i < per * C; i += kOutThreads)
            if (t0 + i % C < T) {
                const size_t o = ((size_t)b * T + t0 + i % C) * H + hk * per + i / C;
                ((bf16*)p.g.domega)[o] = ((bf16*)p.g.dbeta)[o] = __float2bfloat16_rn(nan);
            }
    }
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == 0) ptx::tmem_dealloc(tm, kTmemCols);
    // out through Q's and K's places: whole rows of 128 bytes
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t o = sw_off(row + r + 8 * x, 4 * half + i) + 2 * c;
            tiles::sts32(s.q, o, pack2(dq[i][2 * x], dq[i][2 * x + 1]));
            tiles::sts32(s.k, o, pack2(dk[i][2 * x], dk[i][2 * x + 1]));
        }
    __syncthreads();
    bf16 *oq = (bf16*)p.g.dq + ko, *ok = (bf16*)p.g.dk + ko;
#pragma unroll
    for (int i = 0; i < C * 8 / kOutThreads; ++i) {
        const int t = (tid >> 3) + i * (kOutThreads / 8), ch = tid & 7;
        if (t0 + t < T) {
            const size_t o = (size_t)(t0 + t) * HK * C + 8 * ch;
            *reinterpret_cast<uint4*>(oq + o) = *reinterpret_cast<const uint4*>(s.q + sw_off(t, ch));
            *reinterpret_cast<uint4*>(ok + o) = *reinterpret_cast<const uint4*>(s.k + sw_off(t, ch));
        }
    }
}

template <typename Kernel>
cudaError_t run(bool first, Kernel kernel, unsigned grid, int threads, size_t smem, const Args& a, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (!first) return launch_next(kernel, grid, threads, smem, st, a);
    kernel<<<grid, threads, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

static GdrSegments segments(int B, int T, int H) { return gdr_segments(B, T, H, 2, 3, 3.4f, 3.0f); }

size_t gdr_backward_tc_bytes(int B, int T, int H) {
    const size_t heads = (size_t)B * H;
    return heads * ((T + C - 1) / C) * kBlockBytes +
           4 * sizeof(float) * heads * (segments(B, T, H).count - 1) * C * C;
}

cudaError_t launch_gdr_backward_tc(const GdrIn& in, const float* s_in, const GdrGrads& g, void* ws, long long budget,
                                   cudaStream_t st) {
    Args a{in, g, s_in, static_cast<uint8_t*>(ws), (in.T + C - 1) / C, segments(in.B, in.T, in.H),
           nullptr, nullptr, nullptr, nullptr, budget};
    const unsigned heads = (unsigned)(in.B * in.H), last = a.seg.count - 1;
    const size_t smem = sizeof(ChainSmem) + 1024;
    cudaError_t e;
    if (last > 0) {
        a.at = reinterpret_cast<float*>(a.ws + (size_t)heads * a.blocks * kBlockBytes);
        a.a = a.at + (size_t)heads * last * C * C;
        a.s = a.a + (size_t)heads * last * C * C;
        a.d = a.s + (size_t)heads * last * C * C;
        e = run(true, gated_delta_bwd_maps_kernel, heads * (3 * last - 1), kTcThreads, smem, a, st);
        if (e == cudaSuccess) e = launch_gdr_join(a.at, a.a, a.s, a.d, (int)heads, (int)last, st);
        if (e != cudaSuccess) return e;
    }
    e = run(last == 0, gated_delta_bwd_chains_kernel, 2u * heads * a.seg.count, kTcThreads, smem, a, st);
    if (e != cudaSuccess) return e;
    return run(false, gated_delta_bwd_out_tc_kernel, (unsigned)(in.B * in.HK) * (unsigned)a.blocks, kOutThreads,
               sizeof(OutSmem) + 1024, a, st);
}

}  // namespace goldwkv
