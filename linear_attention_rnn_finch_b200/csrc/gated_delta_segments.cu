// Sequences cut into segments when there are few heads (sm_100a).
//
// A head's chain over its blocks cannot be divided between CTAs, and few heads leave most of the
// device idle.  Its sequence can be divided: over a segment the state goes through an affine map
// S -> A S + B (A 64 x 64, the same for every value column), and the state's gradient through
// G -> A^T G + B'.  One launch forms B (the rule from a zero state), A (from the identity with
// v = 0) and B' of the segments, without outputs; this file's kernel walks the segments'
// borders; the next launch runs all segments at once from the states at their borders.
#include "common.cuh"
#include "dependent_launch.cuh"
#include "gated_delta.h"

namespace goldwkv {

namespace {

constexpr int C = 64;
constexpr int kSms = 148;

// Forward:  m[i] = A_i m[i - 1] + m[i],       i = 1 .. last - 1;
// backward: m[i] = A_{i+1}^T m[i + 1] + m[i], i = last - 2 .. 0;  fp32, over the maps' constant
// parts.  A CTA takes 4 value columns of a head (they are independent).  Lanes are rows, a warp
// contracts 16 of the 64 k for 32 of them: its 16 values of A (of A^T forward, so that lanes read
// adjacent ones) come straight into registers, two borders ahead, and the matrix multiplied is
// read from shared memory by all lanes alike.  The four warps of a row are added up in shared
// memory.  0.58 us a border (with A in shared memory too, four results a thread, 1.9).
constexpr int kThreads = 256, kCols = 4;
template <bool kBack>
__device__ __forceinline__ void join(const float* __restrict__ a, float* m, int last, int cta) {
    __shared__ __align__(16) float sm[C][kCols];
    __shared__ __align__(16) float red[4][C][kCols];
    const int bh = cta / (C / kCols), cols = kCols * (cta % (C / kCols));
    const int tid = threadIdx.x, warp = tid >> 5, row = 32 * (warp & 1) + (tid & 31), part = warp >> 1;
    a += (size_t)bh * last * C * C + 16 * part * C + row;
    const int orow = tid >> 2, ocol = tid & 3;   // this thread's result
    m += (size_t)bh * last * C * C + orow * C + cols + ocol;
    struct Step {
        float a[16];
        float m;
    };
    auto fetch = [&](Step& s, int j) {   // step j of last - 1
        if (j >= last) return;
        const int i = kBack ? last - 1 - j : j;
        const float* from = a + (size_t)(kBack ? i + 1 : i) * C * C;
#pragma unroll
        for (int k = 0; k < 16; ++k) s.a[k] = from[k * C];
        s.m = m[(size_t)i * C * C];
    };
    Step next[2];
    fetch(next[0], 1);
    fetch(next[1], 2);
    sm[orow][ocol] = m[(size_t)(kBack ? last - 1 : 0) * C * C];
    __syncthreads();
    auto border = [&](Step& s, int j) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float4 x = *reinterpret_cast<const float4*>(sm[16 * part + k]);
            acc.x = fmaf(s.a[k], x.x, acc.x);
            acc.y = fmaf(s.a[k], x.y, acc.y);
            acc.z = fmaf(s.a[k], x.z, acc.z);
            acc.w = fmaf(s.a[k], x.w, acc.w);
        }
        *reinterpret_cast<float4*>(red[part][row]) = acc;
        const float x = s.m;
        fetch(s, j + 2);
        __syncthreads();
        const float sum = x + ((red[0][orow][ocol] + red[1][orow][ocol]) + (red[2][orow][ocol] + red[3][orow][ocol]));
        sm[orow][ocol] = sum;
        m[(size_t)(kBack ? last - 1 - j : j) * C * C] = sum;
        __syncthreads();
    };
    for (int j = 1; j < last; j += 2) {
        border(next[0], j);
        if (j + 1 < last) border(next[1], j + 1);
    }
}

// The states, and behind them (where d is given) the gradients.
__global__ void __launch_bounds__(kThreads)
gated_delta_join_kernel(const float* __restrict__ at, const float* __restrict__ a, float* s, float* d, int last, int ctas) {
    previous_ended();
    if ((int)blockIdx.x < ctas) join<false>(behind(at), s, last, blockIdx.x);
    else join<true>(behind(a), d, last, blockIdx.x - ctas);
}

}  // namespace

// By what the launches then take: a CTA needs `full` us for a block with outputs and `part`
// without, and a second CTA on an SM as long again (the schedulers are full); a border costs 0.6
// us, the launches more and their first loads 12 us; a gain below a twentieth is not taken.
GdrSegments gdr_segments(int B, int T, int H, int ctas, int maps, float full, float part) {
    const int blocks = (T + C - 1) / C;
    const long heads = (long)B * H;
    auto turns = [](long n) { return (double)((n + kSms - 1) / kSms); };
    GdrSegments best{1, blocks};
    double least = 0.95 * turns(heads * ctas) * blocks * full;
    for (int want = 2; want <= 64 && heads * want <= 4 * kSms && 4 * want <= blocks; ++want) {
        const int each = (blocks + want - 1) / want, n = (blocks + each - 1) / each;
        if (n < 2) continue;
        const double t = each * (turns(heads * (maps * (n - 1) - 1)) * part + turns(heads * n * ctas) * full) +
                         0.6 * (n - 2) + 12.0;
        if (t < least) {
            least = t;
            best = GdrSegments{n, each};
        }
    }
    return best;
}

cudaError_t launch_gdr_join(const float* at, const float* a, float* s, float* d, int heads, int last, cudaStream_t st) {
    const int ctas = heads * (C / kCols);
    return launch_next(gated_delta_join_kernel, (unsigned)(d ? 2 * ctas : ctas), kThreads, 0, st, at, a, s, d, last, ctas);
}

}  // namespace goldwkv
