// Sequences cut into segments when there are few heads (sm_100a).
//
// A head's chain over its blocks cannot be divided between CTAs, and few heads leave most of the
// device idle.  Its sequence can be divided: over a segment the state goes through an affine map
// S -> A S + B (A 64 x 64, the same for every value column), and the state's gradient through
// G -> A^T G + B'.  One launch forms B (the rule from a zero state), A (from the identity with
// v = 0) and B' of the segments, without outputs; this file's kernel walks the segments'
// borders; the next launch runs all segments at once from the states at their borders.
#include "common.cuh"
#include "gated_delta.h"

namespace goldwkv {

namespace {

constexpr int C = 64;
constexpr int kSms = 148;

// Forward:  m[i] = A_i m[i - 1] + m[i],       i = 1 .. last - 1;
// backward: m[i] = A_{i+1}^T m[i + 1] + m[i], i = last - 2 .. 0;  fp32, over the maps' constant
// parts.  A CTA takes 16 value columns of a head (they are independent), a thread four values of
// a row; the next A is on its way while one is multiplied: 1.2 us a border.
constexpr int kThreads = 256, kCols = 16;
template <bool kBack>
__global__ void __launch_bounds__(kThreads)
gated_delta_join_kernel(const float* __restrict__ a, float* m, int last) {
    __shared__ __align__(16) float sa[C][C + 4];
    __shared__ __align__(16) float sm[C][kCols];
    const int bh = blockIdx.x / (C / kCols), cols = kCols * (blockIdx.x % (C / kCols));
    const int row = threadIdx.x >> 2, part = threadIdx.x & 3;
    a += (size_t)bh * last * C * C + row * C + 16 * part;
    m += (size_t)bh * last * C * C + row * C + cols + 4 * part;
    float4 ra[4], rm;
    auto fetch = [&](int j) {   // step j of last - 1
        const int i = kBack ? last - 1 - j : j;
#pragma unroll
        for (int x = 0; x < 4; ++x) ra[x] = *reinterpret_cast<const float4*>(a + (size_t)(kBack ? i + 1 : i) * C * C + 4 * x);
        rm = *reinterpret_cast<const float4*>(m + (size_t)i * C * C);
    };
    *reinterpret_cast<float4*>(&sm[row][4 * part]) = *reinterpret_cast<const float4*>(m + (size_t)(kBack ? last - 1 : 0) * C * C);
    if (last > 1) fetch(1);
    for (int j = 1; j < last; ++j) {
#pragma unroll
        for (int x = 0; x < 4; ++x) *reinterpret_cast<float4*>(&sa[row][16 * part + 4 * x]) = ra[x];
        float4 x = rm;
        __syncthreads();
        if (j + 1 < last) fetch(j + 1);
#pragma unroll 16
        for (int k = 0; k < C; ++k) {
            const float4 y = *reinterpret_cast<const float4*>(&sm[k][4 * part]);
            const float f = kBack ? sa[k][row] : sa[row][k];
            x.x = fmaf(f, y.x, x.x);
            x.y = fmaf(f, y.y, x.y);
            x.z = fmaf(f, y.z, x.z);
            x.w = fmaf(f, y.w, x.w);
        }
        __syncthreads();
        *reinterpret_cast<float4*>(&sm[row][4 * part]) = x;
        *reinterpret_cast<float4*>(m + (size_t)(kBack ? last - 1 - j : j) * C * C) = x;
    }
}

}  // namespace

// By what the launches then take: a CTA needs `full` us for a block with outputs and `part`
// without, and a second CTA on an SM as long again (the schedulers are full); a border costs 1.2
// us, the launches more 6 us; a gain below a twentieth is not taken.
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
                         1.2 * (n - 2) + 6.0;
        if (t < least) {
            least = t;
            best = GdrSegments{n, each};
        }
    }
    return best;
}

cudaError_t launch_gdr_join(const float* a, float* m, int heads, int last, bool back, cudaStream_t st) {
    const unsigned grid = (unsigned)heads * (C / kCols);
    if (back) gated_delta_join_kernel<true><<<grid, kThreads, 0, st>>>(a, m, last);
    else gated_delta_join_kernel<false><<<grid, kThreads, 0, st>>>(a, m, last);
    return cudaGetLastError();
}

}  // namespace goldwkv
