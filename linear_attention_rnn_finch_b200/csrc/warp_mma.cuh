// Device helpers of the register-resident matrix products (mma.sync m16n8k16, bf16 operands,
// fp32 sums): fragment loads from 128-byte-row tiles, hi/lo splitting, asynchronous copies.
//
// Fragments of a lane, g = lane / 4, c = 2 (lane % 4):
//   accumulator  m16 x n8:  [0,1] = row g, columns c, c+1;  [2,3] = row g + 8
//   A            m16 x k16: [0] = row g, k c, c+1;  [1] = row g + 8;  [2], [3] = k + 8
//   B            k16 x n8:  [0] = k c, c+1, column g;  [1] = k + 8
// Two accumulators side by side (columns 0-7, 8-15), packed to bf16, are an A fragment: a
// result whose row index stays a row and whose column index is contracted next never leaves
// the registers.
#pragma once

#include <stdint.h>

#include "chunk_tiles.cuh"

namespace goldwkv {
namespace wm {

using tiles::pack2;
using tiles::split2;
using tiles::sw_off;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void stsm4t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};"
                 :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void stsm4(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};"
                 :: "r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}
// d += a b
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b
__device__ __forceinline__ void mma0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void clear(float (&d)[4]) { d[0] = d[1] = d[2] = d[3] = 0.f; }

// x[0], x[2] *= s.x; x[1], x[3] *= s.y: a factor for each column
__device__ __forceinline__ void scale_cols(float (&x)[4], float2 s) {
    const float2 a = __fmul2_rn(make_float2(x[0], x[1]), s), b = __fmul2_rn(make_float2(x[2], x[3]), s);
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
}
// x = v - s x, v as two packed pairs of bf16
__device__ __forceinline__ void value_minus(float (&x)[4], float2 s, uint32_t v0, uint32_t v1) {
    const float2 n = make_float2(-s.x, -s.y);
    const float2 a = __ffma2_rn(make_float2(x[0], x[1]), n, tiles::unpack2(v0));
    const float2 b = __ffma2_rn(make_float2(x[2], x[3]), n, tiles::unpack2(v1));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
}

// Two adjacent accumulators as an A fragment in two bf16 parts: x = hi + lo within 2^-17 |x|.
__device__ __forceinline__ void split_a(uint32_t (&hi)[4], uint32_t (&lo)[4], const float (&x)[4], const float (&y)[4]) {
    split2(make_float2(x[0], x[1]), hi[0], lo[0]);
    split2(make_float2(x[2], x[3]), hi[1], lo[1]);
    split2(make_float2(y[0], y[1]), hi[2], lo[2]);
    split2(make_float2(y[2], y[3]), hi[3], lo[3]);
}

// x = a + b + c within 2^-25 |x|.
__device__ __forceinline__ void split3(float2 x, uint32_t& a, uint32_t& b, uint32_t& c) {
    a = tiles::pack2(x.x, x.y);
    const float2 d = __fadd2_rn(x, make_float2(-__uint_as_float(a << 16), -__uint_as_float(a & 0xFFFF0000u)));
    split2(d, b, c);
}
__device__ __forceinline__ void split_a3(uint32_t (&a)[4], uint32_t (&b)[4], uint32_t (&c)[4], const float (&x)[4],
                                         const float (&y)[4]) {
    split3(make_float2(x[0], x[1]), a[0], b[0], c[0]);
    split3(make_float2(x[2], x[3]), a[1], b[1], c[1]);
    split3(make_float2(y[0], y[1]), a[2], b[2], c[2]);
    split3(make_float2(y[2], y[3]), a[3], b[3], c[3]);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// ldmatrix addresses.  Tiles have 128-byte rows whose 16-byte chunks are XORed with the row
// (sw_off); `row` is the first of 16 rows, `chunk` the first of two adjacent 16-byte chunks.
// Tiles lie on 1024-byte boundaries, so that two chunks further (step) is an XOR of the address.
__device__ __forceinline__ uint32_t step(uint32_t addr, int i) { return addr ^ (uint32_t)(i << 5); }
// A operand [m][k], rows m:            registers = a[0..3]
__device__ __forceinline__ uint32_t addr_a(uint32_t tile, int row, int chunk, int lane) {
    return tile + sw_off(row + (lane & 15), chunk + (lane >> 4));
}
// B operand from [n][k] rows, 16 n:    registers = b0, b1 of the first 8 n, then of the next 8
__device__ __forceinline__ uint32_t addr_b(uint32_t tile, int row, int chunk, int lane) {
    return tile + sw_off(row + ((lane >> 4) << 3) + (lane & 7), chunk + ((lane >> 3) & 1));
}
// B operand from [k][n] rows (.trans): 16 k rows, 16 n columns: b0, b1 of n 0-7, then of n 8-15
__device__ __forceinline__ uint32_t addr_bt(uint32_t tile, int row, int chunk, int lane) {
    return tile + sw_off(row + (lane & 15), chunk + (lane >> 4));
}
// Accumulator layout of the transpose of a [n][m] bf16 tile (.trans): registers = (m 0-7, n 0-7),
// (m 8-15, n 0-7), (m 0-7, n 8-15), (m 8-15, n 8-15); also where .trans stores put it back
__device__ __forceinline__ uint32_t addr_ct(uint32_t tile, int row, int chunk, int lane) {
    return tile + sw_off(row + ((lane >> 4) << 3) + (lane & 7), chunk + ((lane >> 3) & 1));
}

}  // namespace wm
}  // namespace goldwkv
