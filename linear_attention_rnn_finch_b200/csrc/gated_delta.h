// Launchers of the gated delta rule (not exported).  Contracts: include/goldwkv.h,
// gated_delta_*.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace goldwkv {

// Inputs of one call: q, k [B][T][HK][64], v [B][T][H][64], omega, beta [B][T][H], all of the
// I/O type; value head h reads key head h / (H / HK).
struct GdrIn {
    const void* q;
    const void* k;
    const void* v;
    const void* omega;
    const void* beta;
    float scale;
    int B, T, H, HK;
};

// Token-by-token recurrence on CUDA cores, fp32 I/O.  s_out may equal s_in or be null; s_in null:
// zero.
cudaError_t launch_gdr_recurrent(const GdrIn& in, const float* s_in, float* s_out, void* y, cudaStream_t st);

// Sequences cut into `count` segments of `blocks` blocks of 64 tokens (count 1: not cut).  ctas:
// CTAs a head and segment; maps: matrices formed for each segment but one (and one less in
// all); full, part: us a CTA needs for a block with and without outputs.
struct GdrSegments {
    int count, blocks;
};
GdrSegments gdr_segments(int B, int T, int H, int ctas, int maps, float full, float part);
// at, a, s, d: [head][last][64][64] fp32, at[i] = a[i]^T.  s[i] += a[i] s[i - 1] upwards and, unless
// a and d are null, d[i] += a[i + 1]^T d[i + 1] downwards, 0 <= i < last.
cudaError_t launch_gdr_join(const float* at, const float* a, float* s, float* d, int heads, int last, cudaStream_t st);

// Chunked on tensor cores, bf16 I/O.  s_out may equal s_in or be null; s_in null: zero.  ws: at
// least gdr_chunked_bytes(B, T, H) bytes.
size_t gdr_chunked_bytes(int B, int T, int H);
cudaError_t launch_gdr_chunked(const GdrIn& in, const float* s_in, float* s_out, void* y, void* ws, cudaStream_t st);

// One token, the state updated in place (T is ignored).
cudaError_t launch_gdr_decode(const GdrIn& in, float* state, void* y, bool bf16, cudaStream_t st);

// Backward on CUDA cores, fp32 I/O, chunk by chunk.  ws: at least gdr_backward_f32_bytes(B, T, H)
// bytes.
struct GdrGrads {
    const void* dy;
    const float* ds_out;   // null: zero
    void* dq;
    void* dk;
    void* dv;
    void* domega;
    void* dbeta;
    float* ds_in;          // null: not written
};
size_t gdr_backward_f32_bytes(int B, int T, int H);
cudaError_t launch_gdr_backward_f32(const GdrIn& in, const float* s_in, const GdrGrads& g, void* ws, cudaStream_t st);

// Backward on tensor cores, bf16 I/O.  ws: at least gdr_backward_tc_bytes(B, T, H) bytes.  budget:
// cycles a wait for the tensor cores may take, after which the block's dq, dk, domega and dbeta
// are NaN.
size_t gdr_backward_tc_bytes(int B, int T, int H);
cudaError_t launch_gdr_backward_tc(const GdrIn& in, const float* s_in, const GdrGrads& g, void* ws, long long budget,
                                   cudaStream_t st);

}  // namespace goldwkv
