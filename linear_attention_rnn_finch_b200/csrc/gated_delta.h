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

// Token-by-token recurrence on CUDA cores.  s_out may equal s_in or be null; s_in null: zero.
cudaError_t launch_gdr_recurrent(const GdrIn& in, const float* s_in, float* s_out, void* y,
                                 bool bf16, cudaStream_t st);

// Chunked on tensor cores, bf16 I/O.  s_out may equal s_in or be null; s_in null: zero.
cudaError_t launch_gdr_chunked(const GdrIn& in, const float* s_in, float* s_out, void* y, cudaStream_t st);

// One token, the state updated in place (T is ignored).
cudaError_t launch_gdr_decode(const GdrIn& in, float* state, void* y, bool bf16, cudaStream_t st);

// Backward on CUDA cores in fp32, chunk by chunk (either I/O type).  ws: at least
// gdr_backward_simt_bytes(B, T, H) bytes.
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
size_t gdr_backward_simt_bytes(int B, int T, int H);
cudaError_t launch_gdr_backward_simt(const GdrIn& in, const float* s_in, const GdrGrads& g,
                                     void* ws, bool bf16, cudaStream_t st);

// Backward on tensor cores, bf16 I/O.  ws: at least gdr_backward_tc_bytes(B, T, H) bytes.
size_t gdr_backward_tc_bytes(int B, int T, int H);
cudaError_t launch_gdr_backward_tc(const GdrIn& in, const float* s_in, const GdrGrads& g, void* ws, cudaStream_t st);

}  // namespace goldwkv
