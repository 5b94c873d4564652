// Launchers of group norm with an activation (not exported).  Contracts: include/goldwkv.h,
// group_norm_act and group_norm_act_backward.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace goldwkv {

struct GroupNorm {
    const void* x;         // [N][L][C], I/O type
    const float* gamma;    // [C]
    const float* beta;     // [C]
    const void* gate;      // layout and type of x, or null
    float eps;
    bool silu;             // the activation: SiLU, else none
    long N, L;
    int C, groups;
};

size_t group_norm_bytes(long N, long L, int C, int groups);
cudaError_t launch_group_norm(const GroupNorm& a, void* y, void* ws, bool bf16, cudaStream_t st);

size_t group_norm_backward_bytes(long N, long L, int C, int groups);
cudaError_t launch_group_norm_backward(const GroupNorm& a, const void* dy, void* dx, float* dgamma,
                                       float* dbeta, void* dgate, void* ws, bool bf16,
                                       cudaStream_t st);

}  // namespace goldwkv
