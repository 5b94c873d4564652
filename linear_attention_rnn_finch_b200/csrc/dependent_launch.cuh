// Launches of one call that follow each other: the next one's CTAs are placed as the present one's
// leave and wait on the device for its end, so that less time passes between two launches (two in
// B8 T4093 C320 of group norm 20.9 -> 18.9 us, four of the fp32 backward of the gated delta rule
// at B2 T333 H4 78 -> 72).  Placed earlier, while all of the present one's still run, they share
// SMs that they would have to themselves: 8 heads of 8192 tokens took a tenth longer.
//
// A call's first launch is an ordinary one, which starts after all that came before it in its
// stream.  A later one goes through launch_next; all of its threads call previous_ended before
// they write anything or read what the call's earlier launches wrote.  Since no CTA ends before
// that, the end of a launch is the end of all before it, and what follows the call in the stream
// waits as for any launch.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace goldwkv {

__device__ __forceinline__ void previous_ended() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The same, for pointers to what the earlier launches wrote: a load through one that is const and
// __restrict__ might be moved ahead of the wait, one through the pointer that comes back cannot.
template <typename T>
__device__ __forceinline__ T* behind(T* p) {
    asm volatile("" : "+l"(p)::"memory");
    return p;
}
template <typename... Params, typename... Args>
cudaError_t launch_next(void (*kernel)(Params...), unsigned grid, int threads, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid);
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    c.attrs = &attr;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, Params(args)...);
}

}  // namespace goldwkv
