// Argument checks shared by the C entry points: spans and overlaps, pointer placement, status
// conversion and the host-side fault injection of the tests.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include "goldwkv.h"

namespace goldwkv {
namespace api {

constexpr int kHeadSizeApi = 64;  // D: the only head size the kernels are built for
constexpr size_t kStatusBytes = 256;  // device status word at the start of the workspace
// Bounded waits inside the chunked kernel: SM cycles (about a second at 1.9 GHz).
constexpr long long kSpinBudget = 2000000000LL;

struct Span {
    uintptr_t lo, hi;  // [lo, hi)
};

inline Span span(const void* p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, a + bytes};
}

inline bool overlaps(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Host-side fault injection for tests of the error paths: GOLDWKV_FAULT=launch makes the
// entry points report a failed launch without launching anything.
inline bool injected(const char* what) {
    const char* f = getenv("GOLDWKV_FAULT");
    return f != nullptr && strcmp(f, what) == 0;
}

// p must be memory the current device can address as device memory.
inline bool on_current_device(const void* p, int dev) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        (void)cudaGetLastError();
        return false;
    }
    if (a.type == cudaMemoryTypeDevice) return a.device == dev;
    if (a.type == cudaMemoryTypeManaged) return true;
    return false;
}

struct Buf {
    const void* p;
    size_t bytes;
    bool required;
};

// Common pointer checks: required non-null, 16-byte aligned, on the current device.
inline wkv_status check_bufs(const Buf* bufs, int n) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        (void)cudaGetLastError();
        return WKV_ERR_CUDA;
    }
    for (int i = 0; i < n; ++i) {
        if (bufs[i].p == nullptr) {
            if (bufs[i].required) return WKV_ERR_INVALID_ARG;
            continue;
        }
        if (!aligned16(bufs[i].p)) return WKV_ERR_INVALID_ARG;
        if (!on_current_device(bufs[i].p, dev)) return WKV_ERR_INVALID_ARG;
    }
    return WKV_OK;
}

inline wkv_status from_cuda(cudaError_t e) { return e == cudaSuccess ? WKV_OK : WKV_ERR_CUDA; }

inline size_t io_size(wkv_dtype io) { return io == WKV_BF16 ? 2 : 4; }

inline bool valid_io(wkv_dtype io) { return io == WKV_F32 || io == WKV_BF16; }

inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace api
}  // namespace goldwkv
