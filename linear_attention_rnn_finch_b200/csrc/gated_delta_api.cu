// C entry points of the gated delta rule and of group norm with an activation: argument
// validation and dispatch.  Declarations and contracts are in include/goldwkv.h.
#include <cuda_runtime.h>
#include <math.h>

#include "api_checks.h"
#include "gated_delta.h"
#include "goldwkv.h"
#include "group_norm_act.h"

namespace {

using namespace goldwkv::api;

// A buffer of a call: an input, or an output that must overlap no other buffer.
struct Arg {
    const void* p;
    size_t bytes;
    bool required;
    bool out;
    size_t align = 16;   // omega and beta are read one value at a time: their own size will do
};

// Placement of every buffer, and no output over another buffer; `may_equal` (an output) may be
// the very buffer `equals`.
wkv_status check_args(const Arg* a, int n, const void* may_equal = nullptr, const void* equals = nullptr) {
    Buf bufs[20];
    for (int i = 0; i < n; ++i) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(a[i].p);
        if (at % a[i].align != 0) return WKV_ERR_INVALID_ARG;
        // the placement check wants 16-byte alignment: the 16 bytes that hold the first value
        bufs[i] = Buf{reinterpret_cast<const void*>(at & ~uintptr_t(15)), a[i].bytes, a[i].required};
    }
    const wkv_status s = check_bufs(bufs, n);
    if (s != WKV_OK) return s;
    for (int i = 0; i < n; ++i) {
        if (!a[i].out || a[i].p == nullptr) continue;
        for (int j = 0; j < n; ++j) {
            if (j == i || a[j].p == nullptr || (a[j].out && j < i)) continue;
            if (a[i].p == a[j].p && may_equal != nullptr && a[i].p == may_equal && a[j].p == equals) continue;
            if (overlaps(span(a[i].p, a[i].bytes), span(a[j].p, a[j].bytes))) return WKV_ERR_INVALID_ARG;
        }
    }
    return WKV_OK;
}

wkv_status check_gdr_sizes(int B, int T, int H, int HK, int D, wkv_dtype io, float scale) {
    if (B < 0 || T < 0 || H < 0 || HK < 0 || !valid_io(io) || !isfinite(scale)) return WKV_ERR_INVALID_ARG;
    if (H > 0 && (HK == 0 || H % HK != 0)) return WKV_ERR_INVALID_ARG;
    if (D != kHeadSizeApi) return WKV_ERR_UNSUPPORTED;
    // token numbers are ints and run up to three blocks of 64 past the end
    if (T > 2147483647 - 256) return WKV_ERR_UNSUPPORTED;
    // one CTA per head, or per head and chunk of 64 tokens
    if ((double)B * H * (T / 64 + 1) > 2147483647.0) return WKV_ERR_UNSUPPORTED;
    return WKV_OK;
}

// An empty sequence hands `from` (null: zeros) on to `to`.
wkv_status pass_state(float* to, const float* from, size_t bytes, cudaStream_t st) {
    if (to == nullptr || to == from || bytes == 0) return WKV_OK;
    return from_cuda(from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, st)
                          : cudaMemsetAsync(to, 0, bytes, st));
}

bool gn_sizes_ok(long N, long L, int C, int groups) {
    if (N < 0 || L < 0 || C <= 0 || groups <= 0 || C % groups != 0) return false;
    return true;
}
// Grids are one-dimensional, over (n, channel tile) pairs: at most C / 128 + groups + 1 tiles.  The
// largest tensors of a 180 GB device stay far below.
bool gn_sizes_built(long N, long L, int C, int groups) {
    const double most = 2147483647.0;
    return (double)N * groups <= most && (L == 1 || (double)N * (C / 128 + groups + 1) <= most) && C <= (1 << 20) &&
           (double)N * (double)L * C < 9e15 && L <= 2147483647L;
}

}  // namespace

extern "C" {

size_t gated_delta_prefill_workspace_bytes(int B, int T, int H, int HK, int D, wkv_dtype io) {
    if (B <= 0 || T <= 0 || H <= 0 || check_gdr_sizes(B, T, H, HK, D, io, 1.f) != WKV_OK) return 0;
    return io == WKV_BF16 ? goldwkv::gdr_chunked_bytes(B, T, H) : 0;
}

wkv_status gated_delta_prefill(const void* q, const void* k, const void* v, const void* omega,
                               const void* beta, float scale, const float* state_in,
                               float* state_out, void* y, int B, int T, int H, int HK, int D,
                               wkv_dtype io, void* workspace, size_t workspace_bytes, void* stream) {
    wkv_status s = check_gdr_sizes(B, T, H, HK, D, io, scale);
    if (s != WKV_OK) return s;
    if (B == 0 || H == 0) return WKV_OK;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t es = io_size(io), bt = (size_t)B * T;
    const size_t kb = bt * HK * D * es, vb = bt * H * D * es, gb = bt * H * es;
    const size_t sb = (size_t)B * H * D * D * sizeof(float);
    const size_t need = gated_delta_prefill_workspace_bytes(B, T, H, HK, D, io);
    const bool tokens = T > 0;
    const Arg args[] = {{q, kb, tokens, false},         {k, kb, tokens, false},
                        {v, vb, tokens, false},         {omega, gb, tokens, false, es},
                        {beta, gb, tokens, false, es},      {state_in, sb, false, false},
                        {state_out, sb, false, true},   {y, vb, tokens, true},
                        {workspace, need, false, true}};
    if ((s = check_args(args, 9, state_out, state_in)) != WKV_OK) return s;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return WKV_ERR_WORKSPACE;
    if (injected("launch")) return WKV_ERR_CUDA;
    if (!tokens) return pass_state(state_out, state_in, sb, st);
    const goldwkv::GdrIn in{q, k, v, omega, beta, scale, B, T, H, HK};
    if (io == WKV_BF16) return from_cuda(goldwkv::launch_gdr_chunked(in, state_in, state_out, y, workspace, st));
    return from_cuda(goldwkv::launch_gdr_recurrent(in, state_in, state_out, y, st));
}

wkv_status gated_delta_decode_step(const void* q, const void* k, const void* v, const void* omega,
                                   const void* beta, float scale, float* state, void* y, int B,
                                   int H, int HK, int D, wkv_dtype io, void* stream) {
    wkv_status s = check_gdr_sizes(B, 1, H, HK, D, io, scale);
    if (s != WKV_OK) return s;
    if (B == 0 || H == 0) return WKV_OK;
    const size_t es = io_size(io);
    const size_t kb = (size_t)B * HK * D * es, vb = (size_t)B * H * D * es, gb = (size_t)B * H * es;
    const Arg args[] = {{q, kb, true, false},     {k, kb, true, false},
                        {v, vb, true, false},     {omega, gb, true, false, es},
                        {beta, gb, true, false, es},  {state, (size_t)B * H * D * D * sizeof(float), true, true},
                        {y, vb, true, true}};
    if ((s = check_args(args, 7)) != WKV_OK) return s;
    if (injected("launch")) return WKV_ERR_CUDA;
    const goldwkv::GdrIn in{q, k, v, omega, beta, scale, B, 1, H, HK};
    return from_cuda(goldwkv::launch_gdr_decode(in, state, y, io == WKV_BF16,
                                                reinterpret_cast<cudaStream_t>(stream)));
}

size_t gated_delta_backward_workspace_bytes(int B, int T, int H, int HK, int D, wkv_dtype io) {
    if (B <= 0 || T <= 0 || H <= 0 || check_gdr_sizes(B, T, H, HK, D, io, 1.f) != WKV_OK) return 0;
    return io == WKV_BF16 ? goldwkv::gdr_backward_tc_bytes(B, T, H) : goldwkv::gdr_backward_f32_bytes(B, T, H);
}

wkv_status gated_delta_backward(const void* q, const void* k, const void* v, const void* omega,
                                const void* beta, float scale, const float* state_in,
                                const void* dy, const float* dstate_out, void* dq, void* dk,
                                void* dv, void* domega, void* dbeta, float* dstate_in, int B,
                                int T, int H, int HK, int D, wkv_dtype io, void* workspace,
                                size_t workspace_bytes, void* stream) {
    wkv_status s = check_gdr_sizes(B, T, H, HK, D, io, scale);
    if (s != WKV_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t es = io_size(io), bt = (size_t)B * T;
    if (B == 0 || H == 0) {   // key heads without value heads: sums of nothing
        const size_t kb = bt * HK * D * es;
        if (kb == 0) return WKV_OK;
        const Arg args[] = {{q, kb, false, false}, {k, kb, false, false}, {dq, kb, true, true}, {dk, kb, true, true}};
        if ((s = check_args(args, 4)) != WKV_OK) return s;
        if (injected("launch")) return WKV_ERR_CUDA;
        const cudaError_t e = cudaMemsetAsync(dq, 0, kb, st);
        return from_cuda(e != cudaSuccess ? e : cudaMemsetAsync(dk, 0, kb, st));
    }
    const size_t kb = bt * HK * D * es, vb = bt * H * D * es, gb = bt * H * es;
    const size_t sb = (size_t)B * H * D * D * sizeof(float);
    const size_t need = gated_delta_backward_workspace_bytes(B, T, H, HK, D, io);
    const bool tokens = T > 0;
    const Arg args[] = {{q, kb, tokens, false},          {k, kb, tokens, false},
                        {v, vb, tokens, false},          {omega, gb, tokens, false, es},
                        {beta, gb, tokens, false, es},       {state_in, sb, false, false},
                        {dy, vb, tokens, false},         {dstate_out, sb, false, false},
                        {dq, kb, tokens, true},          {dk, kb, tokens, true},
                        {dv, vb, tokens, true},          {domega, gb, tokens, true, es},
                        {dbeta, gb, tokens, true, es},       {dstate_in, sb, false, true},
                        {workspace, need, false, true}};
    if ((s = check_args(args, 15)) != WKV_OK) return s;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return WKV_ERR_WORKSPACE;
    if (injected("launch")) return WKV_ERR_CUDA;
    if (!tokens) return pass_state(dstate_in, dstate_out, sb, st);
    const goldwkv::GdrIn in{q, k, v, omega, beta, scale, B, T, H, HK};
    const goldwkv::GdrGrads g{dy, dstate_out, dq, dk, dv, domega, dbeta, dstate_in};
    const long long budget = injected("timeout0") ? 0 : kSpinBudget;
    if (io == WKV_BF16) return from_cuda(goldwkv::launch_gdr_backward_tc(in, state_in, g, workspace, budget, st));
    return from_cuda(goldwkv::launch_gdr_backward_f32(in, state_in, g, workspace, st));
}

size_t group_norm_act_workspace_bytes(long N, long L, int C, int groups, wkv_dtype io) {
    if (N <= 0 || L <= 0 || !gn_sizes_ok(N, L, C, groups) || !gn_sizes_built(N, L, C, groups) || !valid_io(io))
        return 0;
    return goldwkv::group_norm_bytes(N, L, C, groups);
}

static wkv_status check_gn(long N, long L, int C, int groups, wkv_dtype io, float eps, wkv_act act) {
    if (!gn_sizes_ok(N, L, C, groups) || !valid_io(io)) return WKV_ERR_INVALID_ARG;
    if (!(eps > 0.f) || eps > 1e30f) return WKV_ERR_INVALID_ARG;
    if (act != WKV_ACT_NONE && act != WKV_ACT_SILU) return WKV_ERR_INVALID_ARG;
    return gn_sizes_built(N, L, C, groups) ? WKV_OK : WKV_ERR_UNSUPPORTED;
}

wkv_status group_norm_act(const void* x, const float* gamma, const float* beta, float eps,
                          wkv_act act, const void* gate, void* y, long N, long L, int C,
                          int groups, wkv_dtype io, void* workspace, size_t workspace_bytes,
                          void* stream) {
    wkv_status s = check_gn(N, L, C, groups, io, eps, act);
    if (s != WKV_OK) return s;
    if (N == 0 || L == 0) return WKV_OK;
    const size_t xb = (size_t)N * L * C * io_size(io), pb = (size_t)C * sizeof(float);
    const size_t need = group_norm_act_workspace_bytes(N, L, C, groups, io);
    const Arg args[] = {{x, xb, true, false},   {gamma, pb, true, false}, {beta, pb, true, false},
                        {gate, xb, false, false}, {y, xb, true, true},    {workspace, need, false, true}};
    if ((s = check_args(args, 6)) != WKV_OK) return s;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return WKV_ERR_WORKSPACE;
    if (injected("launch")) return WKV_ERR_CUDA;
    const goldwkv::GroupNorm a{x, gamma, beta, gate, eps, act == WKV_ACT_SILU, N, L, C, groups};
    return from_cuda(goldwkv::launch_group_norm(a, y, workspace, io == WKV_BF16,
                                                reinterpret_cast<cudaStream_t>(stream)));
}

size_t group_norm_act_backward_workspace_bytes(long N, long L, int C, int groups, wkv_dtype io) {
    if (N <= 0 || L <= 0 || !gn_sizes_ok(N, L, C, groups) || !gn_sizes_built(N, L, C, groups) || !valid_io(io))
        return 0;
    return goldwkv::group_norm_backward_bytes(N, L, C, groups);
}

wkv_status group_norm_act_backward(const void* x, const float* gamma, const float* beta, float eps,
                                   wkv_act act, const void* gate, const void* dy, void* dx,
                                   float* dgamma, float* dbeta, void* dgate, long N, long L, int C,
                                   int groups, wkv_dtype io, void* workspace,
                                   size_t workspace_bytes, void* stream) {
    wkv_status s = check_gn(N, L, C, groups, io, eps, act);
    if (s != WKV_OK) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool any = N > 0 && L > 0;
    if (any && (gate == nullptr) != (dgate == nullptr)) return WKV_ERR_INVALID_ARG;
    const size_t xb = (size_t)N * L * C * io_size(io), pb = (size_t)C * sizeof(float);
    const size_t need = group_norm_act_backward_workspace_bytes(N, L, C, groups, io);
    const Arg args[] = {{x, xb, any, false},      {gamma, pb, any, false},  {beta, pb, any, false},
                        {gate, xb, false, false}, {dy, xb, any, false},     {dx, xb, any, true},
                        {dgamma, pb, true, true}, {dbeta, pb, true, true},  {dgate, xb, false, true},
                        {workspace, need, false, true}};
    if ((s = check_args(args, 10)) != WKV_OK) return s;
    if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return WKV_ERR_WORKSPACE;
    if (injected("launch")) return WKV_ERR_CUDA;
    if (!any) {
        if (cudaMemsetAsync(dgamma, 0, pb, st) != cudaSuccess || cudaMemsetAsync(dbeta, 0, pb, st) != cudaSuccess)
            return WKV_ERR_CUDA;
        return WKV_OK;
    }
    const goldwkv::GroupNorm a{x, gamma, beta, gate, eps, act == WKV_ACT_SILU, N, L, C, groups};
    return from_cuda(goldwkv::launch_group_norm_backward(a, dy, dx, dgamma, dbeta, dgate, workspace,
                                                         io == WKV_BF16, st));
}

}  // extern "C"
