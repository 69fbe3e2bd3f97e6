// branch_abi.cu -- the C entry points of the residual branch's operators (declared
// in include/dgrad.h): layer norm, the gated pointwise block and dropout, forward and backward.
//
// Host side only: every argument is checked before anything is launched, then
// the launchers enqueue their kernels on the caller's stream.
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"
#include "dgrad.h"
#include "gate_act.cuh"
#include "launchers.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool valid_dtype(dgrad_dtype_t t) { return t == DGRAD_F32 || t == DGRAD_BF16 || t == DGRAD_F16; }
int elem_kind(dgrad_dtype_t t) { return t == DGRAD_F32 ? dgrad::kF32 : t == DGRAD_BF16 ? dgrad::kBF16 : dgrad::kF16; }
int64_t elem_size(dgrad_dtype_t t) { return t == DGRAD_F32 ? 4 : 2; }

// True when the two ranges share bytes but are not the same range: an output may
// be one of the inputs that are read element for element, never a shifted one.
bool clash(const void* a, int64_t na, const void* b, int64_t nb)
{
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    if (x == y && na == nb) return false;
    return x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

// True when the two ranges share any byte.
bool shared(const void* a, int64_t na, const void* b, int64_t nb)
{
    return (a && a == b && na > 0 && nb > 0) || clash(a, na, b, nb);
}

dgrad_status_t done(cudaError_t e)
{
    if (e == cudaSuccess) return DGRAD_OK;
    dgrad::record_cuda_error(e);
    return DGRAD_ERR_CUDA;
}

constexpr int64_t kMaxRows = 0x7FFFFFFFLL;
constexpr int64_t kMaxGatedRows = INT64_C(1) << 30;   // rows rounded up to a tile stay within 32 bits
constexpr int64_t kMaxChannels = 65536;

dgrad_status_t ln_shape(int64_t M, int64_t C, dgrad_dtype_t dtype)
{
    if (!valid_dtype(dtype) || M < 0 || C < 1) return DGRAD_ERR_INVALID;
    if (M > kMaxRows || C > kMaxChannels) return DGRAD_ERR_UNSUPPORTED;
    return DGRAD_OK;
}

dgrad_status_t gated_shape(int64_t M, int64_t C, int64_t F)
{
    if (M < 0 || C < 1 || F < 1) return DGRAD_ERR_INVALID;
    if (M > kMaxGatedRows || C > kMaxChannels || F > kMaxChannels / 2) return DGRAD_ERR_UNSUPPORTED;
    if (C % 8 || F % 8) return DGRAD_ERR_ALIGNMENT;
    return DGRAD_OK;
}

static_assert(int(DGRAD_ACT_SILU) == dgrad::kSilu && int(DGRAD_ACT_GELU) == dgrad::kGelu &&
                  int(DGRAD_ACT_GELU_TANH) == dgrad::kGeluTanh && int(DGRAD_ACT_RELU) == dgrad::kRelu &&
                  int(DGRAD_ACT_SIGMOID) == dgrad::kSigmoid,
              "the kernels' activation codes are the ABI's");

dgrad_status_t gated_types(dgrad_dtype_t dtype, dgrad_act_t act)
{
    if (!valid_dtype(dtype) || act < DGRAD_ACT_SILU || act > DGRAD_ACT_SIGMOID) return DGRAD_ERR_INVALID;
    return dtype == DGRAD_F32 ? DGRAD_ERR_UNSUPPORTED : DGRAD_OK;
}

dgrad_status_t dropout_call(int64_t n, dgrad_dtype_t dtype, double p, uint64_t seed, uint64_t offset, const void* X,
                            const void* residual, void* Y, void* stream)
{
    if (!valid_dtype(dtype) || n < 0 || !(p >= 0.0 && p <= 1.0)) return DGRAD_ERR_INVALID;
    if (n > (INT64_C(1) << 48)) return DGRAD_ERR_UNSUPPORTED;
    if (n == 0) return DGRAD_OK;
    if (!X || !Y) return DGRAD_ERR_INVALID;
    if (!aligned16(X) || !aligned16(residual) || !aligned16(Y)) return DGRAD_ERR_ALIGNMENT;
    const int64_t bytes = n * elem_size(dtype);
    if (clash(X, bytes, Y, bytes) || clash(residual, bytes, Y, bytes)) return DGRAD_ERR_INVALID;
    int* status = nullptr;
    const int s = dgrad::device_status_word(&status);
    if (s != DGRAD_OK) return static_cast<dgrad_status_t>(s);
    const dgrad::DropArgs a{n, elem_kind(dtype), X, residual, Y, seed, offset,
                            static_cast<uint32_t>(std::llrint(p * 65536.0)), status};
    return done(dgrad::launch_dropout(a, static_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

dgrad_status_t dgrad_layernorm_forward(int64_t M, int64_t C, dgrad_dtype_t dtype, double eps, const void* X,
                                       const void* gamma, const void* beta, void* Y, float* mean, float* rstd,
                                       void* stream)
{
    dgrad_status_t s = ln_shape(M, C, dtype);
    if (s != DGRAD_OK) return s;
    if (!(eps >= 0.0) || !std::isfinite(static_cast<float>(eps))) return DGRAD_ERR_INVALID;
    if (M == 0) return DGRAD_OK;
    if (!X || !Y) return DGRAD_ERR_INVALID;
    if (!aligned16(X) || !aligned16(Y) || !aligned16(gamma) || !aligned16(beta) || !aligned4(mean) || !aligned4(rstd))
        return DGRAD_ERR_ALIGNMENT;
    const int64_t es = elem_size(dtype), n = M * C * es;
    if (clash(X, n, Y, n) || shared(gamma, C * es, Y, n) || shared(beta, C * es, Y, n)) return DGRAD_ERR_INVALID;
    for (float* stat : {mean, rstd})
        if (shared(stat, M * 4, X, n) || shared(stat, M * 4, Y, n) || shared(stat, M * 4, gamma, C * es) ||
            shared(stat, M * 4, beta, C * es))
            return DGRAD_ERR_INVALID;
    if (shared(mean, M * 4, rstd, M * 4)) return DGRAD_ERR_INVALID;
    int* status = nullptr;
    s = static_cast<dgrad_status_t>(dgrad::device_status_word(&status));
    if (s != DGRAD_OK) return s;
    const dgrad::LnFwdArgs a{M, C, elem_kind(dtype), static_cast<float>(eps), X, gamma, beta, Y, mean, rstd, status};
    return done(dgrad::launch_layernorm_forward(a, static_cast<cudaStream_t>(stream)));
}

dgrad_status_t dgrad_layernorm_backward_workspace(int64_t M, int64_t C, dgrad_dtype_t dtype, size_t* bytes)
{
    if (!bytes) return DGRAD_ERR_INVALID;
    const dgrad_status_t s = ln_shape(M, C, dtype);
    if (s != DGRAD_OK) return s;
    *bytes = M == 0 ? 0 : dgrad::layernorm_backward_workspace_bytes(M, C, elem_kind(dtype));
    return DGRAD_OK;
}

dgrad_status_t dgrad_layernorm_backward(int64_t M, int64_t C, dgrad_dtype_t dtype, const void* dY, const void* X,
                                        const void* gamma, const float* mean, const float* rstd, void* dX,
                                        void* dgamma, void* dbeta, void* workspace, size_t workspace_bytes,
                                        void* stream)
{
    dgrad_status_t s = ln_shape(M, C, dtype);
    if (s != DGRAD_OK) return s;
    const int64_t es = elem_size(dtype), n = M * C * es;
    if (!aligned16(dY) || !aligned16(X) || !aligned16(gamma) || !aligned4(mean) || !aligned4(rstd) || !aligned16(dX) ||
        !aligned16(dgamma) || !aligned16(dbeta) || !aligned16(workspace))
        return DGRAD_ERR_ALIGNMENT;
    if (shared(dgamma, C * es, dbeta, C * es)) return DGRAD_ERR_INVALID;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (M == 0) {   // sums over no rows
        for (void* g : {dgamma, dbeta})
            if (g) {
                s = done(cudaMemsetAsync(g, 0, static_cast<size_t>(C * es), cs));
                if (s != DGRAD_OK) return s;
            }
        return DGRAD_OK;
    }
    if (!dY || !X || !mean || !rstd || !dX) return DGRAD_ERR_INVALID;
    const bool params = dgamma || dbeta;
    const size_t need = params ? dgrad::layernorm_backward_workspace_bytes(M, C, elem_kind(dtype)) : 0;
    if (params && (!workspace || workspace_bytes < need)) return DGRAD_ERR_INVALID;
    const int64_t ws = static_cast<int64_t>(need);
    if (clash(dX, n, dY, n) || clash(dX, n, X, n) || shared(dX, n, gamma, C * es) || shared(dX, n, mean, M * 4) ||
        shared(dX, n, rstd, M * 4))
        return DGRAD_ERR_INVALID;
    for (void* g : {dgamma, dbeta})
        if (shared(g, C * es, dX, n) || shared(g, C * es, dY, n) || shared(g, C * es, X, n) ||
            shared(g, C * es, gamma, C * es) || shared(g, C * es, mean, M * 4) || shared(g, C * es, rstd, M * 4) ||
            shared(g, C * es, workspace, ws))
            return DGRAD_ERR_INVALID;
    if (shared(workspace, ws, dX, n) || shared(workspace, ws, dY, n) || shared(workspace, ws, X, n) ||
        shared(workspace, ws, gamma, C * es) || shared(workspace, ws, mean, M * 4) || shared(workspace, ws, rstd, M * 4))
        return DGRAD_ERR_INVALID;
    int* status = nullptr;
    s = static_cast<dgrad_status_t>(dgrad::device_status_word(&status));
    if (s != DGRAD_OK) return s;
    const dgrad::LnBwdArgs a{M, C, elem_kind(dtype), dY, X, gamma, mean, rstd, dX, dgamma, dbeta,
                             static_cast<float*>(workspace), status};
    return done(dgrad::launch_layernorm_backward(a, cs));
}

dgrad_status_t dgrad_gated_forward(int64_t M, int64_t C, int64_t F, dgrad_dtype_t dtype, dgrad_act_t act,
                                   const void* X, const void* W, void* H, void* Z, void* stream)
{
    dgrad_status_t s = gated_types(dtype, act);
    if (s == DGRAD_OK) s = gated_shape(M, C, F);
    if (s != DGRAD_OK) return s;
    if (M == 0) return DGRAD_OK;
    if (!X || !W || !H) return DGRAD_ERR_INVALID;
    if (!aligned16(X) || !aligned16(W) || !aligned16(H) || !aligned16(Z)) return DGRAD_ERR_ALIGNMENT;
    const int64_t nx = M * C * 2, nw = 4 * F * C, nh = M * F * 2;
    if (shared(H, nh, X, nx) || shared(H, nh, W, nw) || shared(Z, 2 * nh, X, nx) || shared(Z, 2 * nh, W, nw) ||
        shared(Z, 2 * nh, H, nh))
        return DGRAD_ERR_INVALID;
    int* status = nullptr;
    s = static_cast<dgrad_status_t>(dgrad::device_status_word(&status));
    if (s != DGRAD_OK) return s;
    const dgrad::GatedArgs a{M, C, F, dtype == DGRAD_F16, static_cast<int>(act), X, W, H, Z, status};
    return done(dgrad::launch_gated_forward(a, static_cast<cudaStream_t>(stream)));
}

dgrad_status_t dgrad_gated_backward_workspace(int64_t M, int64_t C, int64_t F, size_t* bytes)
{
    if (!bytes) return DGRAD_ERR_INVALID;
    const dgrad_status_t s = gated_shape(M, C, F);
    if (s != DGRAD_OK) return s;
    *bytes = M == 0 ? 0 : dgrad::gated_backward_workspace_bytes(M, C, F);
    return DGRAD_OK;
}

dgrad_status_t dgrad_gated_backward(int64_t M, int64_t C, int64_t F, dgrad_dtype_t dtype, dgrad_act_t act,
                                    const void* dH, const void* X, const void* Z, const void* W, void* dX, void* dW,
                                    void* workspace, size_t workspace_bytes, void* stream)
{
    dgrad_status_t s = gated_types(dtype, act);
    if (s == DGRAD_OK) s = gated_shape(M, C, F);
    if (s != DGRAD_OK) return s;
    if (!dX && !dW) return DGRAD_ERR_INVALID;
    if (!aligned16(dH) || !aligned16(X) || !aligned16(Z) || !aligned16(W) || !aligned16(dX) || !aligned16(dW) ||
        !aligned16(workspace))
        return DGRAD_ERR_ALIGNMENT;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const int64_t nx = M * C * 2, nw = 4 * F * C, nh = M * F * 2;
    if (M == 0)   // a sum over no rows
        return dW ? done(cudaMemsetAsync(dW, 0, static_cast<size_t>(nw), cs)) : DGRAD_OK;
    if (!dH || !Z || (dW && !X) || (dX && !W) || !workspace) return DGRAD_ERR_INVALID;
    const size_t need = dgrad::gated_backward_workspace_bytes(M, C, F);
    if (workspace_bytes < need) return DGRAD_ERR_INVALID;
    const int64_t ws = static_cast<int64_t>(need);
    struct Range {
        const void* p;
        int64_t n;
    };
    const Range out[3] = {{dX, nx}, {dW, nw}, {workspace, ws}};
    const Range in[4] = {{dH, nh}, {X, dW ? nx : 0}, {Z, 2 * nh}, {W, dX ? nw : 0}};
    for (int i = 0; i < 3; ++i) {
        for (const Range& r : in)
            if (shared(out[i].p, out[i].n, r.p, r.n)) return DGRAD_ERR_INVALID;
        for (int j = 0; j < i; ++j)
            if (shared(out[i].p, out[i].n, out[j].p, out[j].n)) return DGRAD_ERR_INVALID;
    }
    int* status = nullptr;
    s = static_cast<dgrad_status_t>(dgrad::device_status_word(&status));
    if (s != DGRAD_OK) return s;
    const dgrad::GatedBwdArgs a{M, C, F, dtype == DGRAD_F16, static_cast<int>(act), dH, X, Z, W, dX, dW, workspace,
                                status};
    return done(dgrad::launch_gated_backward(a, cs));
}

dgrad_status_t dgrad_dropout_forward(int64_t n, dgrad_dtype_t dtype, double p, uint64_t seed, uint64_t offset,
                                     const void* X, const void* residual, void* Y, void* stream)
{
    return dropout_call(n, dtype, p, seed, offset, X, residual, Y, stream);
}

dgrad_status_t dgrad_dropout_backward(int64_t n, dgrad_dtype_t dtype, double p, uint64_t seed, uint64_t offset,
                                      const void* dY, void* dX, void* stream)
{
    return dropout_call(n, dtype, p, seed, offset, dY, nullptr, dX, stream);
}

}  // extern "C"
