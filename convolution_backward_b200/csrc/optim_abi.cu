// optim_abi.cu -- the C entry points of the optimizer's step and the gradients' norm (declared in
// include/dgrad.h).
//
// Host side only: every argument is checked before anything is launched.  Lists are read in
// place; nothing throws.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "common.cuh"
#include "dgrad.h"
#include "launchers.h"

namespace {

bool on(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool valid_dtype(dgrad_dtype_t t) { return t == DGRAD_F32 || t == DGRAD_BF16 || t == DGRAD_F16; }
int elem_kind(dgrad_dtype_t t) { return t == DGRAD_F32 ? dgrad::kF32 : t == DGRAD_BF16 ? dgrad::kBF16 : dgrad::kF16; }
unsigned elem_size(dgrad_dtype_t t) { return t == DGRAD_F32 ? 4 : 2; }

constexpr int64_t kMostElements = INT64_C(1) << 40;   // of a list: its chunks are counted in 32 bits
constexpr int64_t kMostTensors = INT64_C(1) << 24;

dgrad_status_t done(cudaError_t e)
{
    if (e == cudaSuccess) return DGRAD_OK;
    dgrad::record_cuda_error(e);
    return DGRAD_ERR_CUDA;
}

// The tensors' pointers; *master: whether they have a master copy.
dgrad_status_t check_tensors(int64_t count, const dgrad_adamw_tensor_t* t, dgrad_dtype_t param, dgrad_dtype_t grad,
                             int32_t bits, bool* master)
{
    if (count < 0 || !valid_dtype(param) || !valid_dtype(grad) || (bits != 32 && bits != 8)) return DGRAD_ERR_INVALID;
    if (grad != param && grad != DGRAD_F32) return DGRAD_ERR_UNSUPPORTED;
    if (count > kMostTensors) return DGRAD_ERR_UNSUPPORTED;
    if (count > 0 && !t) return DGRAD_ERR_INVALID;
    int64_t all = 0;
    int with = -1;
    for (int64_t i = 0; i < count; ++i) {
        const dgrad_adamw_tensor_t& s = t[i];
        if (s.n < 0) return DGRAD_ERR_INVALID;
        if (s.n == 0) continue;
        if (s.n > kMostElements || (all += s.n) > kMostElements) return DGRAD_ERR_UNSUPPORTED;
        if (!s.param || !s.m || !s.v || (bits == 8 && (!s.m_max || !s.v_max))) return DGRAD_ERR_INVALID;
        if (with >= 0 && with != (s.master != nullptr)) return DGRAD_ERR_INVALID;
        with = s.master != nullptr;
        if (!on(s.param, elem_size(param)) || !on(s.grad, elem_size(grad)) || !on(s.master, 4)) return DGRAD_ERR_ALIGNMENT;
        if (bits == 32 ? !on(s.m, 4) || !on(s.v, 4) : !on(s.m_max, 4) || !on(s.v_max, 4)) return DGRAD_ERR_ALIGNMENT;
    }
    *master = with == 1;
    return *master && param == DGRAD_F32 ? DGRAD_ERR_UNSUPPORTED : DGRAD_OK;
}

}  // namespace

extern "C" {

dgrad_status_t dgrad_adamw_step(int64_t count, const dgrad_adamw_tensor_t* tensors, dgrad_dtype_t param_type,
                                dgrad_dtype_t grad_type, const dgrad_adamw_t* opt, void* stream)
{
    if (!opt) return DGRAD_ERR_INVALID;
    bool master = false;
    dgrad_status_t s = check_tensors(count, tensors, param_type, grad_type, opt->state_bits, &master);
    if (s != DGRAD_OK) return s;
    if (!(opt->beta1 >= 0.0 && opt->beta1 < 1.0) || !(opt->beta2 >= 0.0 && opt->beta2 < 1.0) || !(opt->eps >= 0.0) ||
        !std::isfinite(static_cast<float>(opt->eps)) || !std::isfinite(static_cast<float>(opt->weight_decay)))
        return DGRAD_ERR_INVALID;
    if (!opt->lr_device && !(std::isfinite(static_cast<float>(opt->lr)) && std::isfinite(static_cast<float>(opt->lr * opt->weight_decay))))
        return DGRAD_ERR_INVALID;
    if (!opt->step_device && opt->step < 1) return DGRAD_ERR_INVALID;
    if (opt->stochastic != 0 && opt->stochastic != 1) return DGRAD_ERR_INVALID;
    if (opt->stochastic && opt->state_bits != 8) return DGRAD_ERR_INVALID;
    if (!on(opt->lr_device, 4) || !on(opt->step_device, 8) || !on(opt->grad_scale, 4)) return DGRAD_ERR_ALIGNMENT;
    if (count == 0) return DGRAD_OK;
    dgrad::AdamWArgs a{};
    a.count = count;
    a.t = tensors;
    a.pk = elem_kind(param_type);
    a.gk = elem_kind(grad_type);
    a.master = master;
    a.bits = opt->state_bits;
    a.stochastic = opt->stochastic != 0;
    a.lr = opt->lr;
    a.beta1 = opt->beta1;
    a.beta2 = opt->beta2;
    a.eps = opt->eps;
    a.weight_decay = opt->weight_decay;
    a.ln_beta1 = std::log(opt->beta1);
    a.ln_beta2 = std::log(opt->beta2);
    const double t = static_cast<double>(opt->step_device ? 1 : opt->step);
    a.bias1 = -1.0 / std::expm1(t * a.ln_beta1);
    a.bias2 = -1.0 / std::expm1(t * a.ln_beta2);
    a.lr_dev = opt->lr_device;
    a.step_dev = opt->step_device;
    a.scale = opt->grad_scale;
    a.seed = opt->seed;
    a.offset = opt->offset;
    s = static_cast<dgrad_status_t>(dgrad::device_status_word(&a.status));
    if (s != DGRAD_OK) return s;
    return done(dgrad::launch_adamw(a, static_cast<cudaStream_t>(stream)));
}

dgrad_status_t dgrad_adamw_check(int64_t count, const dgrad_adamw_tensor_t* tensors, dgrad_dtype_t param_type,
                                 dgrad_dtype_t grad_type, int32_t state_bits)
{
    bool master = false;
    const dgrad_status_t s = check_tensors(count, tensors, param_type, grad_type, state_bits, &master);
    if (s != DGRAD_OK || count == 0) return s;
    struct Range {
        uintptr_t lo, hi;
        bool written;
    };
    std::unique_ptr<Range[]> r(new (std::nothrow) Range[static_cast<size_t>(count) * 7]);
    if (!r) return DGRAD_ERR_UNSUPPORTED;
    size_t n = 0;
    auto add = [&](const void* p, int64_t bytes, bool written) {
        if (p && bytes > 0) r[n++] = {reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + static_cast<uintptr_t>(bytes), written};
    };
    for (int64_t i = 0; i < count; ++i) {
        const dgrad_adamw_tensor_t& t = tensors[i];
        const int64_t blocks = (t.n + 255) / 256;
        add(t.param, t.n * elem_size(param_type), true);
        add(t.grad, t.n * elem_size(grad_type), false);
        add(t.master, t.n * 4, true);
        add(t.m, state_bits == 32 ? t.n * 4 : t.n, true);
        add(t.v, state_bits == 32 ? t.n * 4 : t.n, true);
        if (state_bits == 8) {
            add(t.m_max, blocks * 4, true);
            add(t.v_max, blocks * 4, true);
        }
    }
    std::sort(r.get(), r.get() + n, [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t written = 0, any = 0;   // ends of the ranges so far
    for (size_t i = 0; i < n; ++i) {
        if (r[i].lo < (r[i].written ? any : written)) return DGRAD_ERR_INVALID;
        any = std::max(any, r[i].hi);
        if (r[i].written) written = std::max(written, r[i].hi);
    }
    return DGRAD_OK;
}

dgrad_status_t dgrad_adamw_moments(int64_t count, const dgrad_adamw_tensor_t* tensors, float* const* m_out,
                                   float* const* v_out, void* stream)
{
    if (count < 0) return DGRAD_ERR_INVALID;
    if (count > kMostTensors) return DGRAD_ERR_UNSUPPORTED;
    if (count == 0) return DGRAD_OK;
    if (!tensors || !m_out || !v_out) return DGRAD_ERR_INVALID;
    int64_t all = 0;
    for (int64_t i = 0; i < count; ++i) {
        const dgrad_adamw_tensor_t& s = tensors[i];
        if (s.n < 0) return DGRAD_ERR_INVALID;
        if (s.n == 0) continue;
        if (s.n > kMostElements || (all += s.n) > kMostElements) return DGRAD_ERR_UNSUPPORTED;
        if (!s.m || !s.v || !s.m_max || !s.v_max || !m_out[i] || !v_out[i]) return DGRAD_ERR_INVALID;
        if (!on(s.m_max, 4) || !on(s.v_max, 4) || !on(m_out[i], 4) || !on(v_out[i], 4)) return DGRAD_ERR_ALIGNMENT;
    }
    int* status = nullptr;
    const dgrad_status_t s = static_cast<dgrad_status_t>(dgrad::device_status_word(&status));
    if (s != DGRAD_OK) return s;
    return done(dgrad::launch_adamw_moments(tensors, m_out, v_out, count, status, static_cast<cudaStream_t>(stream)));
}

dgrad_status_t dgrad_grad_norm_workspace(int64_t count, size_t* bytes)
{
    if (!bytes || count < 0) return DGRAD_ERR_INVALID;
    if (count > kMostTensors) return DGRAD_ERR_UNSUPPORTED;
    *bytes = dgrad::grad_norm_workspace_bytes(count);
    return DGRAD_OK;
}

dgrad_status_t dgrad_grad_norm(int64_t count, const void* const* grads, const int64_t* n, dgrad_dtype_t dtype,
                               double max_norm, float* out, void* workspace, size_t workspace_bytes, void* stream)
{
    if (count < 0 || !valid_dtype(dtype) || !(max_norm >= 0.0) || !out) return DGRAD_ERR_INVALID;
    if (count > kMostTensors) return DGRAD_ERR_UNSUPPORTED;
    if (count > 0 && (!grads || !n || !workspace)) return DGRAD_ERR_INVALID;
    if (!on(out, 4) || !on(workspace, 16)) return DGRAD_ERR_ALIGNMENT;
    const size_t need = dgrad::grad_norm_workspace_bytes(count);
    if (workspace_bytes < need) return DGRAD_ERR_INVALID;
    const auto apart = [](const void* a, size_t na, const void* b, size_t nb) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
        return na == 0 || nb == 0 || x + na <= y || y + nb <= x;
    };
    if (!apart(out, 8, workspace, need)) return DGRAD_ERR_INVALID;
    int64_t all = 0;
    for (int64_t i = 0; i < count; ++i) {
        if (n[i] < 0) return DGRAD_ERR_INVALID;
        if (n[i] == 0) continue;
        if (n[i] > kMostElements || (all += n[i]) > kMostElements) return DGRAD_ERR_UNSUPPORTED;
        if (!grads[i]) return DGRAD_ERR_INVALID;
        if (!on(grads[i], elem_size(dtype))) return DGRAD_ERR_ALIGNMENT;
        const size_t bytes = static_cast<size_t>(n[i]) * elem_size(dtype);
        if (!apart(grads[i], bytes, out, 8) || !apart(grads[i], bytes, workspace, need)) return DGRAD_ERR_INVALID;
    }
    int* status = nullptr;
    const dgrad_status_t s = static_cast<dgrad_status_t>(dgrad::device_status_word(&status));
    if (s != DGRAD_OK) return s;
    const dgrad::NormArgs a{count, grads, n, elem_kind(dtype), static_cast<float>(max_norm), out,
                            static_cast<double*>(workspace), status};
    return done(dgrad::launch_grad_norm(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
