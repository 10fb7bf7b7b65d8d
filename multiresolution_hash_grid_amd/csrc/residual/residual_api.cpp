// Host side of the residual head's C entry points (include/hashgrid.h):
// argument checks, then the launch.  Nothing is allocated and nothing
// synchronises.
#include <cmath>

#include "residual_internal.h"

namespace {

using hg::abi_fail;
using hg::abi_ok;

constexpr int64_t kMaxRows = (int64_t)1 << 40;
constexpr int kMaxWidth = 65536;
constexpr int kMaxColumns = 1 << 20;
constexpr int64_t kMaxGradStride = (int64_t)1 << 22;  // of a backward's rows: a step's offsets are 32-bit

int size_of(int dtype) {
    switch (dtype) {
    case HG_F32: return 4;
    case HG_F16:
    case HG_BF16: return 2;
    case HG_F8: return 1;
    }
    return 0;
}

// A matrix [m][cols]: pointer there (or allowed to be NULL), aligned to its
// elements, rows that do not overlap and whose last byte has a 63-bit offset.
int check_rows(const char *name, const void *p, int64_t stride, int64_t m, int64_t cols, int dtype, bool needed) {
    if (!p) return needed ? abi_fail(HG_EINVAL, "%s is NULL", name) : HG_OK;
    if ((uintptr_t)p % size_of(dtype)) return abi_fail(HG_EINVAL, "%s is not aligned to its elements", name);
    if (m > 1 && stride < cols)
        return abi_fail(HG_EINVAL, "%s: row stride %lld < %lld columns", name, (long long)stride, (long long)cols);
    if (stride > (int64_t)1 << 20 && m > ((int64_t)1 << 60) / stride)
        return abi_fail(HG_EINVAL, "%s: rows and stride too large", name);
    return HG_OK;
}

// An output in place of an input: rows of the same stride, or they would meet others.
int check_in_place(const char *out, const void *p, int64_t stride, const char *in, const void *q, int64_t q_stride, int64_t m) {
    if (!p || p != q || m < 2 || stride == q_stride) return HG_OK;
    return abi_fail(HG_EINVAL, "%s in place of %s needs its row stride (%lld, not %lld)", out, in, (long long)q_stride, (long long)stride);
}

int check_vector(const char *name, const float *p, bool needed) {
    if (!p) return needed ? abi_fail(HG_EINVAL, "%s is NULL", name) : HG_OK;
    if ((uintptr_t)p % 4) return abi_fail(HG_EINVAL, "%s is not 4-byte aligned", name);
    return HG_OK;
}

int check_sizes(int64_t m, int32_t k, int32_t n, int32_t act) {
    if (m < 0 || m > kMaxRows) return abi_fail(HG_EINVAL, "m = %lld outside 0..2^40", (long long)m);
    if (k < 1 || k > kMaxWidth || n < 1 || n > kMaxWidth)
        return abi_fail(HG_EINVAL, "k = %d or n = %d outside 1..%d", k, n, kMaxWidth);
    if (act < HG_ACT_NONE || act > HG_ACT_GELU_TANH) return abi_fail(HG_EINVAL, "unknown activation %d", act);
    return HG_OK;
}

int launched(hipError_t e, const char *what) {
    if (e != hipSuccess) return abi_fail(HG_EHIP, "%s: %s", what, hipGetErrorString(e));
    return abi_ok();
}

int check_workspace(const void *workspace, size_t have, size_t need) {
    if (need == 0) return HG_OK;
    if (!workspace || have < need) return abi_fail(HG_EINVAL, "workspace of %zu bytes, %zu needed", workspace ? have : 0, need);
    if ((uintptr_t)workspace % 256) return abi_fail(HG_EINVAL, "workspace is not 256-byte aligned");
    return HG_OK;
}

int check_linear(const hg_linear *op) {
    if (!op) return abi_fail(HG_EINVAL, "op is NULL");
    int rc = check_sizes(op->m, op->k, op->n, op->act);
    if (rc) return rc;
    const bool eight = op->x_dtype == HG_F8;
    if (!eight && op->x_dtype != HG_F16 && op->x_dtype != HG_BF16)
        return abi_fail(HG_EUNSUPPORTED, "x_dtype %d is not HG_F16, HG_BF16 or HG_F8", op->x_dtype);
    if (op->y_dtype != HG_F32 && op->y_dtype != op->x_dtype && !(eight && (op->y_dtype == HG_F16 || op->y_dtype == HG_BF16)))
        return abi_fail(HG_EUNSUPPORTED, "y_dtype %d with x_dtype %d", op->y_dtype, op->x_dtype);
    if (eight && op->y_dtype == HG_F8) return abi_fail(HG_EUNSUPPORTED, "y_dtype HG_F8: an 8-bit output needs a scale");
    if (eight && op->pre) return abi_fail(HG_EUNSUPPORTED, "pre is kept for 16-bit operands only");
    if (!eight && (op->x_scale || op->w_scale)) return abi_fail(HG_EINVAL, "x_scale and w_scale belong to HG_F8 operands");
    if (op->m == 0) return HG_OK;
    if ((rc = check_rows("x", op->x, op->x_stride, op->m, op->k, op->x_dtype, true))) return rc;
    if ((rc = check_rows("w", op->w, op->w_stride, op->n, op->k, op->x_dtype, true))) return rc;
    if ((rc = check_rows("residual", op->residual, op->residual_stride, op->m, op->n, op->y_dtype, false))) return rc;
    if ((rc = check_rows("y", op->y, op->y_stride, op->m, op->n, op->y_dtype, true))) return rc;
    if ((rc = check_rows("pre", op->pre, op->pre_stride, op->m, op->n, op->x_dtype, false))) return rc;
    if ((rc = check_in_place("y", op->y, op->y_stride, "residual", op->residual, op->residual_stride, op->m))) return rc;
    if ((rc = check_vector("x_scale", op->x_scale, eight)) || (rc = check_vector("w_scale", op->w_scale, eight))) return rc;
    return check_vector("bias", op->bias, false);
}

int check_linear_grad(const hg_linear_grad *op) {
    if (!op) return abi_fail(HG_EINVAL, "op is NULL");
    int rc = check_sizes(op->m, op->k, op->n, op->act);
    if (rc) return rc;
    if (op->dtype != HG_F16 && op->dtype != HG_BF16)
        return abi_fail(HG_EUNSUPPORTED, "dtype %d is not HG_F16 or HG_BF16", op->dtype);
    if (op->dy_dtype != op->dtype && op->dy_dtype != HG_F32)
        return abi_fail(HG_EUNSUPPORTED, "dy_dtype %d with dtype %d", op->dy_dtype, op->dtype);
    if (op->dw_dtype != op->dtype && op->dw_dtype != HG_F32)
        return abi_fail(HG_EUNSUPPORTED, "dw_dtype %d with dtype %d", op->dw_dtype, op->dtype);
    const bool rows = op->m > 0;
    if ((rc = check_rows("dy", op->dy, op->dy_stride, op->m, op->n, op->dy_dtype, rows))) return rc;
    if ((rc = check_rows("pre", op->pre, op->pre_stride, op->m, op->n, op->dtype, rows && op->act != HG_ACT_NONE))) return rc;
    if ((rc = check_rows("x", op->x, op->x_stride, op->m, op->k, op->dtype, rows && op->dw))) return rc;
    if ((rc = check_rows("w", op->w, op->w_stride, op->n, op->k, op->dtype, rows && op->dx))) return rc;
    if ((rc = check_rows("dx", op->dx, op->dx_stride, op->m, op->k, op->dtype, false))) return rc;
    if ((rc = check_rows("dw", op->dw, op->dw_stride, op->n, op->k, op->dw_dtype, false))) return rc;
    const struct {
        const void *p;
        int64_t stride;
    } matrices[] = {{op->dy, op->dy_stride}, {op->pre, op->pre_stride}, {op->x, op->x_stride}, {op->dx, op->dx_stride}};
    for (const auto &t : matrices)
        if (t.p && op->m > 1 && t.stride > kMaxGradStride)
            return abi_fail(HG_EINVAL, "row stride %lld > 2^22", (long long)t.stride);
    return check_vector("db", op->db, false);
}

int check_norm_sizes(int64_t m, int32_t c, int dtype) {
    if (m < 0 || m > kMaxRows) return abi_fail(HG_EINVAL, "m = %lld outside 0..2^40", (long long)m);
    if (c < 1 || c > kMaxColumns) return abi_fail(HG_EINVAL, "c = %d outside 1..%d", c, kMaxColumns);
    if (dtype != HG_F32 && dtype != HG_F16 && dtype != HG_BF16)
        return abi_fail(HG_EUNSUPPORTED, "dtype %d is not HG_F32, HG_F16 or HG_BF16", dtype);
    return HG_OK;
}

int check_norm_grad(const hg_rms_norm_grad *op) {
    if (!op) return abi_fail(HG_EINVAL, "op is NULL");
    int rc = check_norm_sizes(op->m, op->c, op->dtype);
    if (rc) return rc;
    const bool rows = op->m > 0;
    if ((rc = check_rows("dy", op->dy, op->dy_stride, op->m, op->c, op->dtype, rows))) return rc;
    if ((rc = check_rows("sum", op->sum, op->sum_stride, op->m, op->c, op->dtype, rows))) return rc;
    if ((rc = check_rows("ds", op->ds, op->ds_stride, op->m, op->c, op->dtype, false))) return rc;
    if ((rc = check_rows("dx", op->dx, op->dx_stride, op->m, op->c, op->dtype, rows))) return rc;
    if (rows && op->c > hg::res::kNormHeld && (op->dx == op->dy || op->dx == op->sum || op->dx == op->ds))
        return abi_fail(HG_EINVAL, "dx in place of dy, sum or ds: c = %d > %d", op->c, hg::res::kNormHeld);
    if ((rc = check_in_place("dx", op->dx, op->dx_stride, "dy", op->dy, op->dy_stride, op->m))) return rc;
    if ((rc = check_in_place("dx", op->dx, op->dx_stride, "sum", op->sum, op->sum_stride, op->m))) return rc;
    if ((rc = check_in_place("dx", op->dx, op->dx_stride, "ds", op->ds, op->ds_stride, op->m))) return rc;
    if ((rc = check_vector("w", op->w, rows)) || (rc = check_vector("rstd", op->rstd, rows))) return rc;
    return check_vector("dw", op->dw, false);
}

}  // namespace

extern "C" {

int hashgrid_linear_forward(const hg_linear *op, void *stream) {
    const int rc = check_linear(op);
    if (rc) return rc;
    if (op->m == 0) return abi_ok();
    return launched(hg::res::launch_linear_forward(*op, (hipStream_t)stream), "linear forward");
}

int hashgrid_linear_backward_workspace_size(const hg_linear_grad *op, size_t *bytes_out) {
    const int rc = check_linear_grad(op);
    if (rc) return rc;
    if (!bytes_out) return abi_fail(HG_EINVAL, "bytes_out is NULL");
    *bytes_out = hg::res::linear_backward_bytes(*op);
    return abi_ok();
}

int hashgrid_linear_backward(const hg_linear_grad *op, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_linear_grad(op);
    if (rc) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, hg::res::linear_backward_bytes(*op)))) return rc;
    return launched(hg::res::launch_linear_backward(*op, workspace, (hipStream_t)stream), "linear backward");
}

int hashgrid_rms_norm_forward(const hg_rms_norm *op, void *stream) {
    if (!op) return abi_fail(HG_EINVAL, "op is NULL");
    int rc = check_norm_sizes(op->m, op->c, op->dtype);
    if (rc) return rc;
    const bool eight = op->y_dtype == HG_F8;
    if (!eight && op->y_dtype != op->dtype)
        return abi_fail(HG_EUNSUPPORTED, "y_dtype %d with dtype %d", op->y_dtype, op->dtype);
    if (!(op->eps >= 0.f) || !std::isfinite(op->eps)) return abi_fail(HG_EINVAL, "eps must be finite and >= 0");
    if (!eight && op->y_scale) return abi_fail(HG_EINVAL, "y_scale belongs to an HG_F8 output");
    if (op->m == 0) return abi_ok();
    if ((rc = check_rows("x", op->x, op->x_stride, op->m, op->c, op->dtype, true))) return rc;
    if ((rc = check_rows("residual", op->residual, op->residual_stride, op->m, op->c, op->dtype, false))) return rc;
    if ((rc = check_rows("y", op->y, op->y_stride, op->m, op->c, op->y_dtype, true))) return rc;
    if ((rc = check_rows("sum", op->sum, op->sum_stride, op->m, op->c, op->dtype, false))) return rc;
    if ((rc = check_vector("w", op->w, true)) || (rc = check_vector("y_scale", op->y_scale, eight))) return rc;
    if ((rc = check_vector("rstd", op->rstd, false))) return rc;
    if (eight && (op->y == op->x || op->y == op->residual)) return abi_fail(HG_EINVAL, "y in place of x or residual needs their type");
    if ((rc = check_in_place("y", op->y, op->y_stride, "x", op->x, op->x_stride, op->m))) return rc;
    if ((rc = check_in_place("y", op->y, op->y_stride, "residual", op->residual, op->residual_stride, op->m))) return rc;
    if ((rc = check_in_place("sum", op->sum, op->sum_stride, "x", op->x, op->x_stride, op->m))) return rc;
    if ((rc = check_in_place("sum", op->sum, op->sum_stride, "residual", op->residual, op->residual_stride, op->m))) return rc;
    return launched(hg::res::launch_rms_norm_forward(*op, (hipStream_t)stream), "rms_norm forward");
}

int hashgrid_rms_norm_backward_workspace_size(const hg_rms_norm_grad *op, size_t *bytes_out) {
    const int rc = check_norm_grad(op);
    if (rc) return rc;
    if (!bytes_out) return abi_fail(HG_EINVAL, "bytes_out is NULL");
    *bytes_out = hg::res::rms_norm_backward_bytes(*op);
    return abi_ok();
}

int hashgrid_rms_norm_backward(const hg_rms_norm_grad *op, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_norm_grad(op);
    if (rc) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, hg::res::rms_norm_backward_bytes(*op)))) return rc;
    return launched(hg::res::launch_rms_norm_backward(*op, workspace, (hipStream_t)stream), "rms_norm backward");
}

int hashgrid_adamw_step(const hg_adamw *opt, const hg_adamw_tensor *tensors, int32_t n, const float *grad_scale,
                        int32_t flags, void *stream) {
    if (!opt) return abi_fail(HG_EINVAL, "opt is NULL");
    const bool clock = (flags & HG_ADAM_CLOCK) != 0;
    if (!clock && opt->step < 1) return abi_fail(HG_EINVAL, "step %d < 1", opt->step);
    if (!(opt->beta1 >= 0.f && opt->beta1 < 1.f) || !(opt->beta2 >= 0.f && opt->beta2 < 1.f))
        return abi_fail(HG_EINVAL, "betas must lie in [0, 1)");
    if (!std::isfinite(opt->eps) || opt->eps < 0.f) return abi_fail(HG_EINVAL, "eps must be finite and >= 0");
    if (flags & ~(HG_ADAM_ZERO_GRAD | HG_ADAM_ZERO_SKIPPED | HG_ADAM_CLOCK))
        return abi_fail(HG_EINVAL, "unknown flags 0x%x", flags);
    if ((flags & (HG_ADAM_ZERO_GRAD | HG_ADAM_ZERO_SKIPPED)) == HG_ADAM_ZERO_SKIPPED)
        return abi_fail(HG_EINVAL, "HG_ADAM_ZERO_SKIPPED belongs to HG_ADAM_ZERO_GRAD");
    if (n < 0 || (n > 0 && !tensors)) return abi_fail(HG_EINVAL, "n = %d tensors at %p", n, (const void *)tensors);
    int rc = check_vector("grad_scale", grad_scale, false);
    if (rc) return rc;
    if (clock && n > 0 && (!opt->clocks || (uintptr_t)opt->clocks % 4))
        return abi_fail(HG_EINVAL, "clocks must be an aligned device pointer with HG_ADAM_CLOCK");
    for (int i = 0; i < n; ++i) {
        const hg_adamw_tensor &t = tensors[i];
        if (t.count < 0 || t.count > kMaxRows) return abi_fail(HG_EINVAL, "tensor %d: count %lld outside 0..2^40", i, (long long)t.count);
        if (t.state_bits != 32 && t.state_bits != 8) return abi_fail(HG_EINVAL, "tensor %d: state_bits %d is neither 32 nor 8", i, t.state_bits);
        if (t.grad_dtype != HG_F32 && t.grad_dtype != HG_F16 && t.grad_dtype != HG_BF16)
            return abi_fail(HG_EINVAL, "tensor %d: grad_dtype %d", i, t.grad_dtype);
        if (t.copy && t.copy_dtype != HG_F16 && t.copy_dtype != HG_BF16)
            return abi_fail(HG_EINVAL, "tensor %d: copy_dtype %d", i, t.copy_dtype);
        if (!std::isfinite(t.lr) || !std::isfinite(t.weight_decay) || t.weight_decay < 0.f)
            return abi_fail(HG_EINVAL, "tensor %d: lr and weight_decay must be finite, weight_decay >= 0", i);
        if (t.reserved) return abi_fail(HG_EINVAL, "tensor %d: reserved must be 0", i);
        if (t.count == 0) continue;
        if (!t.param || !t.grad || !t.m || !t.v || (t.state_bits == 8 && (!t.m_exp || !t.v_exp)))
            return abi_fail(HG_EINVAL, "tensor %d: param, grad and the moments must be device pointers", i);
        const uintptr_t state = t.state_bits == 8 ? 1 : 4;
        if ((uintptr_t)t.param % 4 || (uintptr_t)t.grad % size_of(t.grad_dtype) || (uintptr_t)t.m % state ||
            (uintptr_t)t.v % state || (t.copy && (uintptr_t)t.copy % 2))
            return abi_fail(HG_EINVAL, "tensor %d: misaligned buffer", i);
    }
    return launched(hg::res::launch_adamw(*opt, tensors, n, grad_scale, flags, (hipStream_t)stream),
                    "adamw");
}

}  // extern "C"
