// Host side of the C entry points of codes, layer norms and gated blocks
// (include/hashgrid.h): argument checks, then the launch.  Nothing is allocated
// and nothing synchronises.
#include "api_checks.h"

namespace {

using hg::abi_fail;
using hg::abi_ok;
using namespace hg::res;

constexpr int64_t kMaxSorted = (int64_t)1 << 30;  // ids of a gradient: their places are 32-bit

int check_lookup(int64_t m, int64_t most, int32_t rows, int32_t c, const void *ids, int32_t ids_bits) {
    if (m < 0 || m > most) return abi_fail(HG_EINVAL, "m = %lld outside 0..%lld", (long long)m, (long long)most);
    if (rows < 0) return abi_fail(HG_EINVAL, "rows = %d < 0", rows);
    if (c < 1 || c > kMaxColumns) return abi_fail(HG_EINVAL, "c = %d outside 1..%d", c, kMaxColumns);
    if (ids_bits != 32 && ids_bits != 64) return abi_fail(HG_EINVAL, "ids_bits %d is neither 32 nor 64", ids_bits);
    if (m == 0) return HG_OK;
    if (!ids) return abi_fail(HG_EINVAL, "ids is NULL");
    if ((uintptr_t)ids % (ids_bits / 8)) return abi_fail(HG_EINVAL, "ids is not aligned to its elements");
    return HG_OK;
}

bool is_float(int dtype) { return dtype == HG_F32 || dtype == HG_F16 || dtype == HG_BF16; }

int check_embedding(const hg_embedding *op) {
    if (!op) return abi_fail(HG_EINVAL, "op is NULL");
    int rc = check_lookup(op->m, kMaxRows, op->rows, op->c, op->ids, op->ids_bits);
    if (rc) return rc;
    if (!is_float(op->table_dtype)) return abi_fail(HG_EUNSUPPORTED, "table_dtype %d is not HG_F32, HG_F16 or HG_BF16", op->table_dtype);
    if (!is_float(op->y_dtype) || (op->y_dtype != op->table_dtype && op->table_dtype != HG_F32))
        return abi_fail(HG_EUNSUPPORTED, "y_dtype %d with table_dtype %d", op->y_dtype, op->table_dtype);
    if (op->m == 0) return HG_OK;
    if (op->rows > 0 && (rc = check_rows("table", op->table, op->table_stride, op->rows, op->c, op->table_dtype, true))) return rc;
    if (op->rows > 0 && op->y == op->table) return abi_fail(HG_EINVAL, "y is a buffer of its own");
    return check_rows("y", op->y, op->y_stride, op->m, op->c, op->y_dtype, true);
}

int check_embedding_grad(const hg_embedding_grad *op) {
    if (!op) return abi_fail(HG_EINVAL, "op is NULL");
    int rc = check_lookup(op->m, kMaxSorted, op->rows, op->c, op->ids, op->ids_bits);
    if (rc) return rc;
    if (!is_float(op->dy_dtype)) return abi_fail(HG_EUNSUPPORTED, "dy_dtype %d is not HG_F32, HG_F16 or HG_BF16", op->dy_dtype);
    if (op->dtable_dtype != op->dy_dtype && op->dtable_dtype != HG_F32)
        return abi_fail(HG_EUNSUPPORTED, "dtable_dtype %d with dy_dtype %d", op->dtable_dtype, op->dy_dtype);
    if (op->rows == 0) return HG_OK;
    if ((rc = check_rows("dtable", op->dtable, op->dtable_stride, op->rows, op->c, op->dtable_dtype, true))) return rc;
    if (op->m == 0) return HG_OK;
    if (op->dtable == op->dy) return abi_fail(HG_EINVAL, "dtable is a buffer of its own");
    return check_rows("dy", op->dy, op->dy_stride, op->m, op->c, op->dy_dtype, true);
}

int check_layer_norm(const hg_layer_norm *op) {
    if (!op) return abi_fail(HG_EINVAL, "op is NULL");
    int rc = check_norm_sizes(op->m, op->c, op->dtype);
    if (rc) return rc;
    const bool eight = op->y_dtype == HG_F8;
    if (!eight && op->y_dtype != op->dtype)
        return abi_fail(HG_EUNSUPPORTED, "y_dtype %d with dtype %d", op->y_dtype, op->dtype);
    if (!(op->eps >= 0.f) || !std::isfinite(op->eps)) return abi_fail(HG_EINVAL, "eps must be finite and >= 0");
    if (!eight && op->y_scale) return abi_fail(HG_EINVAL, "y_scale belongs to an HG_F8 output");
    if (op->m == 0) return HG_OK;
    if ((rc = check_rows("x", op->x, op->x_stride, op->m, op->c, op->dtype, true))) return rc;
    if ((rc = check_rows("residual", op->residual, op->residual_stride, op->m, op->c, op->dtype, false))) return rc;
    if ((rc = check_rows("y", op->y, op->y_stride, op->m, op->c, op->y_dtype, true))) return rc;
    if ((rc = check_rows("sum", op->sum, op->sum_stride, op->m, op->c, op->dtype, false))) return rc;
    if ((rc = check_vector("w", op->w, false)) || (rc = check_vector("b", op->b, false))) return rc;
    if ((rc = check_vector("y_scale", op->y_scale, eight)) || (rc = check_vector("mean", op->mean, false))) return rc;
    if ((rc = check_vector("rstd", op->rstd, false))) return rc;
    if (eight && (op->y == op->x || op->y == op->residual)) return abi_fail(HG_EINVAL, "y in place of x or residual needs their type");
    if (op->mean && op->mean == op->rstd) return abi_fail(HG_EINVAL, "mean and rstd are one buffer");
    if (op->sum && op->sum == op->y) return abi_fail(HG_EINVAL, "sum and y are one buffer");
    if ((rc = check_in_place("y", op->y, op->y_stride, "x", op->x, op->x_stride, op->m))) return rc;
    if ((rc = check_in_place("y", op->y, op->y_stride, "residual", op->residual, op->residual_stride, op->m))) return rc;
    if ((rc = check_in_place("sum", op->sum, op->sum_stride, "x", op->x, op->x_stride, op->m))) return rc;
    return check_in_place("sum", op->sum, op->sum_stride, "residual", op->residual, op->residual_stride, op->m);
}

int check_layer_norm_grad(const hg_layer_norm_grad *op) {
    if (!op) return abi_fail(HG_EINVAL, "op is NULL");
    int rc = check_norm_sizes(op->m, op->c, op->dtype);
    if (rc) return rc;
    const bool rows = op->m > 0;
    if ((rc = check_rows("dy", op->dy, op->dy_stride, op->m, op->c, op->dtype, rows))) return rc;
    if ((rc = check_rows("sum", op->sum, op->sum_stride, op->m, op->c, op->dtype, rows))) return rc;
    if ((rc = check_rows("ds", op->ds, op->ds_stride, op->m, op->c, op->dtype, false))) return rc;
    if ((rc = check_rows("dx", op->dx, op->dx_stride, op->m, op->c, op->dtype, rows))) return rc;
    if (rows && op->c > kNormHeld && (op->dx == op->dy || op->dx == op->sum || op->dx == op->ds))
        return abi_fail(HG_EINVAL, "dx in place of dy, sum or ds: c = %d > %d", op->c, kNormHeld);
    if ((rc = check_in_place("dx", op->dx, op->dx_stride, "dy", op->dy, op->dy_stride, op->m))) return rc;
    if ((rc = check_in_place("dx", op->dx, op->dx_stride, "sum", op->sum, op->sum_stride, op->m))) return rc;
    if ((rc = check_in_place("dx", op->dx, op->dx_stride, "ds", op->ds, op->ds_stride, op->m))) return rc;
    if ((rc = check_vector("w", op->w, false)) || (rc = check_vector("mean", op->mean, rows))) return rc;
    if ((rc = check_vector("rstd", op->rstd, rows)) || (rc = check_vector("dw", op->dw, false))) return rc;
    if (op->dw && op->dw == op->db) return abi_fail(HG_EINVAL, "dw and db are one buffer");
    return check_vector("db", op->db, false);
}

int check_gated(const hg_gated *op) {
    if (!op) return abi_fail(HG_EINVAL, "op is NULL");
    int rc = check_sizes(op->m, op->k, op->n, op->act);
    if (rc) return rc;
    const bool eight = op->x_dtype == HG_F8;
    if (!eight && op->x_dtype != HG_F16 && op->x_dtype != HG_BF16)
        return abi_fail(HG_EUNSUPPORTED, "x_dtype %d is not HG_F16, HG_BF16 or HG_F8", op->x_dtype);
    if (eight && op->h_dtype == HG_F8) return abi_fail(HG_EUNSUPPORTED, "h_dtype HG_F8: an 8-bit output needs a scale");
    if (op->h_dtype != HG_F32 && op->h_dtype != op->x_dtype && !(eight && (op->h_dtype == HG_F16 || op->h_dtype == HG_BF16)))
        return abi_fail(HG_EUNSUPPORTED, "h_dtype %d with x_dtype %d", op->h_dtype, op->x_dtype);
    if (eight && (op->gate || op->up)) return abi_fail(HG_EUNSUPPORTED, "gate and up are kept for 16-bit operands only");
    if (!op->gate != !op->up) return abi_fail(HG_EINVAL, "gate and up are kept together");
    if (!eight && (op->x_scale || op->g_scale || op->u_scale))
        return abi_fail(HG_EINVAL, "x_scale, g_scale and u_scale belong to HG_F8 operands");
    if (op->m == 0) return HG_OK;
    if ((rc = check_rows("x", op->x, op->x_stride, op->m, op->k, op->x_dtype, true))) return rc;
    if ((rc = check_rows("wg", op->wg, op->wg_stride, op->n, op->k, op->x_dtype, true))) return rc;
    if ((rc = check_rows("wu", op->wu, op->wu_stride, op->n, op->k, op->x_dtype, true))) return rc;
    if ((rc = check_rows("h", op->h, op->h_stride, op->m, op->n, op->h_dtype, true))) return rc;
    if ((rc = check_rows("gate", op->gate, op->gate_stride, op->m, op->n, op->x_dtype, false))) return rc;
    if ((rc = check_rows("up", op->up, op->up_stride, op->m, op->n, op->x_dtype, false))) return rc;
    if (op->h == op->x || op->gate == op->h || op->up == op->h || (op->gate && op->gate == op->up))
        return abi_fail(HG_EINVAL, "h, gate, up and x are buffers of their own");
    for (const void *p : {(const void *)op->h, (const void *)op->gate, (const void *)op->up})
        if (p && (p == op->wg || p == op->wu || p == op->x)) return abi_fail(HG_EINVAL, "h, gate and up are no buffers of the operands");
    if ((rc = check_vector("x_scale", op->x_scale, eight)) || (rc = check_vector("g_scale", op->g_scale, eight))) return rc;
    if ((rc = check_vector("u_scale", op->u_scale, eight)) || (rc = check_vector("bg", op->bg, false))) return rc;
    return check_vector("bu", op->bu, false);
}

int check_gated_grad(const hg_gated_grad *op) {
    if (!op) return abi_fail(HG_EINVAL, "op is NULL");
    int rc = check_sizes(op->m, op->k, op->n, op->act);
    if (rc) return rc;
    if (op->dtype != HG_F16 && op->dtype != HG_BF16)
        return abi_fail(HG_EUNSUPPORTED, "dtype %d is not HG_F16 or HG_BF16", op->dtype);
    if (op->dw_dtype != op->dtype && op->dw_dtype != HG_F32)
        return abi_fail(HG_EUNSUPPORTED, "dw_dtype %d with dtype %d", op->dw_dtype, op->dtype);
    if (!op->dwg != !op->dwu) return abi_fail(HG_EINVAL, "dwg and dwu are made together");
    if (!op->dbg != !op->dbu) return abi_fail(HG_EINVAL, "dbg and dbu are made together");
    const bool rows = op->m > 0;
    if ((rc = check_rows("dh", op->dh, op->dh_stride, op->m, op->n, op->dtype, rows))) return rc;
    if ((rc = check_rows("gate", op->gate, op->gate_stride, op->m, op->n, op->dtype, rows))) return rc;
    if ((rc = check_rows("up", op->up, op->up_stride, op->m, op->n, op->dtype, rows))) return rc;
    if ((rc = check_rows("x", op->x, op->x_stride, op->m, op->k, op->dtype, rows && op->dwg))) return rc;
    if ((rc = check_rows("wg", op->wg, op->wg_stride, op->n, op->k, op->dtype, rows && op->dx))) return rc;
    if ((rc = check_rows("wu", op->wu, op->wu_stride, op->n, op->k, op->dtype, rows && op->dx))) return rc;
    if ((rc = check_rows("dx", op->dx, op->dx_stride, op->m, op->k, op->dtype, false))) return rc;
    if ((rc = check_rows("dwg", op->dwg, op->dwg_stride, op->n, op->k, op->dw_dtype, false))) return rc;
    if ((rc = check_rows("dwu", op->dwu, op->dwu_stride, op->n, op->k, op->dw_dtype, false))) return rc;
    const struct {
        const char *name;
        const void *p;
        int64_t stride;
    } matrices[] = {{"dh", op->dh, op->dh_stride}, {"gate", op->gate, op->gate_stride}, {"up", op->up, op->up_stride},
                    {"x", op->x, op->x_stride}, {"dx", op->dx, op->dx_stride}};
    for (const auto &t : matrices)
        if (t.p && op->m > 1 && t.stride > kMaxGradStride)
            return abi_fail(HG_EINVAL, "%s: row stride %lld > 2^22", t.name, (long long)t.stride);
    for (const void *p : {(const void *)op->dh, op->gate, op->up, op->x, op->wg, op->wu})
        for (const void *out : {(const void *)op->dx, (const void *)op->dwg, (const void *)op->dwu})
            if (rows && out && out == p) return abi_fail(HG_EINVAL, "dx, dwg and dwu are buffers of their own");
    if ((op->dwg && op->dwg == op->dwu) || (op->dbg && op->dbg == op->dbu))
        return abi_fail(HG_EINVAL, "dwg and dwu, and dbg and dbu, are two buffers");
    if ((rc = check_vector("dbg", op->dbg, false))) return rc;
    return check_vector("dbu", op->dbu, false);
}

}  // namespace

extern "C" {

int hashgrid_embedding_forward(const hg_embedding *op, void *stream) {
    const int rc = check_embedding(op);
    if (rc) return rc;
    if (op->m == 0) return abi_ok();
    return launched(launch_embedding_forward(*op, (hipStream_t)stream), "embedding forward");
}

int hashgrid_embedding_backward_workspace_size(const hg_embedding_grad *op, size_t *bytes_out) {
    const int rc = check_embedding_grad(op);
    if (rc) return rc;
    if (!bytes_out) return abi_fail(HG_EINVAL, "bytes_out is NULL");
    *bytes_out = embedding_backward_bytes(*op);
    return abi_ok();
}

int hashgrid_embedding_backward(const hg_embedding_grad *op, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_embedding_grad(op);
    if (rc) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, embedding_backward_bytes(*op)))) return rc;
    return launched(launch_embedding_backward(*op, workspace, (hipStream_t)stream), "embedding backward");
}

int hashgrid_layer_norm_forward(const hg_layer_norm *op, void *stream) {
    const int rc = check_layer_norm(op);
    if (rc) return rc;
    if (op->m == 0) return abi_ok();
    return launched(launch_layer_norm_forward(*op, (hipStream_t)stream), "layer_norm forward");
}

int hashgrid_layer_norm_backward_workspace_size(const hg_layer_norm_grad *op, size_t *bytes_out) {
    const int rc = check_layer_norm_grad(op);
    if (rc) return rc;
    if (!bytes_out) return abi_fail(HG_EINVAL, "bytes_out is NULL");
    *bytes_out = layer_norm_backward_bytes(*op);
    return abi_ok();
}

int hashgrid_layer_norm_backward(const hg_layer_norm_grad *op, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_layer_norm_grad(op);
    if (rc) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, layer_norm_backward_bytes(*op)))) return rc;
    return launched(launch_layer_norm_backward(*op, workspace, (hipStream_t)stream), "layer_norm backward");
}

int hashgrid_gated_forward(const hg_gated *op, void *stream) {
    const int rc = check_gated(op);
    if (rc) return rc;
    if (op->m == 0) return abi_ok();
    return launched(launch_gated_forward(*op, (hipStream_t)stream), "gated forward");
}

int hashgrid_gated_backward_workspace_size(const hg_gated_grad *op, size_t *bytes_out) {
    const int rc = check_gated_grad(op);
    if (rc) return rc;
    if (!bytes_out) return abi_fail(HG_EINVAL, "bytes_out is NULL");
    *bytes_out = gated_backward_bytes(*op);
    return abi_ok();
}

int hashgrid_gated_backward(const hg_gated_grad *op, void *workspace, size_t workspace_bytes, void *stream) {
    int rc = check_gated_grad(op);
    if (rc) return rc;
    if ((rc = check_workspace(workspace, workspace_bytes, gated_backward_bytes(*op)))) return rc;
    return launched(launch_gated_backward(*op, workspace, (hipStream_t)stream), "gated backward");
}

}  // extern "C"
