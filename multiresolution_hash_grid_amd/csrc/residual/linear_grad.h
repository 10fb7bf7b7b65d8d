// Arguments and plan of the linear layer's backward.
#pragma once

#include "linear_common.h"

namespace hg {
namespace res {

struct GradArgs {
    int64_t m, dys, ps, xs, ws, dxs, dws;
    int k, n, act, accumulate, dw_f32;
    const void *dy, *pre, *x, *w;
    void *dx, *dw;
    float *db;
};

// Rows of a step: enough to give eight waves a 32 x 32 block of dx each and 512
// threads a piece of dz.
constexpr int grad_rows(int nt, int kt) { return kt == 64 ? 128 : kt == 128 || nt == 64 ? 64 : 32; }

// How a backward is cut: tiles of nt outputs by kt inputs, ny x nz of them, each
// with `parts` workgroups over the rows; fused: dx comes from the same pass,
// otherwise (layers wider than a tile) from dz and W^T in the workspace.
struct GradPlan {
    int nt, kt, ny, nz, parts;
    bool fused;
    size_t dz_at, wt_at, bytes;
};

hipError_t linear_grad_f16(const GradArgs &a, bool dy_f32, const GradPlan &p, char *workspace, hipStream_t stream);
hipError_t linear_grad_bf16(const GradArgs &a, bool dy_f32, const GradPlan &p, char *workspace, hipStream_t stream);

}  // namespace res
}  // namespace hg
