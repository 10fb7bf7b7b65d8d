// How a gated block's backward is cut.
#pragma once

#include "gated_common.h"

namespace hg {
namespace res {

// The weights' gradients: tiles of `units` hidden units (gate and up) by kt inputs,
// ny x nz of them, each with `parts` workgroups over the rows.  dx: tiles of 256 rows
// by kp * 32 inputs, the units in `slices` of `per` stretches of 32 (their sums from
// dx_at on in the workspace, where there are several).
struct GatedGradPlan {
    int units, kt, ny, nz, parts, kp, slices, per;
    bool together;  // dx is made with the weights' gradients
    size_t dx_at, bytes;
};
// Rows of a step: the widest tile's sums leave registers for the pieces of 32.
constexpr int gate_rows(int units, int kt) { return units == 128 && kt == 256 ? 32 : 64; }

hipError_t gated_grad_f16(const GatedGradArgs &a, const GatedGradPlan &p, float *part, hipStream_t stream);
hipError_t gated_grad_bf16(const GatedGradArgs &a, const GatedGradPlan &p, float *part, hipStream_t stream);

}  // namespace res
}  // namespace hg
