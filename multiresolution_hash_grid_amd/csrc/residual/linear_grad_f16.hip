// Backward of the linear layer, binary16 operands (gfx950).
#include "linear_grad_kernels.h"

namespace hg {
namespace res {

hipError_t linear_grad_f16(const GradArgs &a, bool dy_f32, const GradPlan &p, char *workspace, hipStream_t stream) {
    return dy_f32 ? grad_run<f16, float>(a, p, workspace, stream, linear_f16, HG_F16)
                  : grad_run<f16, f16>(a, p, workspace, stream, linear_f16, HG_F16);
}

}  // namespace res
}  // namespace hg
