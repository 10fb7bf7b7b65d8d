// Backward of the linear layer, bfloat16 operands (gfx950).
#include "linear_grad_kernels.h"

namespace hg {
namespace res {

hipError_t linear_grad_bf16(const GradArgs &a, bool dy_f32, const GradPlan &p, char *workspace, hipStream_t stream) {
    return dy_f32 ? grad_run<bf16, float>(a, p, workspace, stream, linear_bf16, HG_BF16)
                  : grad_run<bf16, bf16>(a, p, workspace, stream, linear_bf16, HG_BF16);
}

}  // namespace res
}  // namespace hg
