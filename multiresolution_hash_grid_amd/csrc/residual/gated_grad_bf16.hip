// Backward of gated blocks, bfloat16 operands (gfx950).
#include "gated_grad_kernels.h"

namespace hg {
namespace res {

hipError_t gated_grad_bf16(const GatedGradArgs &a, const GatedGradPlan &p, float *part, hipStream_t stream) {
    return gated_grad_run<bf16>(a, p, part, stream);
}

}  // namespace res
}  // namespace hg
