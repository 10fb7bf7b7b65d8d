// Backward of gated blocks, binary16 operands (gfx950).
#include "gated_grad_kernels.h"

namespace hg {
namespace res {

hipError_t gated_grad_f16(const GatedGradArgs &a, const GatedGradPlan &p, float *part, hipStream_t stream) {
    return gated_grad_run<f16>(a, p, part, stream);
}

}  // namespace res
}  // namespace hg
