// Linear layer, 8-bit operands with scales (gfx950).
#include "linear_kernels.h"

namespace hg {
namespace res {

hipError_t linear_f8(const FwdArgs &a, int y_dtype, hipStream_t stream) {
    if (y_dtype == HG_F32) return linear_run<f8, float>(a, stream);
    return y_dtype == HG_F16 ? linear_run<f8, f16>(a, stream) : linear_run<f8, bf16>(a, stream);
}

}  // namespace res
}  // namespace hg
