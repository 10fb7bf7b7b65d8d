// Linear layer, bfloat16 operands (gfx950).
#include "linear_kernels.h"

namespace hg {
namespace res {

hipError_t linear_bf16(const FwdArgs &a, int y_dtype, hipStream_t stream) {
    return y_dtype == HG_F32 ? linear_run<bf16, float>(a, stream) : linear_run<bf16, bf16>(a, stream);
}

}  // namespace res
}  // namespace hg
