// Gated blocks, bfloat16 operands (gfx950).
#include "gated_kernels.h"

namespace hg {
namespace res {

hipError_t gated_bf16(const GatedArgs &a, int h_dtype, hipStream_t stream) {
    return h_dtype == HG_F32 ? gated_run<bf16, float>(a, stream) : gated_run<bf16, bf16>(a, stream);
}

}  // namespace res
}  // namespace hg
