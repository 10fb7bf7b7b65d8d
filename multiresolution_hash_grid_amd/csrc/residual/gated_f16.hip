// Gated blocks, binary16 operands (gfx950).
#include "gated_kernels.h"

namespace hg {
namespace res {

hipError_t gated_f16(const GatedArgs &a, int h_dtype, hipStream_t stream) {
    return h_dtype == HG_F32 ? gated_run<f16, float>(a, stream) : gated_run<f16, f16>(a, stream);
}

}  // namespace res
}  // namespace hg
