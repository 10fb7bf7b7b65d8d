// Gated blocks, 8-bit operands with scales (gfx950).
#include "gated_kernels.h"

namespace hg {
namespace res {

hipError_t gated_f8(const GatedArgs &a, int h_dtype, hipStream_t stream) {
    if (h_dtype == HG_F16) return gated_run<f8, f16>(a, stream);
    return h_dtype == HG_BF16 ? gated_run<f8, bf16>(a, stream) : gated_run<f8, float>(a, stream);
}

}  // namespace res
}  // namespace hg
