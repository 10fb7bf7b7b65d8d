// y = act(x W^T + b) + r: the operands' types, each in a source of its own.
#include "linear_common.h"

namespace hg {
namespace res {

hipError_t launch_linear_forward(const hg_linear &op, hipStream_t stream) {
    const FwdArgs a{op.m, op.x_stride, op.w_stride, op.residual_stride, op.y_stride, op.pre_stride, op.k, op.n, op.act,
                    op.x, op.w, op.residual, op.x_scale, op.w_scale, op.bias, op.y, op.pre};
    if (op.x_dtype == HG_F16) return linear_f16(a, op.y_dtype, stream);
    if (op.x_dtype == HG_BF16) return linear_bf16(a, op.y_dtype, stream);
    return linear_f8(a, op.y_dtype, stream);
}

}  // namespace res
}  // namespace hg
