// Launch descriptions of the residual head's operators (linear, RMS norm,
// AdamW), shared by their host side and their kernels.  Not part of the
// public ABI (include/hashgrid.h is).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hashgrid.h"

namespace hg {

// Error text and return code of the C entry points (defined with the
// encoder's entry points, so that hashgrid_last_error covers both).
int abi_fail(int code, const char *fmt, ...);
int abi_ok();

namespace res {

constexpr int kNormHeld = 4096;  // columns of a norm's row that a workgroup holds in registers (256 threads x 2 vectors of 8)
constexpr int kCus = 256;  // MI355X: 8 XCDs of 32 CUs

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A grid of `groups` workgroups in two dimensions.  One dimension holds less than
// 2^32 threads: a launch of more runs the remainder only, without an error.  The
// kernel's index is blockIdx.y * gridDim.x + blockIdx.x, and some past the end exist.
constexpr int64_t kGridX = (int64_t)1 << 21;  // times 1024 threads at most
inline dim3 grid_of(int64_t groups) {
    if (groups <= kGridX) return dim3((unsigned)groups);
    return dim3((unsigned)kGridX, (unsigned)div_up(groups, kGridX));
}

hipError_t launch_linear_forward(const hg_linear &op, hipStream_t stream);
size_t linear_backward_bytes(const hg_linear_grad &op);
hipError_t launch_linear_backward(const hg_linear_grad &op, void *workspace, hipStream_t stream);

hipError_t launch_rms_norm_forward(const hg_rms_norm &op, hipStream_t stream);
size_t rms_norm_backward_bytes(const hg_rms_norm_grad &op);
hipError_t launch_rms_norm_backward(const hg_rms_norm_grad &op, void *workspace, hipStream_t stream);

// Tensors per launch: their descriptions travel in the kernel's arguments.
constexpr int kAdamwTensors = 36;
hipError_t launch_adamw(const hg_adamw &opt, const hg_adamw_tensor *tensors, int32_t n, const float *grad_scale,
                        int32_t flags, hipStream_t stream);

}  // namespace res
}  // namespace hg
