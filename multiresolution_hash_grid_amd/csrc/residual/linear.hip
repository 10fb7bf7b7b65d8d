// y = act(x W^T + b) + r on the matrix cores (gfx950).
#include "linear_common.h"

namespace hg {
namespace res {
namespace {

// A workgroup computes 16 rows by 16 outputs; its four waves share the
// contraction and add their sums in LDS.  Both operands come straight from
// memory as fragments.
template <typename T, typename Y>
__global__ __launch_bounds__(256) void linear_tile_kernel(const FwdArgs a) {
    __shared__ f32x4 sums[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m0 = (int64_t)blockIdx.y * 16;
    const int n0 = blockIdx.x * 16;
    const int64_t xm = m0 + (lane & 15) < a.m ? m0 + (lane & 15) : a.m - 1;
    const int wn = n0 + (lane & 15) < a.n ? n0 + (lane & 15) : a.n - 1;
    const T *x = (const T *)a.x + xm * a.xs, *w = (const T *)a.w + (int64_t)wn * a.ws;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int k = wave * kStretch<T> + (lane >> 4) * kPiece<T>; k - (lane >> 4) * kPiece<T> < a.k; k += 4 * kStretch<T>)
        acc = mma<T>(load_piece(w + k, a.k - k), load_piece(x + k, a.k - k), acc);
    sums[wave][lane] = acc;
    __syncthreads();
    // thread t: row t / 16, output t % 16; it lies in lane (output / 4) * 16 + row, word output % 4
    const int row = threadIdx.x >> 4, col = threadIdx.x & 15;
    const int64_t m = m0 + row;
    const int n = n0 + col;
    if (m >= a.m || n >= a.n) return;
    float z = 0.f;
    for (int i = 0; i < 4; ++i) z += sums[i][(col >> 2) * 16 + row][col & 3];
    if constexpr (sizeof(T) == 1) z = z * a.x_scale[m] * a.w_scale[n];
    if (a.bias) z += a.bias[n];
    if constexpr (sizeof(T) == 2)
        if (a.pre) ((T *)a.pre)[m * a.ps + n] = (T)z;
    float y = activate(z, a.act);
    if (a.r) y += (float)((const Y *)a.r)[m * a.rs + n];
    ((Y *)a.y)[m * a.ys + n] = (Y)y;
}

template <typename T, typename Y>
void run(const FwdArgs &a, hipStream_t stream) {
    FwdArgs part = a;
    const int64_t most = 65535LL * 16;  // rows a grid's second dimension reaches
    for (int64_t m = 0; m < a.m; m += most) {
        part.m = a.m - m < most ? a.m - m : most;
        part.x = (const T *)a.x + m * a.xs;
        part.r = a.r ? (const Y *)a.r + m * a.rs : nullptr;
        part.y = (Y *)a.y + m * a.ys;
        part.pre = a.pre ? (T *)a.pre + m * a.ps : nullptr;
        part.x_scale = a.x_scale ? a.x_scale + m : nullptr;
        linear_tile_kernel<T, Y><<<dim3((unsigned)div_up(a.n, 16), (unsigned)div_up(part.m, 16)), 256, 0, stream>>>(part);
    }
}

}  // namespace

hipError_t launch_linear_forward(const hg_linear &op, hipStream_t stream) {
    const FwdArgs a{op.m, op.x_stride, op.w_stride, op.residual_stride, op.y_stride, op.pre_stride, op.k, op.n, op.act,
                    op.x, op.w, op.residual, op.x_scale, op.w_scale, op.bias, op.y, op.pre};
    const int x = op.x_dtype, y = op.y_dtype;
    if (x == HG_F16) y == HG_F32 ? run<f16, float>(a, stream) : run<f16, f16>(a, stream);
    else if (x == HG_BF16) y == HG_F32 ? run<bf16, float>(a, stream) : run<bf16, bf16>(a, stream);
    else if (y == HG_F32) run<f8, float>(a, stream);
    else if (y == HG_F16) run<f8, f16>(a, stream);
    else run<f8, bf16>(a, stream);
    return hipGetLastError();
}

}  // namespace res
}  // namespace hg
