// Kernels of h = act(x Wg^T + bg) (x Wu^T + bu) for one pair of types; the sources
// that include this instantiate one operand type each, so that they build at once.
#pragma once

#include "gated_common.h"

namespace hg {
namespace res {
namespace {

// Few rows.  A workgroup computes 16 rows by 16 hidden units; its four waves share
// the contraction and add their sums in LDS.  The rows of x, Wg and Wu come straight
// from memory as fragments, so a single point costs one read of both weights.
template <typename T, typename Y>
__global__ __launch_bounds__(256) void gated_tile_kernel(const GatedArgs a) {
    __shared__ f32x4 sums[2][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, group = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * 16;
    const int n0 = blockIdx.x * 16;
    const int64_t xm = m0 + (lane & 15) < a.m ? m0 + (lane & 15) : a.m - 1;
    const int wn = n0 + (lane & 15) < a.n ? n0 + (lane & 15) : a.n - 1;
    const T *x = (const T *)a.x + xm * a.xs, *wg = (const T *)a.wg + (int64_t)wn * a.gs, *wu = (const T *)a.wu + (int64_t)wn * a.us;
    f32x4 g = {0.f, 0.f, 0.f, 0.f}, u = g;
    if (a.k < kPiece<T>) {
        if (wave == 0) {
            const u32x4 none = {0, 0, 0, 0}, v = group ? none : load_short(x, a.k);
            g = mma<T>(group ? none : load_short(wg, a.k), v, g);
            u = mma<T>(group ? none : load_short(wu, a.k), v, u);
        }
    } else {
        for (int k0 = wave * kStretch<T>; k0 < a.k; k0 += 4 * kStretch<T>) {
            const Cut<T> c = cut_piece<T>(k0 + group * kPiece<T>, a.k);
            const u32x4 v = load_loose<u32x4>(x + c.at) & c.mask;
            g = mma<T>(load_loose<u32x4>(wg + c.at) & c.mask, v, g);
            u = mma<T>(load_loose<u32x4>(wu + c.at) & c.mask, v, u);
        }
    }
    sums[0][wave][lane] = g;
    sums[1][wave][lane] = u;
    __syncthreads();
    // thread t: row t / 16, unit t % 16; it lies in lane (unit / 4) * 16 + row, word unit % 4
    const int row = threadIdx.x >> 4, col = threadIdx.x & 15;
    const int64_t m = m0 + row;
    const int n = n0 + col;
    if (m >= a.m || n >= a.n) return;
    float zg = 0.f, zu = 0.f;
    for (int i = 0; i < 4; ++i) zg += sums[0][i][(col >> 2) * 16 + row][col & 3], zu += sums[1][i][(col >> 2) * 16 + row][col & 3];
    if constexpr (sizeof(T) == 1) zg *= a.x_scale[m] * a.g_scale[n], zu *= a.x_scale[m] * a.u_scale[n];
    if (a.bg) zg += a.bg[n];
    if (a.bu) zu += a.bu[n];
    if constexpr (sizeof(T) == 2)
        if (a.gate) ((T *)a.gate)[m * a.ps + n] = (T)zg, ((T *)a.up)[m * a.qs + n] = (T)zu;
    ((Y *)a.h)[m * a.hs + n] = (Y)(activate(zg, a.act) * zu);
}

template <typename T, typename Y>
hipError_t gated_run(const GatedArgs &a, hipStream_t stream) {
    GatedArgs part = a;
    const int64_t most = 65535LL * 16;  // rows a grid's second dimension reaches
    for (int64_t m = 0; m < a.m; m += most) {
        part.m = a.m - m < most ? a.m - m : most;
        part.x = (const T *)a.x + m * a.xs;
        part.h = (Y *)a.h + m * a.hs;
        part.gate = a.gate ? (T *)a.gate + m * a.ps : nullptr;
        part.up = a.up ? (T *)a.up + m * a.qs : nullptr;
        part.x_scale = a.x_scale ? a.x_scale + m : nullptr;
        gated_tile_kernel<T, Y><<<dim3((unsigned)div_up(a.n, 16), (unsigned)div_up(part.m, 16)), 256, 0, stream>>>(part);
    }
    return hipGetLastError();
}

}  // namespace
}  // namespace res
}  // namespace hg
