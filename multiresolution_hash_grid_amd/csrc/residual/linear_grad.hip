// Backward of y = act(x W^T + b) + r on the matrix cores (gfx950).
//
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum over rows of dz
//
// dz is rounded to the operands' type where it enters a product, as the
// products of 16-bit operands need; db sums it unrounded.
#include "linear_common.h"

namespace hg {
namespace res {
namespace {

struct GradArgs {
    int64_t m, dys, ps, xs, ws, dxs, dws;
    int k, n, act, accumulate;
    const void *dy, *pre, *x, *w;
    void *dx, *dw;
    float *db;
};

template <typename T, typename D>
__device__ __forceinline__ float dz_at(const GradArgs &a, int64_t m, int n) {
    float d = (float)((const D *)a.dy)[m * a.dys + n];
    if (a.act != HG_ACT_NONE) {
        const float s = slope((float)((const T *)a.pre)[m * a.ps + n], a.act);
        d = s == 0.f ? 0.f : d * s;
    }
    return d;
}

template <typename T>
__device__ __forceinline__ void put(u32x4 &v, int j, float f) {
    v[j / 2] |= (uint32_t)__builtin_bit_cast(uint16_t, (T)f) << (16 * (j & 1));
}

// dx: 16 rows by 16 columns a wave, the contraction over the outputs.
template <typename T, typename D>
__global__ __launch_bounds__(64) void dx_tile_kernel(const GradArgs a) {
    const int lane = threadIdx.x, part = (lane >> 4) * 8;
    const int64_t m = (int64_t)blockIdx.y * 16 + (lane & 15), mc = m < a.m ? m : a.m - 1;
    const int k0 = blockIdx.x * 16, kc = k0 + (lane & 15) < a.k ? k0 + (lane & 15) : a.k - 1;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int n = 0; n < a.n; n += 32) {
        u32x4 wt = {0, 0, 0, 0}, dz = {0, 0, 0, 0};
        for (int j = 0; j < 8; ++j) {
            const int i = n + part + j;
            if (i < a.n) {
                put<T>(wt, j, (float)((const T *)a.w)[(int64_t)i * a.ws + kc]);
                put<T>(dz, j, dz_at<T, D>(a, mc, i));
            }
        }
        acc = mma<T>(wt, dz, acc);
    }
    if (m >= a.m) return;
    for (int r = 0; r < 4; ++r) {
        const int k = k0 + (lane >> 4) * 4 + r;
        if (k < a.k) ((T *)a.dx)[m * a.dxs + k] = (T)acc[r];
    }
}

// dW: 16 outputs by 16 columns a wave, the contraction over the rows.
template <typename T, typename D, typename G>
__global__ __launch_bounds__(64) void dw_tile_kernel(const GradArgs a) {
    const int lane = threadIdx.x, part = (lane >> 4) * 8;
    const int k0 = blockIdx.x * 16, n0 = blockIdx.y * 16;
    const int kc = k0 + (lane & 15) < a.k ? k0 + (lane & 15) : a.k - 1, n = n0 + (lane & 15), nc = n < a.n ? n : a.n - 1;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int64_t m = 0; m < a.m; m += 32) {
        u32x4 xt = {0, 0, 0, 0}, dz = {0, 0, 0, 0};
        for (int j = 0; j < 8; ++j) {
            const int64_t i = m + part + j;
            if (i < a.m) {
                put<T>(xt, j, (float)((const T *)a.x)[i * a.xs + kc]);
                put<T>(dz, j, dz_at<T, D>(a, i, nc));
            }
        }
        acc = mma<T>(xt, dz, acc);
    }
    if (n >= a.n) return;
    for (int r = 0; r < 4; ++r) {
        const int k = k0 + (lane >> 4) * 4 + r;
        if (k < a.k) {
            G *p = (G *)a.dw + (int64_t)n * a.dws + k;
            *p = (G)(acc[r] + (a.accumulate ? (float)*p : 0.f));
        }
    }
}

// db: a workgroup an output, its threads' sums added in a fixed order.
template <typename T, typename D>
__global__ __launch_bounds__(256) void db_kernel(const GradArgs a) {
    __shared__ float lds[4];
    const int n = blockIdx.x;
    float t = 0.f;
    for (int64_t m = threadIdx.x; m < a.m; m += 256) t += dz_at<T, D>(a, m, n);
    t = group_sum<64>(t);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = t;
    __syncthreads();
    if (threadIdx.x == 0) {
        t = lds[0] + lds[1] + lds[2] + lds[3];
        a.db[n] = a.accumulate ? a.db[n] + t : t;
    }
}

template <typename T, typename D>
hipError_t run(const GradArgs &a, bool dw_f32, hipStream_t stream) {
    if (a.dx && a.m > 0) {
        GradArgs part = a;
        const int64_t most = 65535LL * 16;
        for (int64_t m = 0; m < a.m; m += most) {
            part.m = a.m - m < most ? a.m - m : most;
            part.dy = (const D *)a.dy + m * a.dys;
            part.pre = a.pre ? (const T *)a.pre + m * a.ps : nullptr;
            part.dx = (T *)a.dx + m * a.dxs;
            dx_tile_kernel<T, D><<<dim3((unsigned)div_up(a.k, 16), (unsigned)div_up(part.m, 16)), 64, 0, stream>>>(part);
        }
    }
    const dim3 tiles((unsigned)div_up(a.k, 16), (unsigned)div_up(a.n, 16));
    if (a.dw && dw_f32) dw_tile_kernel<T, D, float><<<tiles, 64, 0, stream>>>(a);
    else if (a.dw) dw_tile_kernel<T, D, T><<<tiles, 64, 0, stream>>>(a);
    if (a.db) db_kernel<T, D><<<dim3((unsigned)a.n), 256, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

size_t linear_backward_bytes(const hg_linear_grad &) { return 0; }

hipError_t launch_linear_backward(const hg_linear_grad &op, void *, hipStream_t stream) {
    const GradArgs a{op.m, op.dy_stride, op.pre_stride, op.x_stride, op.w_stride, op.dx_stride, op.dw_stride,
                     op.k, op.n, op.act, op.accumulate, op.dy, op.pre, op.x, op.w, op.dx, op.dw, op.db};
    const bool wide = op.dy_dtype == HG_F32, g32 = op.dw_dtype == HG_F32;
    if (op.dtype == HG_F16) return wide ? run<f16, float>(a, g32, stream) : run<f16, f16>(a, g32, stream);
    return wide ? run<bf16, float>(a, g32, stream) : run<bf16, bf16>(a, g32, stream);
}

}  // namespace res
}  // namespace hg
