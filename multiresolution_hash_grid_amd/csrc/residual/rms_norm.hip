// Root-mean-square norm with the residual's addition, and its backward (gfx950).
//
//   s = x + r,  q = 1 / sqrt(mean(s^2) + eps),  y = s q w
//   dx = q (w dy - h mean(w dy h)) + ds,  dw = sum over rows of dy h,  h = s q
//
// One pass over the data: a row lies in the registers of a group of lanes
// between its sum of squares and its output.  Everything is fp32 between the
// loads and the one rounding of each output; y is made from the unrounded s.
// The 8-bit output is e4m3 with one scale a row, max |y| / 448: y is in
// registers when the maximum is known, so the 8 bits cost no second pass.
#include "device_types.h"

namespace hg {
namespace res {
namespace {

constexpr int kThreads = 256;
constexpr int kWide = 4096;  // columns a wave holds (64 lanes x 8 vectors of 8)

struct NormArgs {
    int64_t m, xs, rs, ys, ss;
    int c;
    float eps, inv_c;
    const void *x, *r;
    const float *w;
    void *y, *s;
    float *scale, *rstd;
};

// Rows of at most G * I * 8 columns, G lanes a row.
template <typename T, typename Y, int G, int I>
__global__ __launch_bounds__(kThreads) void norm_kernel(const NormArgs a) {
    const int lane = threadIdx.x % G;
    const int64_t rows = (int64_t)gridDim.x * (kThreads / G);
    float w[I][8];
    int left[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        left[i] = a.c - (i * G + lane) * 8;
        load8(a.w + (i * G + lane) * 8, left[i], w[i]);
    }
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G; row < a.m; row += rows) {
        float v[I][8];
        const T *x = (const T *)a.x + row * a.xs + lane * 8;
        const T *r = (const T *)a.r + row * a.rs + lane * 8;
#pragma unroll
        for (int i = 0; i < I; ++i) load8(x + i * G * 8, left[i], v[i]);
        if (a.r) {
#pragma unroll
            for (int i = 0; i < I; ++i) {
                float t[8];
                load8(r + i * G * 8, left[i], t);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += t[j];
            }
        }
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sq = fmaf(v[i][j], v[i][j], sq);
        sq = group_sum<G>(sq);
        const float q = 1.f / sqrtf(sq * a.inv_c + a.eps);
        if (a.s) {
            T *s = (T *)a.s + row * a.ss + lane * 8;
#pragma unroll
            for (int i = 0; i < I; ++i) store8(s + i * G * 8, left[i], v[i]);
        }
        if (a.rstd && lane == 0) a.rstd[row] = q;
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * q * w[i][j];
        if constexpr (sizeof(Y) == 1) {
            float top = 0.f, bad = 0.f;
#pragma unroll
            for (int i = 0; i < I; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    top = fmaxf(top, fabsf(v[i][j]));
                    bad = v[i][j] != v[i][j] ? 1.f : bad;
                }
            top = group_max<G>(top);
            bad = group_max<G>(bad);
            if (bad != 0.f) top = __builtin_nanf("");  // a row with a NaN has the scale NaN
            const float inv = top > 0.f ? 448.f / top : 0.f;
#pragma unroll
            for (int i = 0; i < I; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = fminf(fmaxf(v[i][j] * inv, -448.f), 448.f);
            if (lane == 0) a.scale[row] = top / 448.f;
        }
        Y *y = (Y *)a.y + row * a.ys + lane * 8;
#pragma unroll
        for (int i = 0; i < I; ++i) store8(y + i * G * 8, left[i], v[i]);
    }
}

// Sum (or maximum) over the workgroup, in every thread.
template <bool kMax>
__device__ __forceinline__ float block_all(float v, float *lds) {
    v = kMax ? group_max<64>(v) : group_sum<64>(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = lds[0];
    for (int i = 1; i < kThreads / 64; ++i) t = kMax ? fmaxf(t, lds[i]) : t + lds[i];
    return t;
}

// Rows of any length, a workgroup a row: the row is read again for its output
// (it is in L2 by then).
template <typename T, typename Y>
__global__ __launch_bounds__(kThreads) void norm_long_kernel(const NormArgs a) {
    __shared__ float lds[kThreads / 64];
    for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x) {
        const T *x = (const T *)a.x + row * a.xs, *r = (const T *)a.r + row * a.rs;
        auto sum8 = [&](int at, float (&v)[8]) {
            load8(x + at, a.c - at, v);
            if (a.r) {
                float t[8];
                load8(r + at, a.c - at, t);
                for (int j = 0; j < 8; ++j) v[j] += t[j];
            }
        };
        float sq = 0.f, v[8], w[8];
        for (int at = threadIdx.x * 8; at < a.c; at += kThreads * 8) {
            sum8(at, v);
            for (int j = 0; j < 8; ++j) sq = fmaf(v[j], v[j], sq);
        }
        sq = block_all<false>(sq, lds);
        const float q = 1.f / sqrtf(sq * a.inv_c + a.eps);
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = q;
        float inv = 1.f;
        if constexpr (sizeof(Y) == 1) {
            float top = 0.f, bad = 0.f;
            for (int at = threadIdx.x * 8; at < a.c; at += kThreads * 8) {
                sum8(at, v);
                load8(a.w + at, a.c - at, w);
                for (int j = 0; j < 8; ++j) {
                    const float y = v[j] * q * w[j];
                    top = fmaxf(top, fabsf(y));
                    bad = y != y ? 1.f : bad;
                }
            }
            top = block_all<true>(top, lds);
            bad = block_all<true>(bad, lds);
            if (bad != 0.f) top = __builtin_nanf("");
            inv = top > 0.f ? 448.f / top : 0.f;
            if (threadIdx.x == 0) a.scale[row] = top / 448.f;
        }
        for (int at = threadIdx.x * 8; at < a.c; at += kThreads * 8) {
            sum8(at, v);
            load8(a.w + at, a.c - at, w);
            // s may be x or r itself: this thread has read what it overwrites
            if (a.s) store8((T *)a.s + row * a.ss + at, a.c - at, v);
            for (int j = 0; j < 8; ++j) {
                v[j] = v[j] * q * w[j];
                if constexpr (sizeof(Y) == 1) v[j] = fminf(fmaxf(v[j] * inv, -448.f), 448.f);
            }
            store8((Y *)a.y + row * a.ys + at, a.c - at, v);
        }
    }
}

template <typename T, typename Y, int G, int I>
void norm_run(const NormArgs &a, hipStream_t stream) {
    const int64_t need = div_up(a.m, kThreads / G);
    const int64_t most = kCus * 8;  // resident workgroups: w is loaded once for many rows
    norm_kernel<T, Y, G, I><<<dim3((unsigned)(need < most ? need : most)), kThreads, 0, stream>>>(a);
}

template <typename T, typename Y>
void norm_pick(const NormArgs &a, hipStream_t stream) {
    const int v = (a.c + 7) / 8;  // vectors of 8 in a row
    if (v <= 4) norm_run<T, Y, 4, 1>(a, stream);
    else if (v <= 8) norm_run<T, Y, 8, 1>(a, stream);
    else if (v <= 16) norm_run<T, Y, 16, 1>(a, stream);
    else if (v <= 32) norm_run<T, Y, 32, 1>(a, stream);
    else if (v <= 64) norm_run<T, Y, 64, 1>(a, stream);
    else if (v <= 128) norm_run<T, Y, 64, 2>(a, stream);
    else if (v <= 256) norm_run<T, Y, 64, 4>(a, stream);
    else if (v <= 512) norm_run<T, Y, 64, 8>(a, stream);
    else {
        const int64_t most = kCus * 8;
        norm_long_kernel<T, Y><<<dim3((unsigned)(a.m < most ? a.m : most)), kThreads, 0, stream>>>(a);
    }
}

struct GradArgs {
    int64_t m, dys, ss, dss, dxs;
    int c;
    float inv_c;
    const void *dy, *s, *ds;
    const float *w, *rstd;
    void *dx;
    float *part;  // [workgroups][c]
};

// Backward of rows of at most G * I * 8 columns.  Each lane keeps its columns'
// share of dw over its rows; a workgroup's shares are added in LDS in lane
// order and written as one partial row, so dw does not depend on scheduling.
template <typename T, int G, int I>
__global__ __launch_bounds__(kThreads) void norm_grad_kernel(const GradArgs a) {
    __shared__ float lds[kThreads * 8];
    const int lane = threadIdx.x % G;
    const int64_t rows = (int64_t)gridDim.x * (kThreads / G);
    float w[I][8], dw[I][8];
    int left[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        left[i] = a.c - (i * G + lane) * 8;
        load8(a.w + (i * G + lane) * 8, left[i], w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    }
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G; row < a.m; row += rows) {
        float dy[I][8], h[I][8];
        const T *py = (const T *)a.dy + row * a.dys + lane * 8, *ps = (const T *)a.s + row * a.ss + lane * 8;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            load8(py + i * G * 8, left[i], dy[i]);
            load8(ps + i * G * 8, left[i], h[i]);
        }
        const float q = a.rstd[row];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[i][j] *= q;
                dw[i][j] = fmaf(dy[i][j], h[i][j], dw[i][j]);
                dy[i][j] *= w[i][j];
                dot = fmaf(dy[i][j], h[i][j], dot);
            }
        dot = group_sum<G>(dot) * a.inv_c;
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) dy[i][j] = q * (dy[i][j] - h[i][j] * dot);
        if (a.ds) {
            const T *pd = (const T *)a.ds + row * a.dss + lane * 8;
#pragma unroll
            for (int i = 0; i < I; ++i) {
                float t[8];
                load8(pd + i * G * 8, left[i], t);
#pragma unroll
                for (int j = 0; j < 8; ++j) dy[i][j] += t[j];
            }
        }
        T *px = (T *)a.dx + row * a.dxs + lane * 8;
#pragma unroll
        for (int i = 0; i < I; ++i) store8(px + i * G * 8, left[i], dy[i]);
    }
    if (!a.part) return;
#pragma unroll
    for (int i = 0; i < I; ++i) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) lds[threadIdx.x * 8 + j] = dw[i][j];
        __syncthreads();
        for (int k = threadIdx.x; k < G * 8; k += kThreads) {
            float t = 0.f;
            for (int g = 0; g < kThreads / G; ++g) t += lds[g * G * 8 + k];
            const int col = i * G * 8 + k;
            if (col < a.c) a.part[(int64_t)blockIdx.x * a.c + col] = t;
        }
    }
}

// dx of rows of any length, and dw in a pass of its own (below).
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_grad_long_kernel(const GradArgs a) {
    __shared__ float lds[kThreads / 64];
    for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x) {
        const T *py = (const T *)a.dy + row * a.dys, *ps = (const T *)a.s + row * a.ss;
        const float q = a.rstd[row];
        float dot = 0.f, dy[8], s[8], w[8], t[8];
        for (int at = threadIdx.x * 8; at < a.c; at += kThreads * 8) {
            load8(py + at, a.c - at, dy);
            load8(ps + at, a.c - at, s);
            load8(a.w + at, a.c - at, w);
            for (int j = 0; j < 8; ++j) dot = fmaf(dy[j] * w[j], s[j] * q, dot);
        }
        dot = block_all<false>(dot, lds) * a.inv_c;
        for (int at = threadIdx.x * 8; at < a.c; at += kThreads * 8) {
            load8(py + at, a.c - at, dy);
            load8(ps + at, a.c - at, s);
            load8(a.w + at, a.c - at, w);
            for (int j = 0; j < 8; ++j) dy[j] = q * (dy[j] * w[j] - s[j] * q * dot);
            if (a.ds) {
                load8((const T *)a.ds + row * a.dss + at, a.c - at, t);
                for (int j = 0; j < 8; ++j) dy[j] += t[j];
            }
            store8((T *)a.dx + row * a.dxs + at, a.c - at, dy);
        }
    }
}
// Partial rows of dw of long rows: workgroup (columns, rows) sums its columns
// over its rows.
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_dw_long_kernel(const GradArgs a) {
    const int at = (blockIdx.x * kThreads + threadIdx.x) * 8;
    if (at >= a.c) return;
    float dw[8] = {}, dy[8], s[8];
    for (int64_t row = blockIdx.y; row < a.m; row += gridDim.y) {
        load8((const T *)a.dy + row * a.dys + at, a.c - at, dy);
        load8((const T *)a.s + row * a.ss + at, a.c - at, s);
        const float q = a.rstd[row];
        for (int j = 0; j < 8; ++j) dw[j] = fmaf(dy[j], s[j] * q, dw[j]);
    }
    store8(a.part + (int64_t)blockIdx.y * a.c + at, a.c - at, dw);
}

// dw = (dw +) the partial rows' sum: 64 columns a workgroup, 16 waves share the rows.
__global__ __launch_bounds__(1024) void dw_join_kernel(const float *part, int rows, int c, float *dw, int accumulate) {
    __shared__ float lds[16][64];
    const int col = blockIdx.x * 64 + (threadIdx.x & 63), wave = threadIdx.x >> 6;
    float t = 0.f;
    if (col < c)
#pragma unroll 8
        for (int r = wave; r < rows; r += 16) t += part[(int64_t)r * c + col];
    lds[wave][threadIdx.x & 63] = t;
    __syncthreads();
    if (wave == 0 && col < c) {
        for (int i = 1; i < 16; ++i) t += lds[i][threadIdx.x];
        dw[col] = accumulate ? dw[col] + t : t;
    }
}

int grad_group(int c) {
    const int v = (c + 7) / 8;
    return v <= 4 ? 4 : v <= 8 ? 8 : v <= 16 ? 16 : v <= 32 ? 32 : 64;
}
// Workgroups (and partial rows) of a backward: enough to fill the chip twice
// over, few enough that the partial rows stay small.
int64_t grad_groups(int64_t m, int c) {
    if (c > kWide) return m < 256 ? m : 256;
    if (m == 0) return 0;
    const int64_t need = div_up(m, kThreads / grad_group(c)), most = kCus * 4;
    return need < most ? need : most;
}

template <typename T, int G, int I>
void grad_run(const GradArgs &a, hipStream_t stream) {
    norm_grad_kernel<T, G, I><<<dim3((unsigned)grad_groups(a.m, a.c)), kThreads, 0, stream>>>(a);
}

template <typename T>
void grad_pick(const GradArgs &a, hipStream_t stream) {
    const int v = (a.c + 7) / 8;
    if (v <= 4) grad_run<T, 4, 1>(a, stream);
    else if (v <= 8) grad_run<T, 8, 1>(a, stream);
    else if (v <= 16) grad_run<T, 16, 1>(a, stream);
    else if (v <= 32) grad_run<T, 32, 1>(a, stream);
    else if (v <= 64) grad_run<T, 64, 1>(a, stream);
    else if (v <= 128) grad_run<T, 64, 2>(a, stream);
    else if (v <= 256) grad_run<T, 64, 4>(a, stream);
    else if (v <= 512) grad_run<T, 64, 8>(a, stream);
    else {
        const int64_t most = kCus * 8;
        norm_grad_long_kernel<T><<<dim3((unsigned)(a.m < most ? a.m : most)), kThreads, 0, stream>>>(a);
        if (a.part)
            norm_dw_long_kernel<T><<<dim3((unsigned)div_up(a.c, kThreads * 8), (unsigned)grad_groups(a.m, a.c)), kThreads, 0,
                                     stream>>>(a);
    }
}

}  // namespace

hipError_t launch_rms_norm_forward(const hg_rms_norm &op, hipStream_t stream) {
    const NormArgs a{op.m, op.x_stride, op.residual_stride, op.y_stride, op.sum_stride, op.c, op.eps, 1.f / (float)op.c,
                     op.x, op.residual, op.w, op.y, op.sum, op.y_scale, op.rstd};
    const bool q = op.y_dtype == HG_F8;
    if (op.dtype == HG_F16) q ? norm_pick<f16, f8>(a, stream) : norm_pick<f16, f16>(a, stream);
    else if (op.dtype == HG_BF16) q ? norm_pick<bf16, f8>(a, stream) : norm_pick<bf16, bf16>(a, stream);
    else q ? norm_pick<float, f8>(a, stream) : norm_pick<float, float>(a, stream);
    return hipGetLastError();
}

size_t rms_norm_backward_bytes(const hg_rms_norm_grad &op) {
    return op.dw ? (size_t)grad_groups(op.m, op.c) * op.c * sizeof(float) : 0;
}

hipError_t launch_rms_norm_backward(const hg_rms_norm_grad &op, void *workspace, hipStream_t stream) {
    const GradArgs a{op.m, op.dy_stride, op.sum_stride, op.ds_stride, op.dx_stride, op.c, 1.f / (float)op.c,
                     op.dy, op.sum, op.ds, op.w, op.rstd, op.dx, op.dw ? (float *)workspace : nullptr};
    if (op.m == 0) {
    } else if (op.dtype == HG_F16) grad_pick<f16>(a, stream);
    else if (op.dtype == HG_BF16) grad_pick<bf16>(a, stream);
    else grad_pick<float>(a, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !op.dw) return e;
    dw_join_kernel<<<dim3((unsigned)div_up(op.c, 64)), 1024, 0, stream>>>((const float *)workspace,
                                                                         (int)grad_groups(op.m, op.c), op.c, op.dw,
                                                                         op.accumulate);
    return hipGetLastError();
}

}  // namespace res
}  // namespace hg
