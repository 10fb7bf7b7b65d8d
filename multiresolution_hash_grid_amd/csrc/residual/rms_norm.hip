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
// Bound by memory: 2^18 x 256 bf16 with s kept 98-101 us (5.4 TB/s), 2^20 x 256 to 8
// bits 254-259 us (5.2 TB/s), backward of 200003 x 96 f16 38 us (4.1 TB/s, a second
// launch that joins dw included).  Backward of few long rows: a workgroup has one row
// and writes a partial row of dw as long, so 2048 x 4096 bf16 takes 33 us.
#include "device_types.h"

namespace hg {
namespace res {
namespace {

constexpr int kThreads = 256;

// Sum or maximum over the G lanes of a row, in each of them: lanes of a wave, or
// (G = 256) the workgroup, through one of two LDS slots in turn, so that one
// barrier is enough.
template <int G, bool kMax>
__device__ __forceinline__ float row_all(float v, float (*lds)[kThreads / 64], int &turn) {
    auto join = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
#pragma unroll
    for (int o = 1; o < (G < 64 ? G : 64); o <<= 1) v = join(v, __shfl_xor(v, o, 64));
    if constexpr (G == kThreads) {
        if ((threadIdx.x & 63) == 0) lds[turn][threadIdx.x >> 6] = v;
        __syncthreads();
        v = lds[turn][0];
#pragma unroll
        for (int i = 1; i < kThreads / 64; ++i) v = join(v, lds[turn][i]);
        turn ^= 1;
    }
    return v;
}

// Of a row whose largest |y| is top: the scale of its 8-bit values, top / 448, and
// the factors up and inv that take y to them.  448 / top leaves fp32 where top is
// below 2^-119, so such rows are first moved up by a power of two, exactly.  A scale
// of 0 (top too small for one) makes a row of zeros, as does NaN.
struct Scaling {
    float scale, up, inv;
};
__device__ __forceinline__ Scaling scaling_of(float top) {
    Scaling s;
    s.scale = top / 448.f;
    s.up = top < 0x1p-100f ? 0x1p100f : 1.f;
    s.inv = s.scale > 0.f ? 448.f / (top * s.up) : 0.f;
    return s;
}

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
    __shared__ float lds[2][kThreads / 64];
    int turn = 0;
    const int lane = threadIdx.x % G;
    const int64_t rows = (int64_t)gridDim.x * (kThreads / G);
    float w[I][8];
    Columns at[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        at[i] = columns_of((i * G + lane) * 8, a.c);
        load8<G == 4>(a.w, at[i], a.c, w[i]);
    }
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G; row < a.m; row += rows) {
        float v[I][8];
#pragma unroll
        for (int i = 0; i < I; ++i) load8<G == 4>((const T *)a.x + row * a.xs, at[i], a.c, v[i]);
        if (a.r) {
#pragma unroll
            for (int i = 0; i < I; ++i) {
                float t[8];
                load8<G == 4>((const T *)a.r + row * a.rs, at[i], a.c, t);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] += t[j];
            }
        }
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            if (a.c % 8 == 0) {
                float t = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) t = fmaf(v[i][j], v[i][j], t);
                sq += at[i].drop ? 0.f : t;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) sq += j < at[i].drop ? 0.f : v[i][j] * v[i][j];
            }
        }
        sq = row_all<G, false>(sq, lds, turn);
        const float q = 1.f / sqrtf(sq * a.inv_c + a.eps);
        if (a.s)
#pragma unroll
            for (int i = 0; i < I; ++i) store8<G == 4>((T *)a.s + row * a.ss, at[i], a.c, v[i]);
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
            if (bad != 0.f) top = __builtin_inff();  // a row with a NaN has the scale NaN: larger than any maximum on the way
            top = row_all<G, true>(top, lds, turn);
            if (top == __builtin_inff()) top = __builtin_nanf("");
            const Scaling sc = scaling_of(top);
            if (sc.up != 1.f)
#pragma unroll
                for (int i = 0; i < I; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[i][j] *= sc.up;
#pragma unroll
            for (int i = 0; i < I; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = fminf(fmaxf(v[i][j] * sc.inv, -448.f), 448.f);
            if (lane == 0) a.scale[row] = sc.scale;
        }
#pragma unroll
        for (int i = 0; i < I; ++i) store8<G == 4>((Y *)a.y + row * a.ys, at[i], a.c, v[i]);
    }
}

// store8 without the slots that the piece before holds too.
template <typename T>
__device__ __forceinline__ void store_own(T *row, Columns c, int width, const float (&v)[8]) {
    if (c.drop == 0) {
        store8<false>(row, c, width, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j >= c.drop) {
            if constexpr (sizeof(T) == 1) row[c.at + j].bits = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[j], v[j], 0, false);
            else row[c.at + j] = (T)v[j];
        }
}

// Rows of any length, a workgroup a row: the row is read again for its output
// (it is in L2 by then).
template <typename T, typename Y>
__global__ __launch_bounds__(kThreads) void norm_long_kernel(const NormArgs a) {
    __shared__ float lds[2][kThreads / 64];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x) {
        const T *x = (const T *)a.x + row * a.xs, *r = (const T *)a.r + row * a.rs;
        auto sum8 = [&](Columns at, float (&v)[8]) {
            load8<false>(x, at, a.c, v);
            if (a.r) {
                float t[8];
                load8<false>(r, at, a.c, t);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] += t[j];
            }
        };
        float sq = 0.f, v[8], w[8];
        for (int k = threadIdx.x * 8; k < a.c; k += kThreads * 8) {
            const Columns at = columns_of(k, a.c);
            sum8(at, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) sq += j < at.drop ? 0.f : v[j] * v[j];
        }
        sq = row_all<kThreads, false>(sq, lds, turn);
        const float q = 1.f / sqrtf(sq * a.inv_c + a.eps);
        if (a.rstd && threadIdx.x == 0) a.rstd[row] = q;
        Scaling sc{};
        if constexpr (sizeof(Y) == 1) {
            float top = 0.f, bad = 0.f;
            for (int k = threadIdx.x * 8; k < a.c; k += kThreads * 8) {
                const Columns at = columns_of(k, a.c);
                sum8(at, v);
                load8<false>(a.w, at, a.c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float y = v[j] * q * w[j];
                    top = fmaxf(top, fabsf(y));
                    bad = y != y ? 1.f : bad;
                }
            }
            if (bad != 0.f) top = __builtin_inff();
            top = row_all<kThreads, true>(top, lds, turn);
            if (top == __builtin_inff()) top = __builtin_nanf("");
            sc = scaling_of(top);
            if (threadIdx.x == 0) a.scale[row] = sc.scale;
        }
        for (int k = threadIdx.x * 8; k < a.c; k += kThreads * 8) {
            const Columns at = columns_of(k, a.c);
            sum8(at, v);
            load8<false>(a.w, at, a.c, w);
            // s and y may be x or r themselves: each thread writes columns of its own
            if (a.s) store_own((T *)a.s + row * a.ss, at, a.c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = v[j] * q * w[j];
                if constexpr (sizeof(Y) == 1) v[j] = fminf(fmaxf(v[j] * sc.up * sc.inv, -448.f), 448.f);
            }
            store_own((Y *)a.y + row * a.ys, at, a.c, v);
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
    else if (v <= 256) norm_run<T, Y, 256, 1>(a, stream);
    else if (v <= 512) norm_run<T, Y, 256, 2>(a, stream);
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
    __shared__ float lds[kThreads * 8], ends[2][kThreads / 64];
    int turn = 0;
    const int lane = threadIdx.x % G;
    const int64_t rows = (int64_t)gridDim.x * (kThreads / G);
    float w[I][8], dw[I][8];
    Columns at[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        at[i] = columns_of((i * G + lane) * 8, a.c);
        load8<G == 4>(a.w, at[i], a.c, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
    }
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G; row < a.m; row += rows) {
        float dy[I][8], h[I][8], ds[I][8];
#pragma unroll
        for (int i = 0; i < I; ++i) {
            load8<G == 4>((const T *)a.dy + row * a.dys, at[i], a.c, dy[i]);
            load8<G == 4>((const T *)a.s + row * a.ss, at[i], a.c, h[i]);
        }
        if (a.ds)
#pragma unroll
            for (int i = 0; i < I; ++i) load8<G == 4>((const T *)a.ds + row * a.dss, at[i], a.c, ds[i]);
        const float q = a.rstd[row];
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            float t = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[i][j] *= q;
                dw[i][j] = fmaf(dy[i][j], h[i][j], dw[i][j]);
                dy[i][j] *= w[i][j];
                if (a.c % 8 == 0) t = fmaf(dy[i][j], h[i][j], t);
                else t += j < at[i].drop ? 0.f : dy[i][j] * h[i][j];
            }
            dot += at[i].drop >= 8 ? 0.f : t;
        }
        dot = row_all<G, false>(dot, ends, turn) * a.inv_c;
#pragma unroll
        for (int i = 0; i < I; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dy[i][j] = q * (dy[i][j] - h[i][j] * dot);
                if (a.ds) dy[i][j] += ds[i][j];
            }
            store8<G == 4>((T *)a.dx + row * a.dxs, at[i], a.c, dy[i]);
        }
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
            const int col = column_of(i * G * 8 + k, a.c);
            if (col >= 0) a.part[(int64_t)blockIdx.x * a.c + col] = t;
        }
    }
}

// dx of rows of any length, and dw in a pass of its own (below).
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_grad_long_kernel(const GradArgs a) {
    __shared__ float lds[2][kThreads / 64];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x) {
        const T *py = (const T *)a.dy + row * a.dys, *ps = (const T *)a.s + row * a.ss;
        const float q = a.rstd[row];
        float dot = 0.f, dy[8], s[8], w[8], t[8];
        for (int k = threadIdx.x * 8; k < a.c; k += kThreads * 8) {
            const Columns at = columns_of(k, a.c);
            load8<false>(py, at, a.c, dy);
            load8<false>(ps, at, a.c, s);
            load8<false>(a.w, at, a.c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) dot += j < at.drop ? 0.f : dy[j] * w[j] * (s[j] * q);
        }
        dot = row_all<kThreads, false>(dot, lds, turn) * a.inv_c;
        for (int k = threadIdx.x * 8; k < a.c; k += kThreads * 8) {
            const Columns at = columns_of(k, a.c);
            load8<false>(py, at, a.c, dy);
            load8<false>(ps, at, a.c, s);
            load8<false>(a.w, at, a.c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) dy[j] = q * (dy[j] * w[j] - s[j] * q * dot);
            if (a.ds) {
                load8<false>((const T *)a.ds + row * a.dss, at, a.c, t);
#pragma unroll
                for (int j = 0; j < 8; ++j) dy[j] += t[j];
            }
            store8<false>((T *)a.dx + row * a.dxs, at, a.c, dy);
        }
    }
}
// Partial rows of dw of long rows: workgroup (columns, rows) sums its columns
// over its rows.
template <typename T>
__global__ __launch_bounds__(kThreads) void norm_dw_long_kernel(const GradArgs a) {
    const Columns at = columns_of((blockIdx.x * kThreads + threadIdx.x) * 8, a.c);
    if (at.drop >= 8) return;
    float dw[8] = {}, dy[8], s[8];
    for (int64_t row = blockIdx.y; row < a.m; row += gridDim.y) {
        load8<false>((const T *)a.dy + row * a.dys, at, a.c, dy);
        load8<false>((const T *)a.s + row * a.ss, at, a.c, s);
        const float q = a.rstd[row];
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[j] = fmaf(dy[j], s[j] * q, dw[j]);
    }
    store8<false>(a.part + (int64_t)blockIdx.y * a.c, at, a.c, dw);
}

// dw = (dw +) the partial rows' sum: 16 columns a workgroup, 64 threads share the
// rows of each, and their sums are added in order, 16 and then four.
__global__ __launch_bounds__(1024) void dw_join_kernel(const float *part, int rows, int c, float *dw, int accumulate) {
    __shared__ float lds[64][16];
    const int slot = threadIdx.x & 15, share = threadIdx.x >> 4, col = blockIdx.x * 16 + slot;
    float t = 0.f;
    if (col < c)
#pragma unroll 8
        for (int r = share; r < rows; r += 64) t += part[(int64_t)r * c + col];
    lds[share][slot] = t;
    __syncthreads();
    if (share < 4) {
        t = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += lds[share * 16 + i][slot];
    }
    __syncthreads();
    if (share < 4) lds[share][slot] = t;
    __syncthreads();
    if (share == 0 && col < c) {
        t = lds[0][slot] + lds[1][slot] + lds[2][slot] + lds[3][slot];
        dw[col] = accumulate ? dw[col] + t : t;
    }
}

int grad_group(int c) {
    const int v = (c + 7) / 8;
    return v <= 4 ? 4 : v <= 8 ? 8 : v <= 16 ? 16 : v <= 32 ? 32 : v <= 128 ? 64 : 256;
}
// Workgroups (and partial rows) of a backward: as many as are resident.
int64_t grad_groups(int64_t m, int c) {
    if (c > kNormHeld) return m < 256 ? m : 256;
    if (m == 0) return 0;
    const int64_t need = div_up(m, kThreads / grad_group(c)), most = kCus * 8;
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
    else if (v <= 256) grad_run<T, 256, 1>(a, stream);
    else if (v <= 512) grad_run<T, 256, 2>(a, stream);
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
    dw_join_kernel<<<dim3((unsigned)div_up(op.c, 16)), 1024, 0, stream>>>((const float *)workspace,
                                                                         (int)grad_groups(op.m, op.c), op.c, op.dw,
                                                                         op.accumulate);
    return hipGetLastError();
}

}  // namespace res
}  // namespace hg
