// Layer norm with the residual's addition, and its backward (gfx950).
//
//   s = x + r,  mu = mean(s),  q = 1 / sqrt(mean((s - mu)^2) + eps),  y = (s - mu) q w + b
//   g = w dy,  h = (s - mu) q,  dx = q (g - mean(g) - h mean(g h)) + ds,  dw = sum dy h,  db = sum dy
//
// One pass over the data: a row lies in the registers of a group of lanes while
// its mean and then the mean square of its differences are found, so the variance
// loses nothing to a large mean and costs no second read.  A mean is a quotient, not
// a product that the compiler may fuse into the differences: rows of one value, whose
// sum is exact, have differences of 0.  Everything is fp32 between the loads and the
// one rounding of each output; y is made from the unrounded s.  8-bit rows as the RMS
// norm's.
// Bound by memory: 2^18 x 256 bf16 with residual, s and statistics kept 104 us (5.2 TB/s),
// 2^20 x 256 to 8 bits 270 (5.0); backward 2^18 x 256 110 (4.9), 200003 x 96 f16 39 (4.0, of it
// 5 the launch that joins dw and db).
#include "norm_common.h"

namespace hg {
namespace res {
namespace {

struct LayerArgs {
    int64_t m, xs, rs, ys, ss;
    int c;
    float eps, inv_c, count;
    const void *x, *r;
    const float *w, *b;
    void *y, *s;
    float *scale, *mean, *rstd;
};

// A piece of a vector that may be left out.
template <bool kShort>
__device__ __forceinline__ void load_or(const float *p, float other, Columns at, int width, float (&v)[8]) {
    if (p) load8<kShort>(p, at, width, v);
    else
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = other;
}

// Sum of a piece's slots that count.  (Rows of whole pieces: all of them, or none.)
__device__ __forceinline__ float piece_sum(const float (&v)[8], Columns at, bool whole) {
    float t = 0.f;
    if (whole) {
#pragma unroll
        for (int j = 0; j < 8; ++j) t += v[j];
        return at.drop ? 0.f : t;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) t += j < at.drop ? 0.f : v[j];
    return t;
}
__device__ __forceinline__ float piece_square(const float (&v)[8], float mu, Columns at, bool whole) {
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float d = v[j] - mu;
        if (whole) t = fmaf(d, d, t);
        else t += j < at.drop ? 0.f : d * d;
    }
    return whole && at.drop ? 0.f : t;
}
// Columns past a row shorter than a piece hold zeros, not values.
__device__ __forceinline__ void clear_past(float (&v)[8], int width) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < width ? v[j] : 0.f;
}

// Rows of at most G * I * 8 columns, G lanes a row.
template <typename T, typename Y, int G, int I>
__global__ __launch_bounds__(kThreads) void layer_kernel(const LayerArgs a) {
    __shared__ float lds[2][kThreads / 64];
    int turn = 0;
    const int lane = threadIdx.x % G;
    const int64_t rows = (int64_t)gridDim.x * (kThreads / G);
    const bool whole = a.c % 8 == 0;
    float w[I][8], b[I][8];
    Columns at[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        at[i] = columns_of((i * G + lane) * 8, a.c);
        load_or<G == 4>(a.w, 1.f, at[i], a.c, w[i]);
        load_or<G == 4>(a.b, 0.f, at[i], a.c, b[i]);
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
        float sum = 0.f, sq = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i) sum += piece_sum(v[i], at[i], whole);
        const float mu = row_all<G, false>(sum, lds, turn) / a.count;
        if (G == 4 && a.c < 8) {  // the slots past the row would count as differences
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = v[0][j] - mu;
                sq += j < a.c && at[0].drop == 0 ? d * d : 0.f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < I; ++i) sq += piece_square(v[i], mu, at[i], whole);
        }
        sq = row_all<G, false>(sq, lds, turn);
        const float q = 1.f / sqrtf(sq * a.inv_c + a.eps);
        if (a.s)
#pragma unroll
            for (int i = 0; i < I; ++i) store8<G == 4>((T *)a.s + row * a.ss, at[i], a.c, v[i]);
        if (lane == 0) {
            if (a.mean) a.mean[row] = mu;
            if (a.rstd) a.rstd[row] = q;
        }
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] = fmaf((v[i][j] - mu) * q, w[i][j], b[i][j]);
        if constexpr (sizeof(Y) == 1) {
            if (G == 4 && a.c < 8) clear_past(v[0], at[0].drop ? 0 : a.c);  // (they are no part of the maximum)
            float top = 0.f, bad = 0.f;
#pragma unroll
            for (int i = 0; i < I; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float t = at[i].drop >= 8 ? 0.f : v[i][j];
                    top = fmaxf(top, fabsf(t));
                    bad = t != t ? 1.f : bad;
                }
            if (bad != 0.f) top = __builtin_inff();  // a row with a NaN has the scale NaN: larger than any maximum on the way
            top = row_all<G, true>(top, lds, turn);
            if (top == __builtin_inff()) top = __builtin_nanf("");
            const Scaling sc = scaling_of(top);
#pragma unroll
            for (int i = 0; i < I; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = fminf(fmaxf(v[i][j] * sc.up * sc.inv, -448.f), 448.f);
            if (lane == 0) a.scale[row] = sc.scale;
        }
#pragma unroll
        for (int i = 0; i < I; ++i) store8<G == 4>((Y *)a.y + row * a.ys, at[i], a.c, v[i]);
    }
}

// Rows of any length, a workgroup a row: the row is read again for its variance
// and its output (it is in L2 by then).
template <typename T, typename Y>
__global__ __launch_bounds__(kThreads) void layer_long_kernel(const LayerArgs a) {
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
        float sum = 0.f, sq = 0.f, v[8], w[8], b[8];
        for (int k = threadIdx.x * 8; k < a.c; k += kThreads * 8) {
            const Columns at = columns_of(k, a.c);
            sum8(at, v);
            sum += piece_sum(v, at, false);
        }
        const float mu = row_all<kThreads, false>(sum, lds, turn) / a.count;
        for (int k = threadIdx.x * 8; k < a.c; k += kThreads * 8) {
            const Columns at = columns_of(k, a.c);
            sum8(at, v);
            sq += piece_square(v, mu, at, false);
        }
        sq = row_all<kThreads, false>(sq, lds, turn);
        const float q = 1.f / sqrtf(sq * a.inv_c + a.eps);
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[row] = mu;
            if (a.rstd) a.rstd[row] = q;
        }
        auto output8 = [&](Columns at, float (&y)[8]) {
            load_or<false>(a.w, 1.f, at, a.c, w);
            load_or<false>(a.b, 0.f, at, a.c, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = fmaf((v[j] - mu) * q, w[j], b[j]);
        };
        Scaling sc{};
        if constexpr (sizeof(Y) == 1) {
            float top = 0.f, bad = 0.f, y[8];
            for (int k = threadIdx.x * 8; k < a.c; k += kThreads * 8) {
                const Columns at = columns_of(k, a.c);
                sum8(at, v);
                output8(at, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    top = fmaxf(top, fabsf(y[j]));
                    bad = y[j] != y[j] ? 1.f : bad;
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
            float y[8];
            sum8(at, v);
            output8(at, y);
            if constexpr (sizeof(Y) == 1)
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = fminf(fmaxf(y[j] * sc.up * sc.inv, -448.f), 448.f);
            // s and y may be x or r themselves: each thread writes columns of its own
            if (a.s) store_own((T *)a.s + row * a.ss, at, a.c, v);
            store_own((Y *)a.y + row * a.ys, at, a.c, y);
        }
    }
}

template <typename T, typename Y, int G, int I>
void layer_run(const LayerArgs &a, hipStream_t stream) {
    const int64_t need = div_up(a.m, kThreads / G);
    const int64_t most = kCus * 8;  // resident workgroups: w and b are loaded once for many rows
    layer_kernel<T, Y, G, I><<<dim3((unsigned)(need < most ? need : most)), kThreads, 0, stream>>>(a);
}

template <typename T, typename Y>
void layer_pick(const LayerArgs &a, hipStream_t stream) {
    const int v = (a.c + 7) / 8;  // vectors of 8 in a row
    if (v <= 4) layer_run<T, Y, 4, 1>(a, stream);
    else if (v <= 8) layer_run<T, Y, 8, 1>(a, stream);
    else if (v <= 16) layer_run<T, Y, 16, 1>(a, stream);
    else if (v <= 32) layer_run<T, Y, 32, 1>(a, stream);
    else if (v <= 64) layer_run<T, Y, 64, 1>(a, stream);
    else if (v <= 128) layer_run<T, Y, 64, 2>(a, stream);
    else if (v <= 256) layer_run<T, Y, 256, 1>(a, stream);
    else if (v <= 512) layer_run<T, Y, 256, 2>(a, stream);
    else {
        const int64_t most = kCus * 8;
        layer_long_kernel<T, Y><<<dim3((unsigned)(a.m < most ? a.m : most)), kThreads, 0, stream>>>(a);
    }
}

struct LayerGradArgs {
    int64_t m, dys, ss, dss, dxs;
    int c, want_dw, want_db;
    float inv_c, count;
    const void *dy, *s, *ds;
    const float *w, *mean, *rstd;
    void *dx;
    float *part;  // [workgroups][dw's c columns, db's c columns: those asked for]
};
__device__ __forceinline__ int64_t part_row(const LayerGradArgs &a) { return (int64_t)(a.want_dw + a.want_db) * a.c; }

// A product that is rounded by itself: where a row's gradients cancel, as in a row
// of one column, g - mean(g) is 0 only if both g are the same number.
__device__ __forceinline__ float product(float a, float b) {
#pragma clang fp contract(off)
    return a * b;
}

// Backward of rows of at most G * I * 8 columns.  Each lane keeps its columns'
// shares of dw and db over its rows; a workgroup's shares are added in LDS in lane
// order and written as one partial row, so they do not depend on scheduling.
template <typename T, int G, int I>
__global__ __launch_bounds__(kThreads) void layer_grad_kernel(const LayerGradArgs a) {
    __shared__ float lds[kThreads * 8], ends[2][kThreads / 64];
    int turn = 0;
    const int lane = threadIdx.x % G;
    const int64_t rows = (int64_t)gridDim.x * (kThreads / G);
    const bool whole = a.c % 8 == 0;
    float w[I][8], dw[I][8], db[I][8];
    Columns at[I];
#pragma unroll
    for (int i = 0; i < I; ++i) {
        at[i] = columns_of((i * G + lane) * 8, a.c);
        load_or<G == 4>(a.w, 1.f, at[i], a.c, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.f;
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
        const float mu = a.mean[row], q = a.rstd[row];
        float sum = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < I; ++i) {
            float t = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                h[i][j] = (h[i][j] - mu) * q;
                dw[i][j] = fmaf(dy[i][j], h[i][j], dw[i][j]);
                db[i][j] += dy[i][j];
                dy[i][j] = product(dy[i][j], w[i][j]);
                if (whole) t = fmaf(dy[i][j], h[i][j], t);
                else t += j < at[i].drop ? 0.f : dy[i][j] * h[i][j];  // (dy past a row shorter than a piece is 0)
            }
            dot += at[i].drop >= 8 ? 0.f : t;
            sum += piece_sum(dy[i], at[i], whole);
        }
        sum = row_all<G, false>(sum, ends, turn) / a.count;
        dot = row_all<G, false>(dot, ends, turn) * a.inv_c;
#pragma unroll
        for (int i = 0; i < I; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                dy[i][j] = q * (dy[i][j] - sum - h[i][j] * dot);
                if (a.ds) dy[i][j] += ds[i][j];
            }
            store8<G == 4>((T *)a.dx + row * a.dxs, at[i], a.c, dy[i]);
        }
    }
    if (!a.part) return;
    float *part = a.part + (int64_t)blockIdx.x * part_row(a);
    auto leave = [&](const float (&mine)[8], int i) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) lds[threadIdx.x * 8 + j] = mine[j];
        __syncthreads();
        for (int k = threadIdx.x; k < G * 8; k += kThreads) {
            float t = 0.f;
            for (int g = 0; g < kThreads / G; ++g) t += lds[g * G * 8 + k];
            const int col = column_of(i * G * 8 + k, a.c);
            if (col >= 0) part[col] = t;
        }
    };
    if (a.want_dw)
#pragma unroll
        for (int i = 0; i < I; ++i) leave(dw[i], i);
    part += a.want_dw ? a.c : 0;
    if (a.want_db)
#pragma unroll
        for (int i = 0; i < I; ++i) leave(db[i], i);
}

// dx of rows of any length, and dw and db in a pass of their own (below).
template <typename T>
__global__ __launch_bounds__(kThreads) void layer_grad_long_kernel(const LayerGradArgs a) {
    __shared__ float lds[2][kThreads / 64];
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x) {
        const T *py = (const T *)a.dy + row * a.dys, *ps = (const T *)a.s + row * a.ss;
        const float mu = a.mean[row], q = a.rstd[row];
        float sum = 0.f, dot = 0.f, dy[8], s[8], w[8], t[8];
        for (int k = threadIdx.x * 8; k < a.c; k += kThreads * 8) {
            const Columns at = columns_of(k, a.c);
            load8<false>(py, at, a.c, dy);
            load8<false>(ps, at, a.c, s);
            load_or<false>(a.w, 1.f, at, a.c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float g = product(dy[j], w[j]);
                sum += j < at.drop ? 0.f : g;
                dot += j < at.drop ? 0.f : g * ((s[j] - mu) * q);
            }
        }
        sum = row_all<kThreads, false>(sum, lds, turn) / a.count;
        dot = row_all<kThreads, false>(dot, lds, turn) * a.inv_c;
        for (int k = threadIdx.x * 8; k < a.c; k += kThreads * 8) {
            const Columns at = columns_of(k, a.c);
            load8<false>(py, at, a.c, dy);
            load8<false>(ps, at, a.c, s);
            load_or<false>(a.w, 1.f, at, a.c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) dy[j] = q * (product(dy[j], w[j]) - sum - (s[j] - mu) * q * dot);
            if (a.ds) {
                load8<false>((const T *)a.ds + row * a.dss, at, a.c, t);
#pragma unroll
                for (int j = 0; j < 8; ++j) dy[j] += t[j];
            }
            store8<false>((T *)a.dx + row * a.dxs, at, a.c, dy);
        }
    }
}
// Partial rows of dw and db of long rows: workgroup (columns, rows) sums its
// columns over its rows.
template <typename T>
__global__ __launch_bounds__(kThreads) void layer_dw_long_kernel(const LayerGradArgs a) {
    const Columns at = columns_of((blockIdx.x * kThreads + threadIdx.x) * 8, a.c);
    if (at.drop >= 8) return;
    float dw[8] = {}, db[8] = {}, dy[8], s[8];
    for (int64_t row = blockIdx.y; row < a.m; row += gridDim.y) {
        load8<false>((const T *)a.dy + row * a.dys, at, a.c, dy);
        load8<false>((const T *)a.s + row * a.ss, at, a.c, s);
        const float mu = a.mean[row], q = a.rstd[row];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[j] = fmaf(dy[j], (s[j] - mu) * q, dw[j]);
            db[j] += dy[j];
        }
    }
    float *part = a.part + (int64_t)blockIdx.y * part_row(a);
    if (a.want_dw) store8<false>(part, at, a.c, dw);
    if (a.want_db) store8<false>(part + (a.want_dw ? a.c : 0), at, a.c, db);
}

// Workgroups (and partial rows) of a backward: as those of the RMS norm, but of rows
// that take a whole workgroup at least four each, where the card stays full: their
// partial rows are as long as the rows, twice (2048 x 4096: 52 us, 28 so).
int64_t layer_groups(int64_t m, int c) {
    const int64_t most = grad_groups(m, c);
    if (c > kNormHeld || grad_group(c) < kThreads || most <= kCus * 2) return most;
    const int64_t want = div_up(m, 4) > kCus * 2 ? div_up(m, 4) : kCus * 2;
    return want < most ? want : most;
}

template <typename T, int G, int I>
void layer_grad_run(const LayerGradArgs &a, hipStream_t stream) {
    layer_grad_kernel<T, G, I><<<dim3((unsigned)layer_groups(a.m, a.c)), kThreads, 0, stream>>>(a);
}

template <typename T>
void layer_grad_pick(const LayerGradArgs &a, hipStream_t stream) {
    const int v = (a.c + 7) / 8;
    if (v <= 4) layer_grad_run<T, 4, 1>(a, stream);
    else if (v <= 8) layer_grad_run<T, 8, 1>(a, stream);
    else if (v <= 16) layer_grad_run<T, 16, 1>(a, stream);
    else if (v <= 32) layer_grad_run<T, 32, 1>(a, stream);
    else if (v <= 64) layer_grad_run<T, 64, 1>(a, stream);
    else if (v <= 128) layer_grad_run<T, 64, 2>(a, stream);
    else if (v <= 256) layer_grad_run<T, 256, 1>(a, stream);
    else if (v <= 512) layer_grad_run<T, 256, 2>(a, stream);
    else {
        const int64_t most = kCus * 8;
        layer_grad_long_kernel<T><<<dim3((unsigned)(a.m < most ? a.m : most)), kThreads, 0, stream>>>(a);
        if (a.part)
            layer_dw_long_kernel<T><<<dim3((unsigned)div_up(a.c, kThreads * 8), (unsigned)layer_groups(a.m, a.c)), kThreads, 0,
                                      stream>>>(a);
    }
}

int outputs_of(const hg_layer_norm_grad &op) { return (op.dw ? 1 : 0) + (op.db ? 1 : 0); }

}  // namespace

hipError_t launch_layer_norm_forward(const hg_layer_norm &op, hipStream_t stream) {
    const LayerArgs a{op.m, op.x_stride, op.residual_stride, op.y_stride, op.sum_stride, op.c, op.eps, 1.f / (float)op.c, (float)op.c,
                      op.x, op.residual, op.w, op.b, op.y, op.sum, op.y_scale, op.mean, op.rstd};
    const bool q = op.y_dtype == HG_F8;
    if (op.dtype == HG_F16) q ? layer_pick<f16, f8>(a, stream) : layer_pick<f16, f16>(a, stream);
    else if (op.dtype == HG_BF16) q ? layer_pick<bf16, f8>(a, stream) : layer_pick<bf16, bf16>(a, stream);
    else q ? layer_pick<float, f8>(a, stream) : layer_pick<float, float>(a, stream);
    return hipGetLastError();
}

size_t layer_norm_backward_bytes(const hg_layer_norm_grad &op) {
    return (size_t)layer_groups(op.m, op.c) * op.c * outputs_of(op) * sizeof(float);
}

hipError_t launch_layer_norm_backward(const hg_layer_norm_grad &op, void *workspace, hipStream_t stream) {
    const int outputs = outputs_of(op);
    const LayerGradArgs a{op.m, op.dy_stride, op.sum_stride, op.ds_stride, op.dx_stride, op.c, op.dw != nullptr, op.db != nullptr,
                          1.f / (float)op.c, (float)op.c, op.dy, op.sum, op.ds, op.w, op.mean, op.rstd, op.dx,
                          outputs ? (float *)workspace : nullptr};
    if (op.m == 0) {
    } else if (op.dtype == HG_F16) layer_grad_pick<f16>(a, stream);
    else if (op.dtype == HG_BF16) layer_grad_pick<bf16>(a, stream);
    else layer_grad_pick<float>(a, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !outputs) return e;
    const int c = op.c * outputs;
    dw_join_kernel<<<dim3((unsigned)div_up(c, 16)), 1024, 0, stream>>>((const float *)workspace, (int)layer_groups(op.m, op.c), c, op.dw,
                                                                       op.dw ? op.c : 0, op.db, op.accumulate);
    return hipGetLastError();
}

}  // namespace res
}  // namespace hg
