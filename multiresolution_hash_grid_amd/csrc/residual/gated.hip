// h = act(x Wg^T + bg) (x Wu^T + bu) and its backward: the operands' types of the
// forward, each in a source of its own, and the backward's path for any width.
//
// Backward: dg and du are worked out once, rounded to the operands' type side by
// side in the workspace (their unrounded sums over the rows are dbg and dbu), and
// then
//   dx = [dg du] [Wg; Wu],  dwg = dg^T x,  dwu = du^T x
// through the linear layer's kernels.
#include "gated_common.h"
#include "norm_common.h"

namespace hg {
namespace res {
namespace {

constexpr int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

// dz [m][2 * padded], columns past n zero, and one partial row of the biases'
// gradients a workgroup.  G lanes a row and 8 columns a lane; blockIdx.y takes 8 G columns.
template <typename T, int G>
__global__ __launch_bounds__(kThreads) void gated_dz_kernel(const GatedGradArgs a, T *dz, int padded, float *part) {
    __shared__ float lds[kThreads * 8];
    const int lane = threadIdx.x % G, first = blockIdx.y * G * 8;
    const Columns col = columns_of(first + lane * 8, a.n);
    const int to = first + lane * 8;  // columns of dz: whole pieces, the first slot that counts in its place
    float dbg[8] = {}, dbu[8] = {};
    const int64_t rows = (int64_t)gridDim.x * (kThreads / G);
    for (int64_t row = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G; row < a.m; row += rows) {
        float g[8], u[8], dh[8], dg[8], du[8];
        load8<G == 4>((const T *)a.gate + row * a.ps, col, a.n, g);
        load8<G == 4>((const T *)a.up + row * a.qs, col, a.n, u);
        load8<G == 4>((const T *)a.dh + row * a.dhs, col, a.n, dh);
        gate_grad_all(g, u, dh, a.act, dg, du);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool counts = j >= col.drop && j < a.n;
            dg[j] = counts ? dg[j] : 0.f, du[j] = counts ? du[j] : 0.f;
            dbg[j] += dg[j], dbu[j] += du[j];
        }
        if (dz && to < padded) {
            T *const p = dz + row * 2 * padded + to;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (col.drop == 0) p[j] = (T)dg[j], p[padded + j] = (T)du[j];
                else if (j >= col.drop) p[j - col.drop] = (T)dg[j], p[padded + j - col.drop] = (T)du[j];
                if (j < col.drop) p[7 - j] = (T)0.f, p[padded + 7 - j] = (T)0.f;
            }
        }
    }
    if (!part) return;
    float *to_part = part + (int64_t)blockIdx.x * 2 * a.n;
    auto leave = [&](const float (&mine)[8]) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) lds[threadIdx.x * 8 + j] = mine[j];
        __syncthreads();
        for (int k = threadIdx.x; k < G * 8; k += kThreads) {
            float t = 0.f;
            for (int r = 0; r < kThreads / G; ++r) t += lds[r * G * 8 + k];
            const int c = column_of(first + k, a.n);
            if (c >= 0) to_part[c] = t;
        }
    };
    leave(dbg);
    to_part += a.n;
    leave(dbu);
}

// [Wg; Wu]^T: [k][2 * padded], zeros where there is no unit.
template <typename T>
__global__ __launch_bounds__(256) void gated_transpose_kernel(const GatedGradArgs a, T *wt, int padded) {
    __shared__ T tile[32][33];
    const int c = threadIdx.x & 31, r0 = threadIdx.x >> 5, half = blockIdx.z;
    const T *const w = (const T *)(half ? a.wu : a.wg);
    const int64_t ws = half ? a.us : a.gs;
    for (int r = r0; r < 32; r += 8) {
        const int i = blockIdx.y * 32 + r, j = blockIdx.x * 32 + c;
        tile[r][c] = i < a.n && j < a.k ? w[(int64_t)i * ws + j] : (T)0.f;
    }
    __syncthreads();
    for (int r = r0; r < 32; r += 8) {
        const int j = blockIdx.x * 32 + r, i = blockIdx.y * 32 + c;
        if (i < padded && j < a.k) wt[(int64_t)j * 2 * padded + half * padded + i] = tile[c][r];
    }
}

struct GatedPlan {
    int padded, lanes, groups;
    int64_t part_at, dz_at, wt_at, inner_at, bytes;
};

hg_linear_grad half_grad(const hg_gated_grad &op, const GatedPlan &p, int half, void *workspace) {
    hg_linear_grad l{};
    l.m = op.m, l.k = op.k, l.n = op.n;
    l.dy = (char *)workspace + p.dz_at + (size_t)half * p.padded * 2, l.dy_stride = 2 * p.padded;
    l.x = op.x, l.x_stride = op.m > 1 ? op.x_stride : op.k;
    l.dw = half ? op.dwu : op.dwg, l.dw_stride = half ? op.dwu_stride : op.dwg_stride;
    l.dtype = l.dy_dtype = op.dtype, l.dw_dtype = op.dw_dtype, l.act = HG_ACT_NONE, l.accumulate = op.accumulate;
    return l;
}

GatedPlan gated_plan(const hg_gated_grad &op) {
    GatedPlan p{};
    p.padded = (op.n + 7) / 8 * 8;
    const int pieces = p.padded / 8;
    p.lanes = pieces <= 4 ? 4 : pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : pieces <= 64 ? 64 : 256;
    const int64_t need = div_up(op.m, kThreads / p.lanes), most = kCus * 8 / div_up(pieces, p.lanes);
    p.groups = (int)(need < most ? need : most < 1 ? 1 : most);
    if (op.m == 0) return p;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t was = at;
        at += up256(bytes);
        return was;
    };
    p.part_at = take(op.dbg ? (int64_t)p.groups * 2 * op.n * 4 : 0);
    p.dz_at = take(op.dx || op.dwg ? op.m * 2 * p.padded * 2 : 0);
    p.wt_at = take(op.dx ? (int64_t)op.k * 2 * p.padded * 2 : 0);
    p.inner_at = at;
    if (op.dwg) at += up256((int64_t)linear_backward_bytes(half_grad(op, p, 0, nullptr)));
    p.bytes = at;
    return p;
}

template <typename T>
hipError_t gated_grad_run(const hg_gated_grad &op, const GatedGradArgs &a, char *ws, hipStream_t stream) {
    const GatedPlan p = gated_plan(op);
    hipError_t e;
    T *const dz = (T *)(ws + p.dz_at), *const wt = (T *)(ws + p.wt_at);
    float *const part = op.dbg ? (float *)(ws + p.part_at) : nullptr;
    if (a.m > 0) {
        const dim3 grid((unsigned)p.groups, (unsigned)div_up(p.padded / 8, p.lanes));
        T *const out = op.dx || op.dwg ? dz : nullptr;
        switch (p.lanes) {
        case 4: gated_dz_kernel<T, 4><<<grid, kThreads, 0, stream>>>(a, out, p.padded, part); break;
        case 8: gated_dz_kernel<T, 8><<<grid, kThreads, 0, stream>>>(a, out, p.padded, part); break;
        case 16: gated_dz_kernel<T, 16><<<grid, kThreads, 0, stream>>>(a, out, p.padded, part); break;
        case 32: gated_dz_kernel<T, 32><<<grid, kThreads, 0, stream>>>(a, out, p.padded, part); break;
        case 64: gated_dz_kernel<T, 64><<<grid, kThreads, 0, stream>>>(a, out, p.padded, part); break;
        default: gated_dz_kernel<T, 256><<<grid, kThreads, 0, stream>>>(a, out, p.padded, part);
        }
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (op.dbg) {
        dw_join_kernel<<<dim3((unsigned)div_up(2 * a.n, 16)), 1024, 0, stream>>>(part, a.m > 0 ? p.groups : 0, 2 * a.n, a.dbg, a.n,
                                                                                 a.dbu, a.accumulate);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (op.dwg)
        for (int half = 0; half < 2; ++half)
            if ((e = launch_linear_backward(half_grad(op, p, half, ws), ws + p.inner_at, stream)) != hipSuccess) return e;
    if (op.dx && a.m > 0) {
        gated_transpose_kernel<T><<<dim3((unsigned)div_up(a.k, 32), (unsigned)div_up(p.padded, 32), 2), 256, 0, stream>>>(a, wt, p.padded);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hg_linear f{};
        f.m = a.m, f.k = 2 * p.padded, f.n = a.k;
        f.x = dz, f.x_stride = 2 * p.padded, f.w = wt, f.w_stride = 2 * p.padded, f.y = op.dx, f.y_stride = op.dx_stride;
        f.x_dtype = f.y_dtype = op.dtype, f.act = HG_ACT_NONE;
        return launch_linear_forward(f, stream);
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_gated_forward(const hg_gated &op, hipStream_t stream) {
    const GatedArgs a{op.m, op.x_stride, op.wg_stride, op.wu_stride, op.h_stride, op.gate_stride, op.up_stride, op.k, op.n, op.act,
                      op.x, op.wg, op.wu, op.x_scale, op.g_scale, op.u_scale, op.bg, op.bu, op.h, op.gate, op.up};
    if (op.x_dtype == HG_F16) return gated_f16(a, op.h_dtype, stream);
    if (op.x_dtype == HG_BF16) return gated_bf16(a, op.h_dtype, stream);
    return gated_f8(a, op.h_dtype, stream);
}

size_t gated_backward_bytes(const hg_gated_grad &op) { return (size_t)gated_plan(op).bytes; }

hipError_t launch_gated_backward(const hg_gated_grad &op, void *workspace, hipStream_t stream) {
    // (one row has no stride)
    auto rows = [&](int64_t stride) { return op.m > 1 ? stride : 0; };
    const GatedGradArgs a{op.m, rows(op.dh_stride), rows(op.gate_stride), rows(op.up_stride), rows(op.x_stride), op.wg_stride,
                          op.wu_stride, rows(op.dx_stride), op.dwg_stride, op.dwu_stride, op.k, op.n, op.act, op.accumulate,
                          op.dw_dtype == HG_F32, op.dh, op.gate, op.up, op.x, op.wg, op.wu, op.dx, op.dwg, op.dwu, op.dbg, op.dbu};
    if (!a.dx && !a.dwg && !a.dbg) return hipSuccess;
    return op.dtype == HG_F16 ? gated_grad_run<f16>(op, a, (char *)workspace, stream)
                              : gated_grad_run<bf16>(op, a, (char *)workspace, stream);
}

}  // namespace res
}  // namespace hg
