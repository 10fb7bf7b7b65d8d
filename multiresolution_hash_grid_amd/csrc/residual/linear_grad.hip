// Backward of the linear layer: how it is cut, and the operands' types, each in
// a source of its own.
#include "linear_grad.h"

namespace hg {
namespace res {
namespace {

int tile_of(int width) { return width <= 64 ? 64 : width <= 128 ? 128 : 256; }

GradPlan plan(const hg_linear_grad &op) {
    GradPlan p;
    p.nt = tile_of(op.n), p.kt = tile_of(op.k);
    p.ny = (int)div_up(op.n, p.nt), p.nz = (int)div_up(op.k, p.kt);
    p.fused = op.dx && p.ny == 1 && p.nz == 1;
    // One workgroup a CU over all tiles (two of the smallest tile, whose registers
    // and LDS leave room), and no more than there are steps; of two steps each where
    // that leaves work for half the CUs: half the partials to write and join (8192 x
    // 256 x 256 39 -> 35 us, 65536 x 64 x 64 19.6 -> 17.8; with fewer workgroups the
    // second step costs more: 8192 x 64 x 64 11.1 -> 12.8, 1000 x 256 x 256 21.7 -> 22.4).
    const int64_t steps = div_up(op.m, grad_rows(p.nt, p.kt));
    int64_t parts = kCus * (p.nt * p.kt == 64 * 64 ? 2 : 1) / (p.ny * p.nz);
    if (parts < 1) parts = 1;
    const int64_t most = steps >= kCus ? div_up(steps, 2) : steps;
    if (parts > most) parts = most;
    p.parts = (int)(parts < 1 ? 1 : parts);
    if (!op.dw) p.nz = 1;  // dz and db need one column of tiles
    const size_t tiles = (size_t)p.ny * p.nz * p.nt * p.kt;
    size_t at = p.parts == 1 ? 0 : ((op.dw ? tiles : 0) + (op.db ? (size_t)p.ny * p.nt : 0)) * p.parts * sizeof(float);
    p.dz_at = p.wt_at = at;
    if (op.dx && !p.fused) {
        auto up = [](size_t v) { return (v + 255) / 256 * 256; };
        p.dz_at = up(at);
        p.wt_at = up(p.dz_at + (size_t)op.m * op.n * 2);
        at = p.wt_at + (size_t)op.k * op.n * 2;
    }
    p.bytes = op.m > 0 ? at : 0;
    return p;
}

}  // namespace

size_t linear_backward_bytes(const hg_linear_grad &op) { return plan(op).bytes; }

hipError_t launch_linear_backward(const hg_linear_grad &op, void *workspace, hipStream_t stream) {
    // (one row has no stride; the kernels' 32-bit offsets hold those of more)
    auto rows = [&](int64_t stride) { return op.m > 1 ? stride : 0; };
    const GradArgs a{op.m, rows(op.dy_stride), rows(op.pre_stride), rows(op.x_stride), op.w_stride, rows(op.dx_stride), op.dw_stride,
                     op.k, op.n, op.act, op.accumulate, op.dw_dtype == HG_F32, op.dy, op.pre, op.x, op.w, op.dx, op.dw, op.db};
    if (!a.dx && !a.dw && !a.db) return hipSuccess;
    const auto run = op.dtype == HG_F16 ? linear_grad_f16 : linear_grad_bf16;
    return run(a, op.dy_dtype == HG_F32, plan(op), (char *)workspace, stream);
}

}  // namespace res
}  // namespace hg
