// h = act(x Wg^T + bg) (x Wu^T + bu) and its backward: how the backward is cut, and
// the operands' types, each in a source of its own.
#include <math.h>

#include "gated_grad.h"

namespace hg {
namespace res {
namespace {

GatedGradPlan plan_of(const hg_gated_grad &op) {
    GatedGradPlan p{};
    p.units = op.n <= 64 ? 64 : 128;
    p.kt = op.k <= 64 ? 64 : op.k <= 128 ? 128 : 256;
    if (op.n < 8 || op.k < 8) p.units = p.kt = 64;  // rows shorter than a piece take the narrowest tiles
    p.kp = p.kt / 32;
    const bool one = op.n <= p.units && op.k <= p.kt && p.units * p.kt <= 128 * 128;
    p.together = one && op.dx && op.dwg && op.m > 0;
    // Fewer tiles of dx than half the CUs: the units in slices, for at the least of
    // stretches / slices * 3 us and what the slices' sums cost, written and joined.
    const int64_t tiles = div_up(op.m, 256) * div_up(op.k, p.kp * 32), stretches = div_up(op.n, 32);
    p.slices = 1;
    if (op.dx && op.m > 0 && !one && tiles < kCus / 2) {
        int64_t want = (int64_t)sqrt(3. * (double)stretches * 5e6 / (8. * (double)op.m * op.k));
        if (want > kCus / tiles) want = kCus / tiles;
        if (want > stretches / 2) want = stretches / 2;
        if (want > 1) p.slices = (int)want;
    }
    p.per = (int)div_up(stretches, p.slices);
    p.slices = (int)div_up(stretches, p.per);
    p.ny = (int)div_up(op.n, p.units), p.nz = (int)div_up(op.k, p.kt);
    // One workgroup a CU over all tiles, and no more than there are steps; fewer where a
    // workgroup's partial sums (written and joined at some 5 MB/us) cost more than the steps
    // (2 us each) it saves: at the least of steps / parts * 2 + parts * its partials.
    const int64_t steps = div_up(op.m, gate_rows(p.units, p.kt));
    const double partial_us = (double)p.ny * p.nz * 2 * p.units * p.kt * 8 / 5e6;
    int64_t parts = kCus / (p.ny * p.nz);
    const int64_t worth = (int64_t)sqrt(2. * (double)steps / partial_us);
    if (parts > worth) parts = worth;
    if (parts > steps) parts = steps;
    p.parts = (int)(parts < 1 ? 1 : parts);
    if (!op.dwg) p.nz = 1;  // the biases' gradients need one column of tiles
    const size_t tile = 2 * (size_t)p.units;
    if (op.m > 0 && p.parts > 1)
        p.bytes = ((op.dwg ? (size_t)p.ny * p.nz * tile * p.kt : 0) + (op.dbg ? (size_t)p.ny * tile : 0)) * p.parts * sizeof(float);
    if (p.slices > 1) {
        p.dx_at = (p.bytes + 255) / 256 * 256;
        p.bytes = p.dx_at + (size_t)p.slices * op.m * op.k * sizeof(float);
    }
    return p;
}

}  // namespace

hipError_t launch_gated_forward(const hg_gated &op, hipStream_t stream) {
    const GatedArgs a{op.m, op.x_stride, op.wg_stride, op.wu_stride, op.h_stride, op.gate_stride, op.up_stride, op.k, op.n, op.act,
                      op.x, op.wg, op.wu, op.x_scale, op.g_scale, op.u_scale, op.bg, op.bu, op.h, op.gate, op.up};
    if (op.x_dtype == HG_F16) return gated_f16(a, op.h_dtype, stream);
    if (op.x_dtype == HG_BF16) return gated_bf16(a, op.h_dtype, stream);
    return gated_f8(a, op.h_dtype, stream);
}

size_t gated_backward_bytes(const hg_gated_grad &op) { return plan_of(op).bytes; }

hipError_t launch_gated_backward(const hg_gated_grad &op, void *workspace, hipStream_t stream) {
    // (one row has no stride; the kernels' 32-bit offsets hold those of more)
    auto rows = [&](int64_t stride) { return op.m > 1 ? stride : 0; };
    const GatedGradArgs a{op.m, rows(op.dh_stride), rows(op.gate_stride), rows(op.up_stride), rows(op.x_stride), op.wg_stride,
                          op.wu_stride, rows(op.dx_stride), op.dwg_stride, op.dwu_stride, op.k, op.n, op.act, op.accumulate,
                          op.dw_dtype == HG_F32, op.dh, op.gate, op.up, op.x, op.wg, op.wu, op.dx, op.dwg, op.dwu, op.dbg, op.dbu};
    if (!a.dx && !a.dwg && !a.dbg) return hipSuccess;
    const auto run = op.dtype == HG_F16 ? gated_grad_f16 : gated_grad_bf16;
    return run(a, plan_of(op), (float *)workspace, stream);
}

}  // namespace res
}  // namespace hg
