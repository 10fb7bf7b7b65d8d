// What the gated blocks' kernels share: their arguments, and the gate's product and
// its gradients.
//
//   g = x Wg^T + bg,  u = x Wu^T + bu,  h = act(g) u
//   dg = dh u act'(g),  du = dh act(g)
#pragma once

#include "linear_common.h"

namespace hg {
namespace res {

struct GatedArgs {
    int64_t m, xs, gs, us, hs, ps, qs;  // strides: x, wg, wu, h, gate, up
    int k, n, act;
    const void *x, *wg, *wu;
    const float *x_scale, *g_scale, *u_scale, *bg, *bu;
    void *h, *gate, *up;
};
hipError_t gated_f16(const GatedArgs &a, int h_dtype, hipStream_t stream);
hipError_t gated_bf16(const GatedArgs &a, int h_dtype, hipStream_t stream);
hipError_t gated_f8(const GatedArgs &a, int h_dtype, hipStream_t stream);

struct GatedGradArgs {
    int64_t m, dhs, ps, qs, xs, gs, us, dxs, dgs, dus;  // strides: dh, gate, up, x, wg, wu, dx, dwg, dwu
    int k, n, act, accumulate, dw_f32;
    const void *dh, *gate, *up, *x, *wg, *wu;
    void *dx, *dwg, *dwu;
    float *dbg, *dbu;
};

// h of one hidden unit, in place of g.
template <int N>
__device__ __forceinline__ void gate_all(float (&g)[N], const float (&u)[N], int act) {
    activate_all(g, act);
#pragma unroll
    for (int j = 0; j < N; ++j) g[j] *= u[j];
}

// dg and du of one hidden unit.  The activation's value v = g p and slope share their
// logistic function p: SiLU's slope is p + v (1 - p), GELU's p + v (1 - p) d(2u)/dg.
template <int kAct>
__device__ __forceinline__ void gate_grad(float g, float u, float dh, float &dg, float &du) {
    if constexpr (kAct == HG_ACT_NONE) {
        dg = dh * u, du = dh * g;
    } else if constexpr (kAct == HG_ACT_RELU) {
        const bool on = !(g <= 0.f);  // (a NaN stays one)
        dg = on ? dh * u * (g != g ? g : 1.f) : 0.f, du = on ? dh * g : 0.f;
    } else {
        const float p = kAct == HG_ACT_SILU ? logistic(g) : gelu_logistic(g), value = mul0(g, p);
        // (1 - p is 0 where g is so large that value may be infinite)
        const float t = kAct == HG_ACT_SILU ? value : mul0(value, fmaf(g * g, 0.21406447f, 1.59576912f));
        dg = dh * u * (p + mul0(t, 1.f - p));
        du = dh * value;
    }
}
template <int N>
__device__ __forceinline__ void gate_grad_all(const float (&g)[N], const float (&u)[N], const float (&dh)[N], int act, float (&dg)[N],
                                              float (&du)[N]) {
    auto each = [&](auto kind) {
#pragma unroll
        for (int j = 0; j < N; ++j) gate_grad<decltype(kind)::value>(g[j], u[j], dh[j], dg[j], du[j]);
    };
    if (act == HG_ACT_NONE) each(std::integral_constant<int, HG_ACT_NONE>{});
    else if (act == HG_ACT_RELU) each(std::integral_constant<int, HG_ACT_RELU>{});
    else if (act == HG_ACT_SILU) each(std::integral_constant<int, HG_ACT_SILU>{});
    else each(std::integral_constant<int, HG_ACT_GELU_TANH>{});
}

}  // namespace res
}  // namespace hg
