// What the norms' kernels share: reductions over a row's lanes, the scale of 8-bit
// rows, and the join of the weights' partial gradients.
#pragma once

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

// dw = (dw +) the partial rows' sum: 16 columns a workgroup, 64 threads share the
// rows of each, and their sums are added in order, 16 and then four.  Columns from
// `split` on go to db.
__global__ __launch_bounds__(1024) void dw_join_kernel(const float *part, int rows, int c, float *dw, int split, float *db,
                                                       int accumulate) {
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
        float *const to = col < split ? dw + col : db + (col - split);
        *to = accumulate ? *to + t : t;
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

}  // namespace
}  // namespace res
}  // namespace hg
