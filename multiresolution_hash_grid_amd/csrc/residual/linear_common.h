// What the linear kernels share: matrix-core fragments, the activations and
// their slopes, and the upstream gradient through the activation.
//
// A fragment is 16 bytes a lane: lane l holds, of row l % 16 of its operand,
// the 16-byte piece l / 16 of a 64-byte stretch of the contraction (32 binary16
// or bfloat16 values, 64 8-bit ones).  Both operands cut the stretch alike, so
// the order inside it does not matter.
#pragma once

#include "device_types.h"

namespace hg {
namespace res {

typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <typename T>
constexpr int kStretch = 64 / (int)sizeof(T);  // elements of a row in a fragment step
template <typename T>
constexpr int kPiece = 16 / (int)sizeof(T);    // elements of a lane

// 16 8-bit values as binary16, which holds every one of them exactly.  The
// matrix cores' own 8-bit products sum with the smaller terms cut at about
// 2^-14 of a step's largest (128 products of random e4m3 codes against their exact
// sum: errors up to 8e-5 of sum |x w|, alike for the 32- and the 128-deep
// instruction; fp32 sums of 128 stay below 8e-6), so 8-bit operands are widened where
// they enter a product and their sums are fp32 like the others'.
struct Widened {
    u32x4 lo, hi;
};
__device__ __forceinline__ Widened widen(u32x4 v) {
    Widened w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        w.lo[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[i], 1.f, false));
        w.lo[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[i], 1.f, true));
        w.hi[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 + i], 1.f, false));
        w.hi[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v[2 + i], 1.f, true));
    }
    return w;
}

template <typename T>
__device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 acc) {
    if constexpr (__is_same(T, bf16))
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), acc, 0, 0, 0);
}

// acc[r] += sum_k a[row = 4 (lane / 16) + r][k] b[row = lane % 16][k], fp32 sums.
template <typename T>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 acc) {
    if constexpr (sizeof(T) == 1) {
        const Widened x = widen(a), y = widen(b);
        return mma16<f16>(x.hi, y.hi, mma16<f16>(x.lo, y.lo, acc));
    } else {
        return mma16<T>(a, b, acc);
    }
}

// The first piece of a row of fewer values than a piece, zeros past it; the loads
// do not wait for each other.
template <typename T>
__device__ __forceinline__ u32x4 load_short(const T *row, int length) {
    T t[kPiece<T>];
#pragma unroll
    for (int j = 0; j < kPiece<T>; ++j) t[j] = row[j < length ? j : length - 1];
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < kPiece<T>; ++j) {
        uint32_t bits;
        if constexpr (sizeof(T) == 2) bits = __builtin_bit_cast(uint16_t, t[j]);
        else bits = t[j].bits;
        constexpr int per = 4 / (int)sizeof(T);
        if (j < length) v[j / per] |= bits << (8 * (int)sizeof(T) * (j % per));
    }
    return v;
}

// A row cut into pieces without branches, for rows of at least a piece: the
// last piece of a row whose length is no multiple of a piece is read so that
// it ends with the row, and what belongs to the piece before it (or, for
// pieces past the row, all of it) is masked to zero.  Both operands are cut
// alike, so products meet their partners.
template <typename T>
struct Cut {
    int64_t at;   // first element of the piece as it is read
    u32x4 mask;
};
template <typename T>
__device__ __forceinline__ Cut<T> cut_piece(int k, int length) {
    const int have = length - k < 0 ? 0 : length - k < kPiece<T> ? length - k : kPiece<T>;
    Cut<T> c;
    c.at = have == kPiece<T> ? k : length - kPiece<T>;
    const int drop = (kPiece<T> - have) * (int)sizeof(T);  // bytes at the front
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int b = drop - 4 * j;
        c.mask[j] = b >= 4 ? 0u : b <= 0 ? ~0u : ~0u << (8 * b);
    }
    return c;
}

// 1 / (1 + 2^t).  The logistic function of z is that of t = -log2(e) z; 2^t overflows to infinity for very negative z, whose
// reciprocal is the right 0.
__device__ __forceinline__ float half_of(float t) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(t)); }
__device__ __forceinline__ float logistic(float z) { return half_of(-1.44269504f * z); }
// The logistic of 2 u, u = sqrt(2 / pi) (z + 0.044715 z^3), constants folded:
// t = -log2(e) 2 u = z (-2.3022082 - 0.10294324 z^2).
__device__ __forceinline__ float gelu_logistic(float z) { return half_of(z * fmaf(z * z, -0.10294324f, -2.3022082f)); }

// A product in which 0 times anything is 0 (v_mul_legacy_f32): an infinite z
// meets a logistic of 0 in both activations and their slopes, and 0 is the limit.
// A NaN z makes the other factor NaN too and stays.
__device__ float fmul_legacy(float a, float b) __asm("llvm.amdgcn.fmul.legacy");
__device__ __forceinline__ float mul0(float a, float b) { return fmul_legacy(a, b); }

// act(z).  GELU is the tanh form: 0.5 z (1 + tanh u) = z logistic(2 u), with
// u = sqrt(2 / pi) (z + 0.044715 z^3).
__device__ __forceinline__ float activate(float z, int act) {
    if (act == HG_ACT_RELU) return z > 0.f ? z : z != z ? z : 0.f;
    if (act == HG_ACT_SILU) return mul0(z, logistic(z));
    if (act == HG_ACT_GELU_TANH) return mul0(z, gelu_logistic(z));
    return z;
}

// Several of them behind one branch.
template <int N>
__device__ __forceinline__ void activate_all(float (&z)[N], int act) {
    if (act == HG_ACT_RELU)
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = activate(z[j], HG_ACT_RELU);
    else if (act == HG_ACT_SILU)
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = activate(z[j], HG_ACT_SILU);
    else if (act == HG_ACT_GELU_TANH)
#pragma unroll
        for (int j = 0; j < N; ++j) z[j] = activate(z[j], HG_ACT_GELU_TANH);
}

// d act / dz.
__device__ __forceinline__ float slope(float z, int act) {
    if (act == HG_ACT_RELU) return z > 0.f ? 1.f : z != z ? z : 0.f;
    if (act == HG_ACT_SILU) {
        const float p = logistic(z);
        return mul0(p, 1.f + mul0(z, 1.f - p));
    }
    if (act == HG_ACT_GELU_TANH) {
        const float p = gelu_logistic(z);
        return mul0(p, 1.f + mul0(z * fmaf(z * z, 0.21406447f, 1.59576912f), 1.f - p));
    }
    return 1.f;
}

struct FwdArgs {
    int64_t m, xs, ws, rs, ys, ps;
    int k, n, act;
    const void *x, *w, *r;
    const float *x_scale, *w_scale, *bias;
    void *y, *pre;
};
hipError_t linear_f16(const FwdArgs &a, int y_dtype, hipStream_t stream);
hipError_t linear_bf16(const FwdArgs &a, int y_dtype, hipStream_t stream);
hipError_t linear_f8(const FwdArgs &a, int y_dtype, hipStream_t stream);

}  // namespace res
}  // namespace hg
