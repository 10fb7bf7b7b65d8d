// Element types and lane helpers of the residual head's kernels (gfx950).
#pragma once

#include "residual_internal.h"

namespace hg {
namespace res {

typedef _Float16 f16;
typedef __bf16 bf16;
struct f8 {  // OCP e4m3: 4 exponent bits (bias 7), 3 mantissa bits, largest value 448
    uint8_t bits;
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// Vectors at any alignment the element type allows: global memory takes wide
// accesses at every address here, so rows of odd strides load as wide as
// aligned ones.
template <typename V>
struct __attribute__((packed, aligned(1))) Loose {
    V v;
};
template <typename V>
__device__ __forceinline__ V load_loose(const void *p) {
    return reinterpret_cast<const Loose<V> *>(p)->v;
}
template <typename V>
__device__ __forceinline__ void store_loose(void *p, V v) {
    reinterpret_cast<Loose<V> *>(p)->v = v;
}

// The columns of one piece of 8 of a row of `width` columns.  The piece that the
// row's end cuts is read so that it ends with the row; its first `drop` slots
// belong to the piece before it, and all 8 of a piece past the row do not count.
// So every piece is one wide access, without branches, and the compiler can count
// the loads in flight.  Slot j is column at + j.  Rows of less than 8 columns are
// read value by value.
struct Columns {
    int at, drop;
};
__device__ __forceinline__ Columns columns_of(int nominal, int width) {
    if (width < 8) return {0, nominal < width ? 0 : 8};
    const int at = nominal < width - 8 ? nominal : width - 8;
    return {at, nominal - at};
}
// The column of a slot, or -1 of one that does not count.
__device__ __forceinline__ int column_of(int slot, int width) {
    const Columns c = columns_of(slot / 8 * 8, width);
    const int j = slot % 8;
    return j < c.drop || c.at + j >= width ? -1 : c.at + j;
}

// A row's piece as floats.  kShort: rows may have less than 8 columns; their loads
// do not wait for each other either, and what is past them is zero.
template <bool kShort, typename T>
__device__ __forceinline__ void load8(const T *row, Columns c, int width, float (&v)[8]) {
    if (!kShort || width >= 8) {
        if constexpr (sizeof(T) == 2) {
            typedef T T8 __attribute__((ext_vector_type(8)));
            const T8 a = load_loose<T8>(row + c.at);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (float)a[j];
        } else {
            const f32x4 a = load_loose<f32x4>(row + c.at), b = load_loose<f32x4>(row + c.at + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = a[j], v[4 + j] = b[j];
        }
        return;
    }
    T t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) t[j] = row[j < width ? j : width - 1];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < width && c.drop == 0 ? (float)t[j] : 0.f;
}

// Stores a row's piece, each value rounded to nearest even.  The slots that the
// piece before holds too are written twice, with the same values.
template <bool kShort, typename T>
__device__ __forceinline__ void store8(T *row, Columns c, int width, const float (&v)[8]) {
    if (c.drop >= 8) return;
    T *const p = row + c.at;
    if constexpr (sizeof(T) == 2) {
        typedef T T8 __attribute__((ext_vector_type(8)));
        T8 a;
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = (T)v[j];
        if (!kShort || width >= 8) {
            store_loose<T8>(p, a);
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < width) p[j] = a[j];
    } else if constexpr (sizeof(T) == 4) {
        if (!kShort || width >= 8) {
            store_loose<f32x4>(p, f32x4{v[0], v[1], v[2], v[3]});
            store_loose<f32x4>(p + 4, f32x4{v[4], v[5], v[6], v[7]});
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < width) p[j] = v[j];
    } else {
        int lo = 0, hi = 0;
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
        if (!kShort || width >= 8) {
            store_loose<u32x2>(p, u32x2{(uint32_t)lo, (uint32_t)hi});
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < width) p[j].bits = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
    }
}

// N values as they lie in memory, to be held until they are used; of those past
// `left` nothing is said.
template <int N, typename T>
struct Held {
    T v __attribute__((ext_vector_type(N)));
};
template <int N, typename T>
__device__ __forceinline__ Held<N, T> hold(const T *p, int left) {
    typedef T V __attribute__((ext_vector_type(N)));
    Held<N, T> h;
    if (left >= N) {
        h.v = load_loose<V>(p);
    } else if (left > 0) {  // loads that do not wait for each other
#pragma unroll
        for (int j = 0; j < N; ++j) h.v[j] = p[j < left ? j : left - 1];
    }
    return h;
}

template <int N, typename T>
__device__ __forceinline__ Held<N, T> rounded(const float (&v)[N]) {
    Held<N, T> h;
#pragma unroll
    for (int j = 0; j < N; ++j) h.v[j] = (T)v[j];
    return h;
}
template <int N, typename T>
__device__ __forceinline__ void put(T *p, int left, Held<N, T> h) {
    if (left >= N) {
        store_loose(p, h.v);
        return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < left) p[j] = h.v[j];
}

// LDS written by other lanes of the wave may be read after this, and what they
// read overwritten.  The hardware keeps a wave's LDS accesses in order; this keeps
// the compiler from moving them.
__device__ __forceinline__ void wave_exchange() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Sum over aligned groups of G lanes, in every lane of the group.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int o = 1; o < G; o <<= 1) v += __shfl_xor(v, o, 64);
    return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int o = 1; o < G; o <<= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}

// Largest of 64 lanes' words, in a scalar register: four steps within rows of
// 16 lanes, two row broadcasts, lane 63.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t x) {
    auto step = [&](auto ctrl, auto rows) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, ctrl.value, rows.value, 0xF, false);
        x = o > x ? o : x;
    };
    step(std::integral_constant<int, 0xB1>{}, std::integral_constant<int, 0xF>{});   // lane ^ 1
    step(std::integral_constant<int, 0x4E>{}, std::integral_constant<int, 0xF>{});   // lane ^ 2
    step(std::integral_constant<int, 0x141>{}, std::integral_constant<int, 0xF>{});  // mirrored half rows
    step(std::integral_constant<int, 0x140>{}, std::integral_constant<int, 0xF>{});  // mirrored rows
    step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});  // row 0 -> 1, row 2 -> 3
    step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});  // row 1 -> 2 and 3
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

}  // namespace res
}  // namespace hg
