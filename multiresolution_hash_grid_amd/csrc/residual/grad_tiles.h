// What the backwards' kernels share: 16-bit tiles in LDS that are read as rows and,
// transposed, as columns, and pieces of rows on their way into them.
#pragma once

#include "linear_common.h"

namespace hg {
namespace res {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// A 16-bit tile in LDS, [rows][C], its 16-byte pieces permuted so that 256 bytes
// at a time come from 64 different banks in both kinds of read: one piece of 16
// rows, and (transposed) 32 bytes of rows r .. r + 3 and r + 8 .. r + 11.
template <int C>
__device__ __forceinline__ int tile_at(int row, int piece) {
    const int turn = C == 64 ? (row & 2) | ((row >> 1) & 4) | ((row >> 2) & 1)
                             : ((row & 3) << 1) | ((row >> 2) & 1) | (row & 8);
    return row * (C * 2) + ((piece ^ turn) << 4);
}

// The fragment of columns 16 q .. of a tile's rows m .. m + 31, transposed: lane
// (i, g) gets column i, rows m + 8 g .. m + 8 g + 7.  The transposing read hands
// lane i of 16 the i-th column of four rows of 16 whose 8-byte parts the lanes'
// addresses name, four lanes a row (found by reading a tile of known values).
template <int C>
__device__ __forceinline__ u32x4 tile_columns(char *tile, int m, int q, int lane) {
    const int i = lane & 15, row = m + (lane >> 4) * 8 + (i >> 2);
    union {
        s16x4 h[2];
        u32x4 v;
    } r;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        r.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_s16x4 *)(tile + tile_at<C>(row + 4 * h, 2 * q + ((i >> 1) & 1)) + (i & 1) * 8));
    return r.v;
}

// The piece at p; kShort: rows may be shorter than a piece (the narrowest tiles').
template <bool kShort, typename T>
__device__ __forceinline__ u32x4 load_columns(const T *p, Columns c, int width) {
    if (!kShort || width >= 8) return load_loose<u32x4>(p);
    return c.drop ? u32x4{0, 0, 0, 0} : load_short(p, width);
}

template <typename T>
__device__ __forceinline__ u32x4 pack8(const float (&v)[8]) {
    typedef T T8 __attribute__((ext_vector_type(8)));
    T8 p;
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = (T)v[j];
    return __builtin_bit_cast(u32x4, p);
}

// A cut piece moved so that its first slot that counts is slot 0.
__device__ __forceinline__ u32x4 shifted(u32x4 v, int drop) {
    if (drop & 4) v = u32x4{v[2], v[3], 0, 0};
    if (drop & 2) v = u32x4{v[1], v[2], v[3], 0};
    if (drop & 1) v = u32x4{v[0] >> 16 | v[1] << 16, v[1] >> 16 | v[2] << 16, v[2] >> 16 | v[3] << 16, v[3] >> 16};
    return v;
}

}  // namespace
}  // namespace res
}  // namespace hg
