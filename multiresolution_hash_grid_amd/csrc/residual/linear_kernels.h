// Kernels of y = act(x W^T + b) + r for one pair of types; the sources that
// include this instantiate one operand type each, so that they build at once.
#pragma once

#include <math.h>

#include "linear_common.h"

namespace hg {
namespace res {
namespace {

// Few rows.  A workgroup computes 16 rows by 16 outputs; its four waves share
// the contraction and add their sums in LDS.  Both operands come straight from
// memory as fragments.  Bound by one chain of load, product and join: 1 x 96 x 64
// takes 2 us on the GPU, and a call of it 7 us of the host's time.
template <typename T, typename Y>
__global__ __launch_bounds__(256) void linear_tile_kernel(const FwdArgs a) {
    __shared__ f32x4 sums[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m0 = (int64_t)blockIdx.y * 16;
    const int n0 = blockIdx.x * 16;
    const int64_t xm = m0 + (lane & 15) < a.m ? m0 + (lane & 15) : a.m - 1;
    const int wn = n0 + (lane & 15) < a.n ? n0 + (lane & 15) : a.n - 1;
    const T *x = (const T *)a.x + xm * a.xs, *w = (const T *)a.w + (int64_t)wn * a.ws;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    const int group = lane >> 4;
    if (a.k < kPiece<T>) {
        if (wave == 0) {
            const u32x4 none = {0, 0, 0, 0};
            acc = mma<T>(group ? none : load_short(w, a.k), group ? none : load_short(x, a.k), acc);
        }
    } else {
        for (int k0 = wave * kStretch<T>; k0 < a.k; k0 += 4 * kStretch<T>) {
            const Cut<T> c = cut_piece<T>(k0 + group * kPiece<T>, a.k);
            acc = mma<T>(load_loose<u32x4>(w + c.at) & c.mask, load_loose<u32x4>(x + c.at) & c.mask, acc);
        }
    }
    sums[wave][lane] = acc;
    __syncthreads();
    // thread t: row t / 16, output t % 16; it lies in lane (output / 4) * 16 + row, word output % 4
    const int row = threadIdx.x >> 4, col = threadIdx.x & 15;
    const int64_t m = m0 + row;
    const int n = n0 + col;
    if (m >= a.m || n >= a.n) return;
    float z = 0.f;
    for (int i = 0; i < 4; ++i) z += sums[i][(col >> 2) * 16 + row][col & 3];
    if constexpr (sizeof(T) == 1) z = z * a.x_scale[m] * a.w_scale[n];
    if (a.bias) z += a.bias[n];
    if constexpr (sizeof(T) == 2)
        if (a.pre) ((T *)a.pre)[m * a.ps + n] = (T)z;
    float y = activate(z, a.act);
    if (a.r) y += (float)((const Y *)a.r)[m * a.rs + n];
    ((Y *)a.y)[m * a.ys + n] = (Y)y;
}

// A wave's buffer of 16 rows by 512 bytes: 8 values of 16 or 32 bits are one or
// two pieces of 16 bytes, permuted in their row by the row's number.
constexpr int kStageBytes = 16 * 512;
template <typename V>
__device__ __forceinline__ void stage_put(char *stage, int row, int eight, Held<8, V> h) {
    if constexpr (sizeof(V) == 2) {
        *(u32x4 *)(stage + row * 512 + ((eight ^ row) << 4)) = __builtin_bit_cast(u32x4, h.v);
    } else {
        f32x4 lo, hi;
#pragma unroll
        for (int j = 0; j < 4; ++j) lo[j] = h.v[j], hi[j] = h.v[4 + j];
        *(f32x4 *)(stage + row * 512 + (((2 * eight) ^ row) << 4)) = lo;
        *(f32x4 *)(stage + row * 512 + (((2 * eight + 1) ^ row) << 4)) = hi;
    }
}
// The first `pairs` * 32 values of each row to columns n .. of rows m1 ..; only
// rows below `rows` and columns below `width` exist.
template <typename V>
__device__ __forceinline__ void stage_store(V *y, int64_t stride, int64_t m1, int64_t rows, int n, int width, const char *stage,
                                            int pairs, int lane) {
    constexpr int per = 16 / (int)sizeof(V);  // values of a piece
    const int pieces = pairs * 32 / per;      // of a row: a multiple of 4
    wave_exchange();
#pragma unroll 1
    for (int at = lane; at < pieces * 16; at += 64) {
        const int row = at / pieces, c = at - row * pieces;
        typedef V VP __attribute__((ext_vector_type(16 / (int)sizeof(V))));
        const Held<per, V> h = {__builtin_bit_cast(VP, *(const u32x4 *)(stage + row * 512 + ((c ^ row) << 4)))};
        if (m1 + row < rows) put(y + (m1 + row) * stride + n + c * per, width - n - c * per, h);
    }
    wave_exchange();
}

// Many rows, a weight that fits LDS in a few slices.  A workgroup keeps its
// slice of W in LDS for good, in fragment order (a wave reads 1 KB in a row,
// without conflicts; 8-bit weights are widened once, here), and its waves walk
// row tiles of 16 rows on their own: a tile's rows go straight from memory
// into registers as fragments, all of the contraction at once, and each set of
// FR 16-output fragments is finished -- bias, activation, residual, rounding --
// before the next is begun.  No barrier after the start: the waves of a CU hide
// each other's loads.
// A pair of fragments deals its 32 outputs so that a lane has 8 consecutive ones
// of one row: row i of fragment h is output (i / 4) * 8 + h * 4 + i % 4.  A set of
// two pairs reads and writes whole 128-byte lines (16-bit outputs): with one pair
// a set, half lines left L2 before their other halves came, and 1.35 times the
// bytes were written and 1.45 times read (2^20 x 256 x 256).  The outputs of GS
// sets are held, rounded, and stored together: rows of 512 bytes written in runs
// of 128, 256 and 512 bytes go to memory at 3.6, 4.7 and 5.5 TB/s.
// kStage: where the weights leave LDS room, 512 bytes of each row are collected in
// a buffer of the wave's own, pieces permuted against bank conflicts, and stored
// 1 KB at a time in memory order (2^18 x 32 x 256 with z kept: 74 -> 60 us).
// Slices of W are workgroups next to each other on one XCD that walk the same
// rows, so x comes from HBM once.  A weight of more slices than an XCD's share of
// the workgroups has fewer than 8 walkers a slice (1, 2 or 4): each keeps to its
// XCDs, and the slices go around all of them.
// Bound by memory, and at 8 bits by what a wave does (widening, GELU, residual)
// between its loads, eight waves a CU: the VALU is 42 % busy, the matrix units 28.
// 2^20 x 256 x 256 bf16 with SiLU and residual: 300-309 us, 5.2-5.4 TB/s; 2^18 x 32 x
// 256 f16 with z kept: 60 us, 4.7 TB/s; 10^5 x 256 x 4: 10.8 us; 2^18 x 512 x 512 e4m3
// with GELU and residual: 198-206 us, 3.3 TB/s.
// kCut: 0 the contraction is whole fragments; 1 its last fragment is cut; 2 it
// is shorter than a piece.
template <typename T, typename Y, int KU, int RF, int FR, int GS, int kCut, bool kStage>
__global__ __launch_bounds__(RF == 1 ? 1024 : 512) void linear_stream_kernel(const FwdArgs a, int slices, int slice_n) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int kHalves = sizeof(T) == 1 ? 2 : 1;
    constexpr int kPairs = FR == 1 ? 1 : FR / 2, kOut = FR == 1 ? 4 : 8;  // pairs of a set; consecutive outputs of a lane
    constexpr bool kWide = sizeof(T) == 1 && KU <= 4;       // 8-bit rows are widened as they come; longer ones at each use
    u32x4 *const wl = (u32x4 *)lds;
    const int waves = blockDim.x >> 6;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row16 = lane & 15, group = lane >> 4;
    // workgroups b, b + 8, b + 16, ... share an XCD
    const int xcd = blockIdx.x & 7, in_xcd = blockIdx.x >> 3, walkers = gridDim.x / slices;
    const int n0 = (walkers < 8 ? blockIdx.x / walkers : in_xcd % slices) * slice_n;
    const int walker = walkers < 8 ? xcd & (walkers - 1) : in_xcd / slices * 8 + xcd;
    const int nn = a.n - n0 < slice_n ? a.n - n0 : slice_n;
    const int sets = (nn + 16 * FR - 1) / (16 * FR);
    float *const bias = (float *)(lds + (size_t)(slice_n / 16) * KU * kHalves * 1024), *const wsc = bias + slice_n;
    char *const stage = (char *)(wsc + slice_n) + wave * kStageBytes;

    // The last fragment's piece of this lane.
    const Cut<T> last = cut_piece<T>((KU - 1) * kStretch<T> + group * kPiece<T>, a.k);
    auto piece = [&](const T *row, int u) -> u32x4 {
        if constexpr (kCut == 2) return group ? u32x4{0, 0, 0, 0} : load_short(row, a.k);
        if (kCut == 1 && u == KU - 1) return load_loose<u32x4>(row + last.at) & last.mask;
        return load_loose<u32x4>(row + group * kPiece<T> + u * kStretch<T>);
    };

    for (int b = wave; b < sets * FR; b += waves) {
        const int n = FR == 1 ? row16 : (b >> 1) * 32 + (row16 >> 2) * 8 + (b & 1) * 4 + (row16 & 3);
        const T *w = (const T *)a.w + (int64_t)(n0 + (n < nn ? n : nn - 1)) * a.ws;
#pragma unroll
        for (int u = 0; u < KU; ++u) {
            if constexpr (sizeof(T) == 1) {
                const Widened v = widen(piece(w, u));
                wl[((b * KU + u) * 2) * 64 + lane] = v.lo;
                wl[((b * KU + u) * 2 + 1) * 64 + lane] = v.hi;
            } else {
                wl[(b * KU + u) * 64 + lane] = piece(w, u);
            }
        }
    }
    for (int n = threadIdx.x; n < slice_n; n += blockDim.x) {
        bias[n] = a.bias && n < nn ? a.bias[n0 + n] : 0.f;
        if constexpr (sizeof(T) == 1) wsc[n] = n < nn ? a.w_scale[n0 + n] : 0.f;
    }
    __syncthreads();

    const int64_t tiles = (a.m + RF * 16 - 1) / (RF * 16);
    for (int64_t tile = (int64_t)wave * walkers + walker; tile < tiles; tile += (int64_t)waves * walkers) {
        const int64_t m0 = tile * (RF * 16) + row16;
        u32x4 x[RF][KU * (kWide ? 2 : 1)];
        float xsc[RF];
#pragma unroll
        for (int r = 0; r < RF; ++r) {
            const int64_t m = m0 + r * 16 < a.m ? m0 + r * 16 : a.m - 1;
#pragma unroll
            for (int u = 0; u < KU; ++u) x[r][u] = piece((const T *)a.x + m * a.xs, u);
            if constexpr (sizeof(T) == 1) xsc[r] = a.x_scale[m];
        }
        if constexpr (kWide)
#pragma unroll
            for (int r = 0; r < RF; ++r)
#pragma unroll
                for (int u = KU - 1; u >= 0; --u) {
                    const Widened v = widen(x[r][u]);
                    x[r][2 * u] = v.lo, x[r][2 * u + 1] = v.hi;
                }
        for (int s0 = 0; s0 < sets; s0 += GS) {
            Held<kOut, Y> y[RF][kStage ? 1 : GS][kPairs];
            typedef std::conditional_t<sizeof(T) == 1, f16, T> P;  // (8-bit operands keep no pre-activation)
            Held<kOut, P> pre[RF][GS][kPairs];
#pragma unroll
            for (int i = 0; i < GS; ++i) {
                const int s = s0 + i;
                if (s >= sets) break;
                const int n = s * 16 * FR + group * kOut;  // this lane's outputs: kOut from n, and from n + 32
                // The residual is asked for before the products.
                Held<kOut, Y> res[RF][kPairs];
                if (a.r)
#pragma unroll
                    for (int r = 0; r < RF; ++r) {
                        const int64_t m = m0 + r * 16 < a.m ? m0 + r * 16 : a.m - 1;
#pragma unroll
                        for (int q = 0; q < kPairs; ++q)
                            res[r][q] = hold<kOut>((const Y *)a.r + m * a.rs + n0 + n + q * 32, nn - n - q * 32);
                    }
                f32x4 acc[RF][FR];
#pragma unroll
                for (int f = 0; f < FR; ++f) {
                    // sums begin with the bias; 8-bit ones are scaled first
                    if constexpr (sizeof(T) == 1) acc[0][f] = f32x4{0.f, 0.f, 0.f, 0.f};
                    else acc[0][f] = *(const f32x4 *)(bias + n + (f >> 1) * 32 + (f & 1) * 4);
#pragma unroll
                    for (int r = 1; r < RF; ++r) acc[r][f] = acc[0][f];
                }
#pragma unroll
                for (int u = 0; u < KU; ++u) {
                    Widened xw[RF];
                    if constexpr (sizeof(T) == 1 && !kWide)
#pragma unroll
                        for (int r = 0; r < RF; ++r) {
                            asm volatile("" : "+v"(x[r][u]));  // widen here, not once before all sets: the registers are not there
                            xw[r] = widen(x[r][u]);
                        }
#pragma unroll
                    for (int f = 0; f < FR; ++f)
#pragma unroll
                        for (int h = 0; h < kHalves; ++h) {
                            const u32x4 w = wl[(((s * FR + f) * KU + u) * kHalves + h) * 64 + lane];
#pragma unroll
                            for (int r = 0; r < RF; ++r) {
                                u32x4 v;
                                if constexpr (sizeof(T) == 1 && !kWide) v = h ? xw[r].hi : xw[r].lo;
                                else v = x[r][u * kHalves + h];
                                acc[r][f] = mma16<T>(w, v, acc[r][f]);
                            }
                        }
                }
#pragma unroll
                for (int r = 0; r < RF; ++r)
#pragma unroll
                    for (int q = 0; q < kPairs; ++q) {
                        float z[kOut];
#pragma unroll
                        for (int j = 0; j < kOut; ++j) {
                            z[j] = acc[r][q * 2 + j / 4][j % 4];
                            if constexpr (sizeof(T) == 1) z[j] = fmaf(z[j] * xsc[r], wsc[n + q * 32 + j], bias[n + q * 32 + j]);
                        }
                        if constexpr (sizeof(T) == 2)
                            if (a.pre) pre[r][i][q] = rounded<kOut, T>(z);
                        activate_all(z, a.act);
                        if (a.r)
#pragma unroll
                            for (int j = 0; j < kOut; ++j) z[j] += (float)res[r][q].v[j];
                        if constexpr (kStage) stage_put(stage, row16, (i * kPairs + q) * 4 + group, rounded<kOut, Y>(z));
                        else y[r][i][q] = rounded<kOut, Y>(z);
                    }
            }
            if constexpr (kStage) {
                static_assert(RF == 1);
                const int count = (sets - s0 < GS ? sets - s0 : GS) * kPairs;  // pairs of this round
                const int64_t m1 = tile * 16;
                stage_store((Y *)a.y, a.ys, m1, a.m, n0 + s0 * 16 * FR, n0 + nn, stage, count, lane);
                if constexpr (sizeof(T) == 2)
                    if (a.pre) {
#pragma unroll
                        for (int q = 0; q < GS * kPairs; ++q)
                            if (q < count) stage_put(stage, row16, q * 4 + group, pre[0][q / kPairs][q % kPairs]);
                        stage_store((T *)a.pre, a.ps, m1, a.m, n0 + s0 * 16 * FR, n0 + nn, stage, count, lane);
                    }
            } else {
                const int at = n0 + s0 * 16 * FR + group * kOut, left = n0 + nn - at;
#pragma unroll
                for (int r = 0; r < RF; ++r) {
                    const int64_t m = m0 + r * 16;
                    if (m >= a.m) break;
                    if constexpr (sizeof(T) == 2)
                        if (a.pre)
#pragma unroll
                            for (int q = 0; q < GS * kPairs; ++q)
                                put((T *)a.pre + m * a.ps + at + q * 32, left - q * 32, pre[r][q / kPairs][q % kPairs]);
#pragma unroll
                    for (int q = 0; q < GS * kPairs; ++q)
                        put((Y *)a.y + m * a.ys + at + q * 32, left - q * 32, y[r][q / kPairs][q % kPairs]);
                }
            }
        }
    }
}

constexpr int kLdsBytes = 160 * 1024;
// LDS of one output's weights, bias and scale.
template <typename T, int KU>
constexpr int kWeightBytes = KU * 64 * (sizeof(T) == 1 ? 2 : 1) + 8;

// With few rows a workgroup mostly reads weights: a CU fetches some 14 KB/us that
// its own L1 misses, so 128 KB of weights take 9 us.  Slices of W cost their rows'
// x again: bytes W / s + s x / CUs are least at s = sqrt(n CUs / m).
inline int few_rows_slices(const FwdArgs &a) {
    const int most = (int)div_up(a.n, 64), want = (int)sqrt((double)a.n * kCus / (double)a.m);
    return want < most ? want : most;
}

template <typename T, typename Y, int KU, int RF, int FR, int GS, int kCut, bool kStage = false>
hipError_t stream_launch(const FwdArgs &a, hipStream_t stream) {
    const auto kernel = linear_stream_kernel<T, Y, KU, RF, FR, GS, kCut, kStage>;
    constexpr int per = kWeightBytes<T, KU>, set = 16 * FR;  // LDS bytes of an output; outputs of a set
    const int fit = kLdsBytes / per / set * set;
    int slices = (int)div_up(a.n, fit);
    if (FR == 4 && few_rows_slices(a) > slices) slices = few_rows_slices(a);
    const int slice_n = (int)div_up(div_up(a.n, slices), set) * set;
    slices = (int)div_up(a.n, slice_n);
    const int bytes = slice_n * per + (kStage ? 16 * kStageBytes : 0);
    if (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    // 16 waves a CU in one workgroup, or in two of eight where two slices fit its
    // LDS (three where the registers allow six waves a SIMD): they start and end
    // apart, and the last tiles are dealt more evenly.
    const int groups = RF == 2 || bytes > kLdsBytes / 2 ? 1 : KU > 1 || bytes > kLdsBytes / 3 ? 2 : 3;
    const int64_t tiles = div_up(a.m, RF * 16);
    int64_t walkers = kCus * groups / slices;  // workgroups that share the rows
    if (walkers > tiles) walkers = tiles;
    // Whole rounds over the XCDs; below 8 a power of two, and at least one (more slices
    // than workgroups are resident).  Always 8, each slice of W is brought in 8 times:
    // 512 x 512 x 32768 f16 104 us, 37 so; 4096 x 512 x 50304 410 and 343.
    walkers = walkers >= 8 ? div_up(walkers, 8) * 8 : walkers >= 4 ? 4 : walkers >= 2 ? 2 : 1;
    kernel<<<dim3((unsigned)(walkers * slices)), RF == 1 && groups == 1 ? 1024 : 512, bytes, stream>>>(a, slices, slice_n);
    return hipGetLastError();
}

template <typename T, typename Y, int KU, int kCut>
hipError_t stream_set(const FwdArgs &a, hipStream_t stream) {
    if (a.n <= 16) return stream_launch<T, Y, KU, 1, 1, 1, kCut>(a, stream);
    if (a.n <= 32) return stream_launch<T, Y, KU, 1, 2, 1, kCut>(a, stream);
    if (a.n <= 64) return stream_launch<T, Y, KU, 1, 4, 1, kCut>(a, stream);
    if constexpr (KU <= 4)  // rows of more than one set, weights beside 16 waves' buffers
        if (div_up(a.n, 64) * 64 * kWeightBytes<T, KU> <= kLdsBytes - 16 * kStageBytes)
            return stream_launch<T, Y, KU, 1, 4, sizeof(Y) == 4 ? 2 : 4, kCut, true>(a, stream);
    constexpr int GS = sizeof(Y) == 4 ? (KU <= 4 ? 2 : 1) : KU <= 12 ? 2 : 1;  // what the registers hold
    if constexpr (KU >= 5) return stream_launch<T, Y, KU, 2, 4, GS, kCut>(a, stream);
    return stream_launch<T, Y, KU, 1, 4, GS, kCut>(a, stream);
}

// Many rows, a contraction longer than a wave's registers hold, few outputs: W in
// LDS and a wave's own row tiles as above, and the rows come in chunks of KC
// fragments, the next chunk on its way while one is multiplied.  W's fragments are
// padded with zeros to whole chunks, and the rows' with zeros too (what is past a
// row need not be finite).
constexpr int kChunkFragments = 4;
constexpr int kLongSlices = 2;
template <typename T, typename Y, int FR>
__global__ __launch_bounds__(1024) void linear_long_kernel(const FwdArgs a, int slices, int units) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int KC = kChunkFragments, kHalves = sizeof(T) == 1 ? 2 : 1;
    constexpr int kPairs = FR == 1 ? 1 : FR / 2, kOut = FR == 1 ? 4 : 8;  // as in the stream kernel
    u32x4 *const wl = (u32x4 *)lds;
    const int chunks = (units + KC - 1) / KC, whole = chunks * KC;
    float *const bias = (float *)(lds + (size_t)FR * whole * kHalves * 1024), *const wsc = bias + 16 * FR;
    const int waves = blockDim.x >> 6;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row16 = lane & 15, group = lane >> 4;
    const int xcd = blockIdx.x & 7, in_xcd = blockIdx.x >> 3;
    const int n0 = (in_xcd % slices) * 16 * FR;
    const int walkers = (gridDim.x >> 3) / slices * 8, walker = in_xcd / slices * 8 + xcd;
    const int nn = a.n - n0 < 16 * FR ? a.n - n0 : 16 * FR;

    const Cut<T> last = cut_piece<T>((units - 1) * kStretch<T> + group * kPiece<T>, a.k);
    auto piece = [&](const T *row, int u) {  // fragments past the row read the last one
        return load_loose<u32x4>(row + (u < units - 1 ? u * kStretch<T> + group * kPiece<T> : last.at));
    };
    auto masked = [&](u32x4 v, int u) {
        return u < units - 1 ? v : u == units - 1 ? v & last.mask : u32x4{0, 0, 0, 0};
    };
    for (int b = wave; b < FR * whole; b += waves) {
        const int f = b / whole, u = b % whole;
        const int n = FR == 1 ? row16 : (f >> 1) * 32 + (row16 >> 2) * 8 + (f & 1) * 4 + (row16 & 3);
        const u32x4 v = masked(piece((const T *)a.w + (int64_t)(n0 + (n < nn ? n : nn - 1)) * a.ws, u), u);
        if constexpr (sizeof(T) == 1) {
            const Widened w = widen(v);
            wl[(b * 2) * 64 + lane] = w.lo;
            wl[(b * 2 + 1) * 64 + lane] = w.hi;
        } else {
            wl[b * 64 + lane] = v;
        }
    }
    for (int n = threadIdx.x; n < 16 * FR; n += blockDim.x) {
        bias[n] = a.bias && n < nn ? a.bias[n0 + n] : 0.f;
        if constexpr (sizeof(T) == 1) wsc[n] = n < nn ? a.w_scale[n0 + n] : 0.f;
    }
    __syncthreads();

    const int64_t tiles = (a.m + 15) / 16;
    for (int64_t tile = (int64_t)wave * walkers + walker; tile < tiles; tile += (int64_t)waves * walkers) {
        const int64_t m = tile * 16 + row16, mr = m < a.m ? m : a.m - 1;
        const T *const row = (const T *)a.x + mr * a.xs;
        const int n = group * kOut;  // this lane's outputs: kOut from n, and from n + 32
        f32x4 acc[FR];
#pragma unroll
        for (int f = 0; f < FR; ++f) {
            if constexpr (sizeof(T) == 1) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
            else acc[f] = *(const f32x4 *)(bias + n + (f >> 1) * 32 + (f & 1) * 4);
        }
        u32x4 even[KC], odd[KC];
        auto load = [&](u32x4(&x)[KC], int c) {
            if (c < chunks - 1) {
                const T *const p = row + group * kPiece<T> + c * KC * kStretch<T>;
#pragma unroll
                for (int j = 0; j < KC; ++j) x[j] = load_loose<u32x4>(p + j * kStretch<T>);
            } else {
#pragma unroll
                for (int j = 0; j < KC; ++j) x[j] = piece(row, c * KC + j);
            }
        };
        auto multiply = [&](u32x4(&x)[KC], int c) {
            if (c == chunks - 1)
#pragma unroll
                for (int j = 0; j < KC; ++j) x[j] = masked(x[j], c * KC + j);
#pragma unroll
            for (int j = 0; j < KC; ++j) {
                Widened xw;
                if constexpr (sizeof(T) == 1) xw = widen(x[j]);
#pragma unroll
                for (int f = 0; f < FR; ++f)
#pragma unroll
                    for (int h = 0; h < kHalves; ++h) {
                        u32x4 v;
                        if constexpr (sizeof(T) == 1) v = h ? xw.hi : xw.lo;
                        else v = x[j];
                        acc[f] = mma16<T>(wl[((f * whole + c * KC + j) * kHalves + h) * 64 + lane], v, acc[f]);
                    }
            }
        };
        load(even, 0);
        for (int c = 0; c < chunks; c += 2) {
            if (c + 1 < chunks) load(odd, c + 1);
            multiply(even, c);
            if (c + 1 >= chunks) break;
            if (c + 2 < chunks) load(even, c + 2);
            multiply(odd, c + 1);
        }
        float xsc = 1.f;
        if constexpr (sizeof(T) == 1) xsc = a.x_scale[mr];
#pragma unroll
        for (int q = 0; q < kPairs; ++q) {
            const int at = n + q * 32, left = nn - at;
            float z[kOut];
#pragma unroll
            for (int j = 0; j < kOut; ++j) {
                z[j] = acc[q * 2 + j / 4][j % 4];
                if constexpr (sizeof(T) == 1) z[j] = fmaf(z[j] * xsc, wsc[at + j], bias[at + j]);
            }
            if constexpr (sizeof(T) == 2)
                if (a.pre && m < a.m) put((T *)a.pre + m * a.ps + n0 + at, left, rounded<kOut, T>(z));
            activate_all(z, a.act);
            if (a.r) {
                const Held<kOut, Y> res = hold<kOut>((const Y *)a.r + mr * a.rs + n0 + at, left);
#pragma unroll
                for (int j = 0; j < kOut; ++j) z[j] += (float)res.v[j];
            }
            if (m < a.m) put((Y *)a.y + m * a.ys + n0 + at, left, rounded<kOut, Y>(z));
        }
    }
}

// LDS of linear_long_kernel with fr fragments of outputs.
template <typename T>
int long_bytes(const FwdArgs &a, int fr) {
    const int64_t chunks = div_up(div_up(a.k, kStretch<T>), kChunkFragments);
    const int64_t bytes = chunks * kChunkFragments * fr * (sizeof(T) == 1 ? 2048 : 1024) + 16 * fr * 8;
    return bytes > kLdsBytes ? 0 : (int)bytes;
}
template <typename T, typename Y, int FR>
hipError_t long_launch(const FwdArgs &a, hipStream_t stream) {
    const auto kernel = linear_long_kernel<T, Y, FR>;
    const int bytes = long_bytes<T>(a, FR), slices = (int)div_up(a.n, 16 * FR);
    if (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    const int64_t tiles = div_up(a.m, 16);
    int64_t walkers = kCus / slices;
    if (walkers > tiles) walkers = tiles;
    walkers = div_up(walkers, 8) * 8;
    kernel<<<dim3((unsigned)(walkers * slices)), 1024, bytes, stream>>>(a, slices, (int)div_up(a.k, kStretch<T>));
    return hipGetLastError();
}
// The fragments of outputs a workgroup of linear_long_kernel takes; 0: not its case.
template <typename T>
int long_fragments(const FwdArgs &a) {
    const int fr = a.n <= 16 ? 1 : a.n <= 32 ? 2 : 4;
    return div_up(a.n, 16 * fr) <= kLongSlices && long_bytes<T>(a, fr) ? fr : 0;
}
template <typename T, typename Y>
hipError_t run_long(const FwdArgs &a, hipStream_t stream) {
    switch (long_fragments<T>(a)) {
        case 1: return long_launch<T, Y, 1>(a, stream);
        case 2: return long_launch<T, Y, 2>(a, stream);
        default: return long_launch<T, Y, 4>(a, stream);
    }
}

// Many rows, a weight too large to stay in LDS.  A workgroup makes a block of 128
// rows by 256 outputs, its eight waves 64 x 64 each, over steps of 128 bytes of
// the contraction: the next step's pieces of x and W are on their way into
// registers while this step's are read from LDS as fragments.  Two workgroups a
// CU (128 registers a wave, 48 KB of LDS each) fill each other's barriers and
// epilogues.  Row and output tiles are dealt to the XCDs in runs, the output
// tiles of one row tile next to each other, so x and W come from an XCD's L2 after
// their first reader.
// In LDS a row's eight pieces are permuted by three bits of its number, those in
// which the 16 rows of a fragment read differ, lines of 256 bytes apart: rows
// follow each other in x, and in W go as the outputs are dealt to the lanes.
// No unit is: the matrix units are 23 % busy, LDS is active 18-20 % of the cycles
// without conflicts.  A step's LDS writes, its reads and its products follow one
// another between two barriers, and two workgroups a CU do not fill the gaps.  y
// leaves in half lines: 1.7 times its bytes are written.  2^16 x 1024 x 1024 bf16
// 240-290 us, 0.5-0.57 PFLOP/s.
template <bool kDealt>
__device__ __forceinline__ int block_at(int row, int piece) {
    const int turn = kDealt ? ((row >> 1) & 1) | ((row >> 2) & 6) : (row >> 1) & 7;
    return row * 128 + ((piece ^ turn) << 4);
}
constexpr int kBlockM = 128, kBlockN = 256;
template <typename T, typename Y>
__global__ __launch_bounds__(512, 4) void linear_block_kernel(const FwdArgs a, int tiles_n, int per_xcd, int tiles) {
    __shared__ __attribute__((aligned(16))) char xt[kBlockM * 128], wt[kBlockN * 128];
    constexpr int kStep = 128 / (int)sizeof(T), kX = kBlockM * 8 / 512, kW = kBlockN * 8 / 512;
    const int tile = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
    if (tile >= tiles) return;
    const int64_t m0 = (int64_t)(tile / tiles_n) * kBlockM;
    const int n0 = tile % tiles_n * kBlockN;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, row16 = lane & 15, group = lane >> 4;
    const int wm = wave & 1, wn = wave >> 1;
    const int p = threadIdx.x & 7, row = threadIdx.x >> 3;  // this thread's piece of its rows row, row + 64, ...

    const T *xr[kX], *wr[kW];
#pragma unroll
    for (int i = 0; i < kX; ++i) {
        const int64_t m = m0 + row + i * 64;
        xr[i] = (const T *)a.x + (m < a.m ? m : a.m - 1) * a.xs;
    }
#pragma unroll
    for (int i = 0; i < kW; ++i) {
        const int n = n0 + row + i * 64;
        wr[i] = (const T *)a.w + (int64_t)(n < a.n ? n : a.n - 1) * a.ws;
    }
    u32x4 nx[kX], nw[kW];
    auto fetch = [&](int k0) {
        const int k = k0 + p * kPiece<T>, at = k + kPiece<T> <= a.k ? k : a.k - kPiece<T>;
#pragma unroll
        for (int i = 0; i < kX; ++i) nx[i] = load_loose<u32x4>(xr[i] + at);
#pragma unroll
        for (int i = 0; i < kW; ++i) nw[i] = load_loose<u32x4>(wr[i] + at);
    };

    f32x4 acc[4][4] = {};
    fetch(0);
    for (int k0 = 0; k0 < a.k; k0 += kStep) {
        if (k0 + kStep > a.k) {  // the step that the contraction's end cuts
            const u32x4 mask = cut_piece<T>(k0 + p * kPiece<T>, a.k).mask;
#pragma unroll
            for (int i = 0; i < kX; ++i) nx[i] &= mask;
#pragma unroll
            for (int i = 0; i < kW; ++i) nw[i] &= mask;
        }
        __syncthreads();  // the last step's reads are done
#pragma unroll
        for (int i = 0; i < kX; ++i) *(u32x4 *)(xt + block_at<false>(row + i * 64, p)) = nx[i];
#pragma unroll
        for (int i = 0; i < kW; ++i) *(u32x4 *)(wt + block_at<true>(row + i * 64, p)) = nw[i];
        __syncthreads();
        if (k0 + kStep < a.k) fetch(k0 + kStep);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            u32x4 x[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) x[r] = *(const u32x4 *)(xt + block_at<false>(wm * 64 + r * 16 + row16, u * 4 + group));
            if constexpr (sizeof(T) == 1) {
                Widened xw[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) xw[r] = widen(x[r]);
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const int n = wn * 64 + (f >> 1) * 32 + (row16 >> 2) * 8 + (f & 1) * 4 + (row16 & 3);
                    const Widened w = widen(*(const u32x4 *)(wt + block_at<true>(n, u * 4 + group)));
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[r][f] = mma16<f16>(w.hi, xw[r].hi, mma16<f16>(w.lo, xw[r].lo, acc[r][f]));
                }
            } else {
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const int n = wn * 64 + (f >> 1) * 32 + (row16 >> 2) * 8 + (f & 1) * 4 + (row16 & 3);
                    const u32x4 w = *(const u32x4 *)(wt + block_at<true>(n, u * 4 + group));
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[r][f] = mma16<T>(w, x[r], acc[r][f]);
                }
            }
        }
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int n = n0 + wn * 64 + q * 32 + group * 8, left = a.n - n;
        float bs[8], ws[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            bs[j] = a.bias && j < left ? a.bias[n + j] : 0.f;
            if constexpr (sizeof(T) == 1) ws[j] = j < left ? a.w_scale[n + j] : 0.f;
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t m = m0 + wm * 64 + r * 16 + row16;
            if (m >= a.m || left <= 0) continue;
            Held<8, Y> res;
            if (a.r) res = hold<8>((const Y *)a.r + m * a.rs + n, left);
            float z[8];
            float xsc = 1.f;
            if constexpr (sizeof(T) == 1) xsc = a.x_scale[m];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                z[j] = acc[r][q * 2 + j / 4][j % 4];
                if constexpr (sizeof(T) == 1) z[j] = fmaf(z[j] * xsc, ws[j], bs[j]);
                else z[j] += bs[j];
            }
            if constexpr (sizeof(T) == 2)
                if (a.pre) put((T *)a.pre + m * a.ps + n, left, rounded<8, T>(z));
            activate_all(z, a.act);
            if (a.r)
#pragma unroll
                for (int j = 0; j < 8; ++j) z[j] += (float)res.v[j];
            put((Y *)a.y + m * a.ys + n, left, rounded<8, Y>(z));
        }
    }
}

template <typename T, typename Y>
hipError_t run_block(const FwdArgs &a, hipStream_t stream) {
    const int tiles_n = (int)div_up(a.n, kBlockN);
    FwdArgs part = a;
    const int64_t most = ((int64_t)1 << 29) / tiles_n / kBlockM * kBlockM;  // rows of a launch: 2^31 threads at most
    for (int64_t m = 0; m < a.m; m += most) {
        part.m = a.m - m < most ? a.m - m : most;
        part.x = (const T *)a.x + m * a.xs;
        part.r = a.r ? (const Y *)a.r + m * a.rs : nullptr;
        part.y = (Y *)a.y + m * a.ys;
        part.pre = a.pre ? (T *)a.pre + m * a.ps : nullptr;
        part.x_scale = a.x_scale ? a.x_scale + m : nullptr;
        const int tiles = (int)div_up(part.m, kBlockM) * tiles_n, per_xcd = (int)div_up(tiles, 8);
        linear_block_kernel<T, Y><<<dim3((unsigned)per_xcd * 8), 512, 0, stream>>>(part, tiles_n, per_xcd, tiles);
    }
    return hipGetLastError();
}

template <typename T, typename Y>
hipError_t run_stream(const FwdArgs &a, hipStream_t stream) {
    if (a.k < kPiece<T>) return stream_set<T, Y, 1, 2>(a, stream);
    const bool cut = a.k % kStretch<T> != 0;
    switch (div_up(a.k, kStretch<T>)) {
#define HG_STREAM(KU) \
    case KU: return cut ? stream_set<T, Y, KU, 1>(a, stream) : stream_set<T, Y, KU, 0>(a, stream);
        HG_STREAM(1)
        HG_STREAM(2)
        HG_STREAM(3)
        HG_STREAM(4)
        HG_STREAM(5)
        HG_STREAM(6)
        HG_STREAM(7)
        HG_STREAM(8)
        HG_STREAM(9)
        HG_STREAM(10)
        HG_STREAM(11)
        HG_STREAM(12)
        HG_STREAM(13)
        HG_STREAM(14)
        HG_STREAM(15)
        HG_STREAM(16)
#undef HG_STREAM
    }
    return hipErrorInvalidValue;
}

template <typename T, typename Y>
hipError_t linear_run(const FwdArgs &a, hipStream_t stream) {
    // The tile kernel reads W, in whole 16 x 32 tiles, for every 16 rows (30 us per
    // 10^9 multiply-adds, at 64 x 64 to 1024 x 1024 alike); the others first bring W
    // in: the stream kernel a slice of it (14 KB/us and CU, and x again for every
    // further slice), the block kernel a step of 128 bytes of the contraction in
    // 2.2 us.  At 256 x 256 they meet near 2^11 rows (6 us), at 64 x 64 near 2^13
    // (3.4 us), at 1024 x 1024 near 1200 (36 us).
    const double tile_us = 3e-8 * (double)a.m * (16 * div_up(a.n, 16)) * (32 * div_up(a.k, 32));
    const double row = (double)a.k * sizeof(T);
    const bool stream_fits = div_up(a.k, kStretch<T>) <= 16;
    const double slices = few_rows_slices(a) > 1 ? few_rows_slices(a) : 1;
    const bool long_fits = !stream_fits && long_fragments<T>(a);
    const double other_us = stream_fits ? 0.5 + (a.n * row / slices + a.m * row * (slices - 1) / kCus) / 14500.
                            : long_fits ? 0.5 + (a.n < 64 ? a.n : 64) * row / 14500.
                                        : 2.2 * div_up((int64_t)row, 128);
    if (tile_us > other_us)
        return stream_fits ? run_stream<T, Y>(a, stream) : long_fits ? run_long<T, Y>(a, stream) : run_block<T, Y>(a, stream);
    FwdArgs part = a;
    const int64_t most = 65535LL * 16;  // rows a grid's second dimension reaches
    for (int64_t m = 0; m < a.m; m += most) {
        part.m = a.m - m < most ? a.m - m : most;
        part.x = (const T *)a.x + m * a.xs;
        part.r = a.r ? (const Y *)a.r + m * a.rs : nullptr;
        part.y = (Y *)a.y + m * a.ys;
        part.pre = a.pre ? (T *)a.pre + m * a.ps : nullptr;
        part.x_scale = a.x_scale ? a.x_scale + m : nullptr;
        linear_tile_kernel<T, Y><<<dim3((unsigned)div_up(a.n, 16), (unsigned)div_up(part.m, 16)), 256, 0, stream>>>(part);
    }
    return hipGetLastError();
}

}  // namespace
}  // namespace res
}  // namespace hg
