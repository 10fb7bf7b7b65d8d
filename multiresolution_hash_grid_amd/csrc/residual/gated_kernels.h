// Kernels of h = act(x Wg^T + bg) (x Wu^T + bu) for one pair of types; the sources
// that include this instantiate one operand type each, so that they build at once.
#pragma once

#include "gated_common.h"

namespace hg {
namespace res {
namespace {

// Few rows.  A workgroup computes 16 rows by 16 hidden units; its four waves share
// the contraction and add their sums in LDS.  The rows of x, Wg and Wu come straight
// from memory as fragments, so a single point costs one read of both weights.
// Bound by the loads' latency: 1 x 256 -> 512 bf16 3.4 us, 256 rows of it 4.2.
template <typename T, typename Y>
__global__ __launch_bounds__(256) void gated_tile_kernel(const GatedArgs a) {
    __shared__ f32x4 sums[2][4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, group = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.y * 16;
    const int n0 = blockIdx.x * 16;
    const int64_t xm = m0 + (lane & 15) < a.m ? m0 + (lane & 15) : a.m - 1;
    const int wn = n0 + (lane & 15) < a.n ? n0 + (lane & 15) : a.n - 1;
    const T *x = (const T *)a.x + xm * a.xs, *wg = (const T *)a.wg + (int64_t)wn * a.gs, *wu = (const T *)a.wu + (int64_t)wn * a.us;
    f32x4 g = {0.f, 0.f, 0.f, 0.f}, u = g;
    if (a.k < kPiece<T>) {
        if (wave == 0) {
            const u32x4 none = {0, 0, 0, 0}, v = group ? none : load_short(x, a.k);
            g = mma<T>(group ? none : load_short(wg, a.k), v, g);
            u = mma<T>(group ? none : load_short(wu, a.k), v, u);
        }
    } else {
        for (int k0 = wave * kStretch<T>; k0 < a.k; k0 += 4 * kStretch<T>) {
            const Cut<T> c = cut_piece<T>(k0 + group * kPiece<T>, a.k);
            const u32x4 v = load_loose<u32x4>(x + c.at) & c.mask;
            g = mma<T>(load_loose<u32x4>(wg + c.at) & c.mask, v, g);
            u = mma<T>(load_loose<u32x4>(wu + c.at) & c.mask, v, u);
        }
    }
    sums[0][wave][lane] = g;
    sums[1][wave][lane] = u;
    __syncthreads();
    // thread t: row t / 16, unit t % 16; it lies in lane (unit / 4) * 16 + row, word unit % 4
    const int row = threadIdx.x >> 4, col = threadIdx.x & 15;
    const int64_t m = m0 + row;
    const int n = n0 + col;
    if (m >= a.m || n >= a.n) return;
    float zg = 0.f, zu = 0.f;
    for (int i = 0; i < 4; ++i) zg += sums[0][i][(col >> 2) * 16 + row][col & 3], zu += sums[1][i][(col >> 2) * 16 + row][col & 3];
    // (one after the other: two scales of usable rows may multiply to 0 or infinity)
    if constexpr (sizeof(T) == 1) zg = zg * a.x_scale[m] * a.g_scale[n], zu = zu * a.x_scale[m] * a.u_scale[n];
    if (a.bg) zg += a.bg[n];
    if (a.bu) zu += a.bu[n];
    if constexpr (sizeof(T) == 2)
        if (a.gate) ((T *)a.gate)[m * a.ps + n] = (T)zg, ((T *)a.up)[m * a.qs + n] = (T)zu;
    ((Y *)a.h)[m * a.hs + n] = (Y)(activate(zg, a.act) * zu);
}

// Many rows, weights that fit LDS: they stay there in fragment order, and waves walk
// row tiles on their own, without barriers.  A set is 32 hidden units, two fragments
// of gate rows and two of up rows, dealt so that a lane ends with 8 consecutive units
// of both for each of its rows; a wave holds the fragments of 16 rows for all of the
// contraction.  Sixteen waves of them hide each other's loads better than eight with 32
// rows each (2^18 x 256 -> 128 51 us and 60, 65537 x 35 -> 93 8.9 and 12.3).  Rows shorter
// than a piece are read value by value (2^18 x 3 -> 64 bf16 13 us, in tiles 69).  Bound by
// memory and by the products that the loads wait for (2^18 x 256 -> 128: 4.0 TB/s).
constexpr int kLdsBytes = 160 * 1024;
template <typename T, int KU>
constexpr int kSetBytes = 4 * KU * 1024 * (sizeof(T) == 1 ? 2 : 1) + 2 * 64 * 4;  // fragments, biases, scales

template <typename T, typename Y, int KU, bool kPre>
__global__ __launch_bounds__(1024) void gated_rows_kernel(const GatedArgs a, int slices, int slice_n, int64_t tiles) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int kHalves = sizeof(T) == 1 ? 2 : 1, kFloats = 4 * KU * kHalves * 1024;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), row16 = lane & 15, group = lane >> 4;
    const int waves = blockDim.x >> 6;
    // workgroups b, b + 8, ... share an XCD: the slices of one tile do
    const int xcd = blockIdx.x & 7, in_xcd = blockIdx.x >> 3;
    const int n0 = in_xcd % slices * slice_n, nn = a.n - n0 < slice_n ? a.n - n0 : slice_n;
    const int64_t walker = (int64_t)(in_xcd / slices) * 8 + xcd, walkers = (int64_t)(gridDim.x >> 3) / slices * 8;
    const int sets = (nn + 31) / 32;
    // Piece u of a row of k values; one shorter than a piece lies in the first group's.
    auto piece = [&](const T *row, int u, int k) __attribute__((always_inline)) {
        if (KU == 1 && k < kPiece<T>) return group ? u32x4{0, 0, 0, 0} : load_short(row, k);
        const Cut<T> c = cut_piece<T>(u * kStretch<T> + group * kPiece<T>, k);
        return load_loose<u32x4>(row + c.at) & c.mask;
    };

    for (int b = wave; b < sets * 4 * KU; b += waves) {
        const int s = b / (4 * KU), f = b / KU % 4, u = b % KU;
        const int unit = s * 32 + (row16 >> 2) * 8 + (f & 1) * 4 + (row16 & 3);
        const int64_t n = n0 + (unit < nn ? unit : nn - 1);
        const T *const w = f >> 1 ? (const T *)a.wu + n * a.us : (const T *)a.wg + n * a.gs;
        const u32x4 v = piece(w, u, a.k);
        u32x4 *const to = (u32x4 *)(lds + s * kSetBytes<T, KU>) + (b - s * 4 * KU) * kHalves * 64 + lane;
        if constexpr (sizeof(T) == 1) {
            const Widened x = widen(v);
            to[0] = x.lo, to[64] = x.hi;
        } else {
            *to = v;
        }
    }
    for (int i = threadIdx.x; i < sets * 64; i += blockDim.x) {
        const int unit = i / 64 * 32 + (i & 31), n = n0 + (unit < nn ? unit : nn - 1);
        const bool up = i & 32;
        float *const to = (float *)(lds + i / 64 * kSetBytes<T, KU> + kFloats) + (i & 63);
        const float *const bias = up ? a.bu : a.bg;
        to[0] = bias ? bias[n] : 0.f;
        if constexpr (sizeof(T) == 1) to[64] = (up ? a.u_scale : a.g_scale)[n];
    }
    __syncthreads();

    for (int64_t tile = (int64_t)wave * walkers + walker; tile < tiles; tile += (int64_t)waves * walkers) {
        const int64_t m = tile * 16 + row16, mr = m < a.m ? m : a.m - 1;
        u32x4 x[KU];
        float xsc = 1.f;
        int k = a.k;
        asm volatile("" : "+s"(k));  // where pieces are cut is worked out anew for each tile: held, it would cost registers
#pragma unroll
        for (int u = 0; u < KU; ++u) x[u] = piece((const T *)a.x + mr * a.xs, u, k);
        if constexpr (sizeof(T) == 1) xsc = a.x_scale[mr];
        for (int s = 0; s < sets; ++s) {
            const char *const buffer = lds + s * kSetBytes<T, KU>;
            const float *const bias = (const float *)(buffer + kFloats) + group * 8, *const scale = bias + 64;
            f32x4 acc[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                // sums begin with the bias; 8-bit ones are scaled first
                if constexpr (sizeof(T) == 1) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
                else acc[f] = *(const f32x4 *)(bias + (f >> 1) * 32 + (f & 1) * 4);
            }
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                Widened xw;
                if constexpr (sizeof(T) == 1) {
                    asm volatile("" : "+v"(x[u]));  // widen here, not once before all sets: the registers are not there
                    xw = widen(x[u]);
                }
#pragma unroll
                for (int f = 0; f < 4; ++f)
#pragma unroll
                    for (int i = 0; i < kHalves; ++i) {
                        const u32x4 v = ((const u32x4 *)buffer)[((f * KU + u) * kHalves + i) * 64 + lane];
                        if constexpr (sizeof(T) == 1) acc[f] = mma16<f16>(v, i ? xw.hi : xw.lo, acc[f]);
                        else acc[f] = mma16<T>(v, x[u], acc[f]);
                    }
            }
            const int at = n0 + s * 32 + group * 8, left = n0 + nn - at;
            float g[8], v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g[j] = acc[j / 4][j % 4], v[j] = acc[2 + j / 4][j % 4];
                if constexpr (sizeof(T) == 1) g[j] = fmaf(g[j] * xsc, scale[j], bias[j]), v[j] = fmaf(v[j] * xsc, scale[32 + j], bias[32 + j]);
            }
            if (m < a.m) {
                if constexpr (kPre) {
                    put((T *)a.gate + m * a.ps + at, left, rounded<8, T>(g));
                    put((T *)a.up + m * a.qs + at, left, rounded<8, T>(v));
                }
                gate_all(g, v, a.act);
                put((Y *)a.h + m * a.hs + at, left, rounded<8, Y>(g));
            }
        }
    }
}

// How the rows kernel is cut: 16 waves a workgroup, a workgroup a CU.  With fewer
// rows than fill the card, the units go to several workgroups, in whole sets.
struct RowsPlan {
    int slices, slice_n, bytes;
    int64_t tiles, rounds;  // of 16 rows; of 16 waves
};
template <typename T, int KU>
RowsPlan rows_plan(const GatedArgs &a) {
    RowsPlan p;
    p.tiles = div_up(a.m, 16), p.rounds = div_up(p.tiles, 16);
    const int sets = (int)div_up(a.n, 32);
    const int want = p.rounds < kCus ? (int)(kCus / p.rounds) : 1;
    p.slice_n = (int)div_up(sets, want < sets ? want : sets) * 32;
    p.slices = (int)div_up(a.n, p.slice_n);
    p.bytes = p.slice_n / 32 * kSetBytes<T, KU>;
    return p;
}
template <typename T, typename Y, int KU, bool kPre>
hipError_t rows_launch(const GatedArgs &a, const RowsPlan &p, hipStream_t stream) {
    const auto kernel = gated_rows_kernel<T, Y, KU, kPre>;
    if (p.bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, p.bytes);
        if (e != hipSuccess) return e;
    }
    int64_t walkers = kCus / p.slices < p.rounds ? kCus / p.slices : p.rounds;
    walkers = div_up(walkers < 1 ? 1 : walkers, 8) * 8;  // whole rounds over the XCDs
    kernel<<<dim3((unsigned)(walkers * p.slices)), 1024, p.bytes, stream>>>(a, p.slices, p.slice_n, p.tiles);
    return hipGetLastError();
}

// Many rows, weights too large for LDS: the weights stay in registers and the rows
// come by.  Each wave keeps the gate and up fragments of its 32 * HS hidden units for
// all of the contraction, a workgroup 256 * HS units; the rows' fragments lie in LDS,
// in chunks of kRows rows that all waves read, the next chunk's pieces on their way
// into registers meanwhile.  A row fragment read from LDS meets 4 * HS weight
// fragments, x is read once for every slice of 256 * HS units (the slices of a row
// chunk are on one XCD, next to each other), and nothing but rows moves, so loads,
// products and stores overlap all the way.
// One barrier a chunk.  The last units of a chunk are stored after the next chunk's rows
// have come and before those of the one after are asked for, so that a wait for loads
// never waits for young stores.
// Bound by the products and the gating, which the two waves of a SIMD hardly overlap
// (matrix units 44 %, VALU 50 % busy): 2^20 x 256 -> 512 bf16 551 - 585 us, 0.94 - 1.0
// PFLOP/s; 8-bit 2^17 x 512 -> 1024 257 - 286, where widening is VALU work too.  With both
// projections kept by the writes: 2^18 x 256 -> 512 222 - 232 us, 4.1 TB/s, 806 MB written.
constexpr int kUnitThreads = 512;
template <int KU>
constexpr int kUnitRows = KU <= 4 ? 128 : 64;
template <typename T, int KU>
constexpr int kUnitBuffer = kUnitRows<KU> * (KU * 64 * (sizeof(T) == 1 ? 2 : 1) + 4);  // fragments, scales
// Sets of 32 hidden units of a wave: two where registers hold their weights, sums and
// outputs (2^18 x 64 -> 1024 bf16 145 us, one set 153; 8-bit x 128 -> 1024 to fp32, with whose
// second set they spill, 293 and 339).
template <typename T, typename Y, int KU>
constexpr int kUnitSets = KU <= (sizeof(T) == 1 && sizeof(Y) == 4 ? 1 : 2) ? 2 : 1;

template <typename T, typename Y, int KU, int RF, bool kPre>
__global__ __launch_bounds__(kUnitThreads) void gated_units_kernel(const GatedArgs a, int slices, int slice_n, int64_t tiles) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int kHalves = sizeof(T) == 1 ? 2 : 1, HS = kUnitSets<T, Y, KU>, R = kUnitRows<KU>, kPer = R / 16 * KU / 8;
    constexpr int kBuffer = kUnitBuffer<T, KU>, kScales = R * KU * 64 * kHalves, kUnits = 256 * HS, kRounds = R / 16 / RF;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), row16 = lane & 15, group = lane >> 4;
    const int xcd = blockIdx.x & 7, in_xcd = blockIdx.x >> 3;
    const int n0 = in_xcd % slices * slice_n, nn = a.n - n0 < slice_n ? a.n - n0 : slice_n;
    const int64_t walker = (int64_t)(in_xcd / slices) * 8 + xcd, walkers = (int64_t)(gridDim.x >> 3) / slices * 8;
    const int first = wave * 32 * HS;  // this wave's units
    float *const bias = (float *)(lds + 2 * kBuffer), *const scale = bias + 2 * kUnits;  // [gate, up][units]
    if (walker >= tiles) return;

    u32x4 w[HS][4][KU];
#pragma unroll
    for (int h = 0; h < HS; ++h)
#pragma unroll
        for (int f = 0; f < 4; ++f) {
            const int unit = first + h * 32 + (row16 >> 2) * 8 + (f & 1) * 4 + (row16 & 3);
            const int64_t n = n0 + (unit < nn ? unit : nn - 1);
            const T *const row = f >> 1 ? (const T *)a.wu + n * a.us : (const T *)a.wg + n * a.gs;
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                const Cut<T> c = cut_piece<T>(u * kStretch<T> + group * kPiece<T>, a.k);
                w[h][f][u] = load_loose<u32x4>(row + c.at) & c.mask;
            }
        }
    for (int i = threadIdx.x; i < 2 * kUnits; i += kUnitThreads) {
        const bool up = i >= kUnits;
        const int unit = i - (up ? kUnits : 0), n = n0 + (unit < nn ? unit : nn - 1);
        const float *const b = up ? a.bu : a.bg;
        bias[i] = b ? b[n] : 0.f;
        if constexpr (sizeof(T) == 1) scale[i] = (up ? a.u_scale : a.g_scale)[n];
    }

    // Where pieces are cut is worked out anew each time: held, it would cost registers
    // that the weights and the sums need.
    auto width = [&] {
        int k = a.k;
        asm volatile("" : "+s"(k));
        return k;
    };
    u32x4 staged[kPer];
    float staged_scale = 0.f;
    int64_t ahead = walker;  // the chunk of rows that is fetched next
    auto fetch = [&] {
        const int k = width();
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int b = wave * kPer + j;
            const int64_t m = ahead * R + b / KU * 16 + row16;
            staged[j] = load_loose<u32x4>((const T *)a.x + (m < a.m ? m : a.m - 1) * a.xs +
                                          cut_piece<T>(b % KU * kStretch<T> + group * kPiece<T>, k).at);
        }
        if constexpr (sizeof(T) == 1)
            if (threadIdx.x < R) staged_scale = a.x_scale[ahead * R + threadIdx.x < a.m ? ahead * R + threadIdx.x : a.m - 1];
        ahead += walkers;
    };
    auto stage = [&](char *to) {
        const int k = width();
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int b = wave * kPer + j;
            const u32x4 v = staged[j] & cut_piece<T>(b % KU * kStretch<T> + group * kPiece<T>, k).mask;
            if constexpr (sizeof(T) == 1) {
                const Widened x = widen(v);
                ((u32x4 *)to)[b * 128 + lane] = x.lo;
                ((u32x4 *)to)[b * 128 + 64 + lane] = x.hi;
            } else {
                ((u32x4 *)to)[b * 64 + lane] = v;
            }
        }
        if constexpr (sizeof(T) == 1)
            if (threadIdx.x < R) ((float *)(to + kScales))[threadIdx.x] = staged_scale;
    };

    Held<8, Y> h[HS][RF];
    typedef std::conditional_t<sizeof(T) == 1, f16, T> P;  // (8-bit operands keep no projections)
    Held<8, P> gate[kPre ? HS : 1][RF], up[kPre ? HS : 1][RF];
    int64_t pending = -1;  // row of the finished units that are still to be stored
    auto flush = [&] {
        if (pending < 0) return;
#pragma unroll
        for (int s = 0; s < HS; ++s) {
            const int unit = first + s * 32 + group * 8, left = nn - unit, at = n0 + unit;
#pragma unroll
            for (int r = 0; r < RF; ++r) {
                const int64_t m = pending + r * 16;
                if (m < a.m) {
                    put((Y *)a.h + m * a.hs + at, left, h[s][r]);
                    if constexpr (kPre) {
                        put((P *)a.gate + m * a.ps + at, left, gate[s][r]);
                        put((P *)a.up + m * a.qs + at, left, up[s][r]);
                    }
                }
            }
        }
        pending = -1;
    };

    const int64_t all = (tiles - 1 - walker) / walkers + 1;  // chunks of this workgroup
    int64_t q = 0;
    auto barrier = [] {  // this wave's LDS writes are done, and so are the others'
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    };
    // Chunk q is in its buffer, and the one before is done with.
    auto advance = [&] {
        barrier();
        if (q + 1 < all) stage(lds + ((q + 1) & 1) * kBuffer);
        flush();
        if (q + 2 < all) fetch();
    };
    fetch();
    stage(lds);
    if (all > 1) fetch();
    advance();
    while (q < all) {
        const int64_t m0 = (walker + q * walkers) * R + row16;
        const char *const buffer = lds + (q & 1) * kBuffer;
#pragma unroll
        for (int p = 0; p < kRounds; ++p) {
            f32x4 acc[HS][RF][4];
            if (first < nn) {
#pragma unroll
                for (int s = 0; s < HS; ++s)
#pragma unroll
                    for (int f = 0; f < 4; ++f) {
                        // sums begin with the bias; 8-bit ones are scaled first
                        if constexpr (sizeof(T) == 1) acc[s][0][f] = f32x4{0.f, 0.f, 0.f, 0.f};
                        else acc[s][0][f] = *(const f32x4 *)(bias + (f >> 1) * kUnits + first + s * 32 + group * 8 + (f & 1) * 4);
#pragma unroll
                        for (int r = 1; r < RF; ++r) acc[s][r][f] = acc[s][0][f];
                    }
#pragma unroll
                for (int u = 0; u < KU; ++u) {
                    u32x4 x[RF][kHalves];
#pragma unroll
                    for (int r = 0; r < RF; ++r)
#pragma unroll
                        for (int i = 0; i < kHalves; ++i) x[r][i] = ((const u32x4 *)buffer)[(((p * RF + r) * KU + u) * kHalves + i) * 64 + lane];
#pragma unroll
                    for (int s = 0; s < HS; ++s)
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            if constexpr (sizeof(T) == 1) {
                                asm volatile("" : "+v"(w[s][f][u]));  // widen here, not once: the registers are not there
                                const Widened v = widen(w[s][f][u]);
#pragma unroll
                                for (int r = 0; r < RF; ++r) acc[s][r][f] = mma16<f16>(v.hi, x[r][kHalves - 1], mma16<f16>(v.lo, x[r][0], acc[s][r][f]));
                            } else {
#pragma unroll
                                for (int r = 0; r < RF; ++r) acc[s][r][f] = mma16<T>(w[s][f][u], x[r][0], acc[s][r][f]);
                            }
                        }
                }
                if constexpr (sizeof(T) == 1)
#pragma unroll
                    for (int r = 0; r < RF; ++r) {
                        const float xs = ((const float *)(buffer + kScales))[(p * RF + r) * 16 + row16];
#pragma unroll
                        for (int s = 0; s < HS; ++s)
#pragma unroll
                            for (int f = 0; f < 4; ++f) {
                                const int at = (f >> 1) * kUnits + first + s * 32 + group * 8 + (f & 1) * 4;
                                const f32x4 sc = *(const f32x4 *)(scale + at), b = *(const f32x4 *)(bias + at);
#pragma unroll
                                for (int j = 0; j < 4; ++j) acc[s][r][f][j] = fmaf(acc[s][r][f][j] * xs, sc[j], b[j]);
                            }
                    }
            }
            if (first < nn) {
                flush();
#pragma unroll
                for (int s = 0; s < HS; ++s)
#pragma unroll
                    for (int r = 0; r < RF; ++r) {
                        float g[8], v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) g[j] = acc[s][r][j / 4][j % 4], v[j] = acc[s][r][2 + j / 4][j % 4];
                        if constexpr (kPre) gate[s][r] = rounded<8, P>(g), up[s][r] = rounded<8, P>(v);
                        gate_all(g, v, a.act);
                        h[s][r] = rounded<8, Y>(g);
                    }
                pending = m0 + p * RF * 16;
            }
        }
        if (++q < all) advance();
    }
    flush();
}

template <typename T, typename Y, int KU, int RF, bool kPre>
hipError_t units_launch(const GatedArgs &a, hipStream_t stream) {
    const auto kernel = gated_units_kernel<T, Y, KU, RF, kPre>;
    const int64_t tiles = div_up(a.m, kUnitRows<KU>);
    constexpr int most = 256 * kUnitSets<T, Y, KU>;
    int slices = (int)div_up(a.n, most);
    const int slice_n = (int)div_up(div_up(a.n, slices), 32) * 32;
    const int bytes = 2 * kUnitBuffer<T, KU> + 2 * most * 4 * (sizeof(T) == 1 ? 2 : 1);
    if (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    int64_t walkers = kCus / slices < tiles ? kCus / slices : tiles;
    walkers = div_up(walkers < 1 ? 1 : walkers, 8) * 8;  // whole rounds over the XCDs
    kernel<<<dim3((unsigned)(walkers * slices)), kUnitThreads, bytes, stream>>>(a, slices, slice_n, tiles);
    return hipGetLastError();
}

template <typename T, typename Y, int KU>
hipError_t rows_pick(const GatedArgs &a, hipStream_t stream) {
    const RowsPlan p = rows_plan<T, KU>(a);
    const bool fits = p.bytes <= kLdsBytes;
    if constexpr (sizeof(T) == 2)
        if (a.gate) return fits ? rows_launch<T, Y, KU, true>(a, p, stream) : units_launch<T, Y, KU, 2, true>(a, stream);
    return fits ? rows_launch<T, Y, KU, false>(a, p, stream) : units_launch<T, Y, KU, 2, false>(a, stream);
}

// Many rows, a contraction longer than a wave's registers hold: blocks of 256 rows by
// 128 hidden units (256 rows of weights) over steps of 64 values of the contraction.
// Eight waves make 128 rows by 32 units of both projections each.  A step's pieces lie
// in LDS as fragments, in one of two buffers; the next step's are written into the
// other, and those of the one after are on their way into registers, across the ends
// of blocks too: one barrier a step, and a workgroup's next block begins while its last
// one is gated.
// The blocks of an XCD are dealt in runs, those of one row tile next to each other, so
// x and the weights come from its L2 after their first reader.
// 2^16 x 1024 -> 1024 bf16 310 us, 0.89 PFLOP/s (2691 with the tile kernel): matrix units
// 33 %, VALU 29 %, LDS 22 % busy; what is left are the steps' barriers and the blocks' ends.
constexpr int kBlockRows = 256, kBlockUnits = 128, kBlockThreads = 512;
template <typename T, typename Y, bool kPre>
__global__ __launch_bounds__(kBlockThreads) void gated_block_kernel(const GatedArgs a, int tiles_n, int64_t tiles, int64_t per_xcd) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    constexpr int kHalves = sizeof(T) == 1 ? 2 : 1, kU = sizeof(T) == 1 ? 1 : 2;  // f16 fragments of a raw one; raw ones of a step
    constexpr int kStep = 64, kSide = 16 * 2 * 1024, kBuffer = 2 * kSide;        // x's 16 row fragments, then the weights' 16
    constexpr int kPer = 32 * kU / 8;                                             // raw fragments a wave brings
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), row16 = lane & 15, group = lane >> 4;
    const int wm = wave & 1, wn = wave >> 1;
    const int64_t walker = blockIdx.x >> 3, walkers = gridDim.x >> 3, base = (int64_t)(blockIdx.x & 7) * per_xcd;
    const int64_t mine = tiles - base < per_xcd ? tiles - base : per_xcd;  // blocks of this XCD
    if (walker >= mine) return;
    const int steps = (a.k + kStep - 1) / kStep;
    const int64_t all = ((mine - 1 - walker) / walkers + 1) * steps;

    // What is fetched next: a block and a step of it.
    int64_t next_tile = walker;
    int next_k = 0;
    u32x4 staged[kPer];
    auto fetch = [&]() __attribute__((always_inline)) {
        const int64_t tile = base + (next_tile < mine ? next_tile : mine - 1);
        const int64_t m0 = tile / tiles_n * kBlockRows;
        const int n0 = (int)(tile % tiles_n) * kBlockUnits;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int b = wave * (kPer / 2) + j % (kPer / 2), f = b / kU, u = b % kU;  // half of them x's, half the weights'
            const int k = next_k + u * kStretch<T> + group * kPiece<T>, at = k + kPiece<T> <= a.k ? k : a.k - kPiece<T>;
            const T *row;
            if (j < kPer / 2) {
                const int64_t m = m0 + f * 16 + row16;
                row = (const T *)a.x + (m < a.m ? m : a.m - 1) * a.xs;
            } else {
                // 32 units: fragments of gate rows 2, of up rows 2
                const int unit = n0 + (f >> 2) * 32 + (row16 >> 2) * 8 + (f & 1) * 4 + (row16 & 3), n = unit < a.n ? unit : a.n - 1;
                row = f & 2 ? (const T *)a.wu + (int64_t)n * a.us : (const T *)a.wg + (int64_t)n * a.gs;
            }
            staged[j] = load_loose<u32x4>(row + at);
        }
        next_tile += next_k + kStep < a.k ? 0 : walkers;
        next_k = next_k + kStep < a.k ? next_k + kStep : 0;
    };
    auto stage = [&](char *to, int k0) __attribute__((always_inline)) {
        if (k0 + kStep > a.k)  // the step that the contraction's end cuts
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                staged[j] &= cut_piece<T>(k0 + (wave * (kPer / 2) + j % (kPer / 2)) % kU * kStretch<T> + group * kPiece<T>, a.k).mask;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            u32x4 *const p = (u32x4 *)(to + (j < kPer / 2 ? 0 : kSide)) + (wave * (kPer / 2) + j % (kPer / 2)) * kHalves * 64 + lane;
            if constexpr (sizeof(T) == 1) {
                const Widened v = widen(staged[j]);
                p[0] = v.lo, p[64] = v.hi;
            } else {
                *p = staged[j];
            }
        }
    };
    auto barrier = [] {  // this wave's LDS writes are done, and so are the others'
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    };

    fetch();
    stage(lds, 0);
    fetch();
    f32x4 acc[8][4];
    int k0 = 0;
    int64_t tile = walker;
    for (int64_t q = 0; q < all; ++q) {
        barrier();  // this step is in its buffer, and the last one's is done with
        const int next = k0 + kStep < a.k ? k0 + kStep : 0;
        stage(lds + ((q + 1) & 1) * kBuffer, next);
        fetch();
        if (k0 == 0)
#pragma unroll
            for (int r = 0; r < 8; ++r)
#pragma unroll
                for (int f = 0; f < 4; ++f) acc[r][f] = f32x4{0.f, 0.f, 0.f, 0.f};
        const u32x4 *const x = (const u32x4 *)(lds + (q & 1) * kBuffer), *const w = (const u32x4 *)(lds + (q & 1) * kBuffer + kSide);
        typedef std::conditional_t<sizeof(T) == 1, f16, T> P;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            u32x4 v[4];
#pragma unroll
            for (int f = 0; f < 4; ++f) v[f] = w[((wn * 4 + f) * 2 + u) * 64 + lane];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const u32x4 t = x[((wm * 8 + r) * 2 + u) * 64 + lane];
#pragma unroll
                for (int f = 0; f < 4; ++f) acc[r][f] = mma16<P>(v[f], t, acc[r][f]);
            }
        }
        k0 = next;
        if (next) continue;
        // The block is whole.
        const int64_t at = base + tile, m0 = at / tiles_n * kBlockRows + wm * 128 + row16;
        const int n = (int)(at % tiles_n) * kBlockUnits + wn * 32 + group * 8, left = a.n - n;
        tile += walkers;
        if (left <= 0) continue;
        float bg[8], bu[8], sg[8], su[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = j < left ? n + j : n;
            bg[j] = a.bg ? a.bg[c] : 0.f, bu[j] = a.bu ? a.bu[c] : 0.f;
            if constexpr (sizeof(T) == 1) sg[j] = a.g_scale[c], su[j] = a.u_scale[c];
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int64_t m = m0 + r * 16;
            if (m >= a.m) continue;
            float xs = 1.f;
            if constexpr (sizeof(T) == 1) xs = a.x_scale[m];
            float g[8], v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g[j] = acc[r][j / 4][j % 4], v[j] = acc[r][2 + j / 4][j % 4];
                if constexpr (sizeof(T) == 1) g[j] = fmaf(g[j] * xs, sg[j], bg[j]), v[j] = fmaf(v[j] * xs, su[j], bu[j]);
                else g[j] += bg[j], v[j] += bu[j];
            }
            if constexpr (kPre) {
                put((T *)a.gate + m * a.ps + n, left, rounded<8, T>(g));
                put((T *)a.up + m * a.qs + n, left, rounded<8, T>(v));
            }
            gate_all(g, v, a.act);
            put((Y *)a.h + m * a.hs + n, left, rounded<8, Y>(g));
        }
    }
}

template <typename T, typename Y, bool kPre>
hipError_t block_launch(const GatedArgs &a, hipStream_t stream) {
    const auto kernel = gated_block_kernel<T, Y, kPre>;
    constexpr int bytes = 2 * 2 * 16 * 2 * 1024;
    const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
    const int tiles_n = (int)div_up(a.n, kBlockUnits);
    const int64_t tiles = div_up(a.m, kBlockRows) * tiles_n, per_xcd = div_up(tiles, 8);
    const int64_t walkers = per_xcd < kCus / 8 ? per_xcd : kCus / 8;
    kernel<<<dim3((unsigned)(walkers * 8)), kBlockThreads, bytes, stream>>>(a, tiles_n, tiles, per_xcd);
    return hipGetLastError();
}
template <typename T, typename Y>
hipError_t run_block(const GatedArgs &a, hipStream_t stream) {
    if constexpr (sizeof(T) == 2)
        if (a.gate) return block_launch<T, Y, true>(a, stream);
    return block_launch<T, Y, false>(a, stream);
}

// Fragments of the contraction: those that are instantiated.  0: more, or rows shorter than a
// piece and weights too large for LDS.
template <typename T>
int rows_fragments(const GatedArgs &a) {
    const int64_t u = div_up(a.k, kStretch<T>);
    if (a.k < kPiece<T> && rows_plan<T, 1>(a).bytes > kLdsBytes) return 0;
    return u > 8 ? 0 : u <= 4 ? (int)u : u <= 6 ? 6 : 8;
}

template <typename T, typename Y>
hipError_t run_rows(const GatedArgs &a, hipStream_t stream) {
    switch (rows_fragments<T>(a)) {
    case 1: return rows_pick<T, Y, 1>(a, stream);
    case 2: return rows_pick<T, Y, 2>(a, stream);
    case 3: return rows_pick<T, Y, 3>(a, stream);
    case 4: return rows_pick<T, Y, 4>(a, stream);
    case 6: return rows_pick<T, Y, 6>(a, stream);
    default: return rows_pick<T, Y, 8>(a, stream);
    }
}

template <typename T, typename Y>
hipError_t gated_run(const GatedArgs &a, hipStream_t stream) {
    // The tile kernel reads both weights for every 16 rows, in whole 16 x 32 tiles; the
    // others first bring weights in: some units' (6 us: 256 x 256 -> 512 takes 4.2 with tiles, 512 rows of it 5.4 with
    // weights in LDS), or a step of 64 of the contraction at a time in 2.1 us (1024 x 512 -> 512 takes 14.3 with tiles,
    // 2048 rows of it 24 in blocks).
    const double tile_us = 2.5 + 4e-8 * (16 * div_up(a.m, 16)) * (double)(16 * div_up(a.n, 16)) * (32 * div_up(a.k, 32));
    const double block_us = 7 + 2.1 * div_up(a.k, 64) * div_up(div_up(a.m, kBlockRows) * div_up(a.n, kBlockUnits), kCus);
    if (rows_fragments<T>(a) ? tile_us > 6 : a.k >= kPiece<T> && tile_us > block_us)
        return rows_fragments<T>(a) ? run_rows<T, Y>(a, stream) : run_block<T, Y>(a, stream);
    GatedArgs part = a;
    const int64_t most = 65535LL * 16;  // rows a grid's second dimension reaches
    for (int64_t m = 0; m < a.m; m += most) {
        part.m = a.m - m < most ? a.m - m : most;
        part.x = (const T *)a.x + m * a.xs;
        part.h = (Y *)a.h + m * a.hs;
        part.gate = a.gate ? (T *)a.gate + m * a.ps : nullptr;
        part.up = a.up ? (T *)a.up + m * a.qs : nullptr;
        part.x_scale = a.x_scale ? a.x_scale + m : nullptr;
        gated_tile_kernel<T, Y><<<dim3((unsigned)div_up(a.n, 16), (unsigned)div_up(part.m, 16)), 256, 0, stream>>>(part);
    }
    return hipGetLastError();
}

}  // namespace
}  // namespace res
}  // namespace hg
