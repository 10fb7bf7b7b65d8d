// Backward of h = act(x Wg^T + bg) (x Wu^T + bu) on the matrix cores; the sources
// that include this instantiate one operand type each.
//
//   dg = dh u act'(g),  du = dh act(g)
//   dx = dg Wg + du Wu,  dwg = dg^T x,  dwu = du^T x,  dbg, dbu = sums over the rows
//
// Blocks that one tile holds (up to 128 hidden units by 128 inputs, or 64 by 256) take one
// pass.  Of larger ones two kernels read dh, g and u and each works dg and du out
// for itself, on their way into a product: written once and read twice they would cost
// as many bytes, and a workspace of two hidden layers.  They are rounded to the operands' type there, as
// products of 16-bit operands need; the biases' gradients sum them unrounded.  Against 64 bits dx and
// dW are off by 2.3e-3 in bfloat16 (1.7e-3 if products were fp32 and outputs alone rounded) and 2.9e-4
// in binary16, there of values below 2^-14 by half a step of 2^-24 each (dh of 4e-6: 8e-3).  A second
// product of what the rounding cuts off would undo it for twice the matrix work, twice the tiles of dg
// and du in LDS and registers that dx does not have; a loss scale undoes binary16's ends for nothing.
#pragma once

#include "gated_grad.h"
#include "grad_tiles.h"

namespace hg {
namespace res {
namespace {

constexpr int kGateThreads = 512;

// Pieces of dh, g and u, and what becomes of them.
struct RawGate {
    u32x4 dh, g, u;
};
template <typename T>
__device__ __forceinline__ void values(u32x4 v, float (&f)[8]) {
    typedef T T8 __attribute__((ext_vector_type(8)));
    const T8 t = __builtin_bit_cast(T8, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (float)t[j];
}
template <typename T>
__device__ __forceinline__ void gate_of(const RawGate &raw, int act, float (&dg)[8], float (&du)[8]) {
    float g[8], u[8], dh[8];
    values<T>(raw.g, g);
    values<T>(raw.u, u);
    values<T>(raw.dh, dh);
    gate_grad_all(g, u, dh, act, dg, du);
}

// The first `left` values of a piece.
template <typename T>
__device__ __forceinline__ void put_piece(T *p, int left, u32x4 v) {
    if (left >= 8) {
        store_loose(p, v);
        return;
    }
    if (left <= 0) return;
    if (left & 4) {
        store_loose(p, u32x2{v[0], v[1]});
        v[0] = v[2], v[1] = v[3], p += 4;
    }
    if (left & 2) {
        store_loose(p, v[0]);
        v[0] = v[1], p += 2;
    }
    if (left & 1) store_loose(p, (uint16_t)v[0]);
}

// tile_columns of the tile of 32 rows at `tile` + m rows: the lane's place is worked
// out once, and a fragment's number only turns bits of it.
// (A multiple of 512 bytes may be added to the place, as to `tile`.)
template <int C>
__device__ __forceinline__ int columns_base(int lane) {
    const int i = lane & 15;
    return tile_at<C>((lane >> 4) * 8 + (i >> 2), (i >> 1) & 1) + (i & 1) * 8;
}
template <int C>
__device__ __forceinline__ u32x4 columns_at(char *tile, int base, int m, int q) {
    union {
        s16x4 h[2];
        u32x4 v;
    } r;
#pragma unroll
    for (int h = 0; h < 2; ++h)  // rows four on: one bit of the turn, which a piece's place is XORed with
        r.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(tile + ((base ^ ((2 * q ^ h) << 4)) + (m + 4 * h) * (C * 2))));
    return r.v;
}

// This wave's LDS accesses are done, and so are the others'.
__device__ __forceinline__ void step_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// dx of 256 rows by KP * 32 inputs a workgroup.  A wave has 32 rows and all of the
// tile's inputs: the sums lie in its registers while the hidden units come by, 32 at
// a time.  Their dh, g and u come straight from memory as fragments (a lane has 8
// units of one row) and become fragments of dg and du in place; the units' rows of
// Wg and Wu lie in LDS, the next units' on their way into registers, and are read
// transposed.  Their columns are dealt so that a lane ends with 8 consecutive inputs
// of a row.
// One barrier a stretch of units.  Between two of them half of the waves multiply first
// and then work out the next dg and du, the others the other way around: of the two
// waves of a SIMD one multiplies while the other computes.
// Both kinds of loads, weights and units, are asked for a stretch ahead and
// unconditionally (past the end they repeat others): the two orders are loops of
// their own and without branches around loads, so that the compiler can count those
// in flight and a wait for the older kind leaves the younger on its way.
// With few rows the units are cut into slices, whose sums dx_join_kernel adds
// (256 rows, 256 -> 512: 18.7 + 4 us; the whole backward 40 instead of 57).
// 2^18 rows, 256 -> 512 bf16 254 us; its bytes at the copy's rate take 179.  Bound by memory:
// a stretch is half a line of each row of dh, g and u, and most lines are fetched
// again for the other half (1499 MB of 805); one stretch's loads (48 KB a workgroup) are
// on their way, a second's leave no registers.  Less by the slopes and the products
// (VALU 40 %, matrix units 22 % busy).
// kShort: rows of units or inputs may be shorter than a piece.
template <typename T, int KP, bool kShort>
__global__ __launch_bounds__(kGateThreads) void gated_dx_kernel(const GatedGradArgs a, int tiles_k, int64_t tiles_m, int slices, int per,
                                                                   float *part) {
    extern __shared__ __attribute__((aligned(16))) char lds[];
    // A row of C weights and 32 bytes: eight rows in a row begin in different banks.
    constexpr int C = KP * 32, S = C * 2 + 32, kHalf = 32 * S, kBuffer = 2 * kHalf, kPer = C / 64;  // kPer: pieces of a thread
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), row16 = lane & 15, group = lane >> 4;
    // workgroups b, b + 8, ... share an XCD: the tiles of the same rows do
    const int xcd = blockIdx.x & 7, in_xcd = blockIdx.x >> 3;
    const int k0 = in_xcd % tiles_k * C, slice = in_xcd / tiles_k % slices, u0 = slice * per * 32;
    const int64_t walker = (int64_t)(in_xcd / tiles_k / slices) * 8 + xcd, walkers = (int64_t)(gridDim.x >> 3) / tiles_k / slices * 8;
    if (walker >= tiles_m) return;
    const int units = a.n - u0 < per * 32 ? a.n - u0 : per * 32, chunks = (units + 31) / 32;  // of this slice
    const int64_t all = ((tiles_m - 1 - walker) / walkers + 1) * chunks;

    // This thread's pieces of a stretch's weights: one column, rows kStep apart of the
    // gate's 32 and then of up's.
    constexpr int kRow = C / 8, kStep = kGateThreads / kRow;
    auto thread = [] {  // where this thread's pieces lie is worked out anew each time: held, it would cost registers
        int t = threadIdx.x;
        asm volatile("" : "+v"(t));
        return t;
    };
    u32x4 staged[kPer];
    int ahead = 0;  // the units whose weights are fetched next
    auto fetch = [&]() __attribute__((always_inline)) {
        const int t = thread(), w_row = t / kRow, room = units - 1 - ahead * 32;
        const Columns w_col = columns_of(k0 + t % kRow * 8, a.k);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int at = kPer == 1 ? w_row : j * kStep % 32 + w_row, row = kPer == 1 ? at & 31 : at;
            const bool up = kPer == 1 ? at >= 32 : j * kStep >= 32;
            const T *const w = (const T *)(up ? a.wu : a.wg) + (int64_t)(u0 + ahead * 32 + (row < room ? row : room)) * (up ? a.us : a.gs);
            staged[j] = load_columns<kShort>(w + w_col.at, w_col, a.k);
        }
        ahead = ahead + 1 < chunks ? ahead + 1 : 0;
    };
    // Columns 8 b .. + 3 of 32 become columns 4 b .. of the pair's first fragment, the next
    // four those of its second.  Unit 8 g + 4 h + t lies in row 16 h + 4 g + t: the rows that
    // a transposing read takes together, t of two g, are eight in a row, and all its
    // places are one address and constants.  Columns past k become inputs that are not
    // stored; units past n must be zero.
    auto stage = [&](char *to, int chunk) __attribute__((always_inline)) {
        const int t = thread(), w_row = t / kRow, w_piece = t % kRow;
        const int w_to = (kPer == 1 ? (w_row >> 5) * kHalf : 0) + ((w_row >> 2 & 1) * 16 + (w_row >> 3 & 3) * 4 + (w_row & 3)) * S +
                         (w_piece >> 2) * 64 + (w_piece & 3) * 8;
        if (a.k % 8) {
            const int drop = columns_of(k0 + w_piece * 8, a.k).drop & 7;
#pragma unroll
            for (int j = 0; j < kPer; ++j) staged[j] = shifted(staged[j], drop);
        }
        const int room = units - chunk * 32;
        if (room < 32)
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (((kPer == 1 ? 0 : j * kStep % 32) + w_row) % 32 >= room) staged[j] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int skip = j * kStep / 32 * kHalf + j * kStep % 32 / 2 * S;  // (units 16 on: 8 rows)
            *(u32x2 *)(to + w_to + skip) = u32x2{staged[j][0], staged[j][1]};
            *(u32x2 *)(to + w_to + skip + 32) = u32x2{staged[j][2], staged[j][3]};
        }
    };

    RawGate raw[2];
    u32x4 dz[2][2];  // gate and up, row fragments
    int64_t raw_tile = walker;
    int raw_chunk = 0;
    auto load = [&]() __attribute__((always_inline)) {  // the units after the last loaded ones
        const Columns c = columns_of(u0 + raw_chunk * 32 + group * 8, a.n);
        const int64_t m = (raw_tile < tiles_m ? raw_tile : tiles_m - 1) * 256;
        const int last = a.m - m < 256 ? (int)(a.m - m) - 1 : 255;  // rows past the end read the last one
        const char *const dh = (const char *)a.dh + m * a.dhs * 2, *const g = (const char *)a.gate + m * a.ps * 2,
                   *const u = (const char *)a.up + m * a.qs * 2;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = wave * 32 + r * 16 + row16;
            const uint32_t at = row < last ? row : last;  // (row strides are below 2^22)
            raw[r] = {load_columns<kShort>((const T *)(dh + (at * (uint32_t)a.dhs + c.at) * 2u), c, a.n),
                      load_columns<kShort>((const T *)(g + (at * (uint32_t)a.ps + c.at) * 2u), c, a.n),
                      load_columns<kShort>((const T *)(u + (at * (uint32_t)a.qs + c.at) * 2u), c, a.n)};
        }
        raw_tile += raw_chunk + 1 < chunks ? 0 : walkers;
        raw_chunk = raw_chunk + 1 < chunks ? raw_chunk + 1 : 0;
    };
    auto derive = [&](int chunk) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            float dg[8], du[8];
            gate_of<T>(raw[r], a.act, dg, du);
            dz[0][r] = pack8<T>(dg);
            dz[1][r] = pack8<T>(du);
        }
        if (u0 + chunk * 32 + 32 > a.n) {  // pieces that the rows' end cuts, and those past it
            const int drop = columns_of(u0 + chunk * 32 + group * 8, a.n).drop;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) dz[h][r] = drop >= 8 ? u32x4{0, 0, 0, 0} : shifted(dz[h][r], drop);
        }
    };

    const int columns = (group * 4 + (row16 >> 2)) * S + (row16 & 3) * 8;
    f32x4 acc[KP][2][2];  // pairs, fragments of a pair, row fragments
    int64_t m0 = walker * 256 + wave * 32 + row16;
    auto walk = [&](auto late) __attribute__((always_inline)) {
        constexpr bool kLate = decltype(late)::value;
        fetch();
        stage(lds, 0);
        fetch();
        __builtin_amdgcn_sched_barrier(0);  // (the order of the loads in flight is the loop's)
        load();
        if constexpr (!kLate) {
            derive(0);
            load();
        }
        __builtin_amdgcn_sched_barrier(0);
        int chunk = 0;
        for (int64_t q = 0; q < all; ++q) {
            step_barrier();  // these units' weights are in their buffer, and the last ones are done with
            const int next = chunk + 1 < chunks ? chunk + 1 : 0;
            stage(lds + ((q + 1) & 1) * kBuffer, next);
            fetch();
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (kLate) {
                derive(chunk);
                load();
                __builtin_amdgcn_sched_barrier(0);
            }
            if (chunk == 0)
#pragma unroll
                for (int p = 0; p < KP; ++p)
#pragma unroll
                    for (int f = 0; f < 2; ++f) acc[p][f][0] = acc[p][f][1] = f32x4{0.f, 0.f, 0.f, 0.f};
            // A weight fragment is read kAhead fragments before its products, and no earlier:
            // the registers hold no more.
            constexpr int kAll = 4 * KP, kAhead = 4;
            u32x4 w[kAhead];
            char *const at = lds + columns + (int)(q & 1) * kBuffer;
            auto read = [&](int i) __attribute__((always_inline)) {
                union {
                    s16x4 h[2];
                    u32x4 v;
                } r;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    r.h[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(at + i / (2 * KP) * kHalf + i % (2 * KP) * 32 + h * 16 * S));
                w[i % kAhead] = r.v;
            };
#pragma unroll
            for (int i = 0; i < kAhead; ++i) read(i);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < kAll; ++i) {
                const int h = i / (2 * KP), p = i / 2 % KP, f = i & 1;
#pragma unroll
                for (int r = 0; r < 2; ++r) acc[p][f][r] = mma<T>(w[i % kAhead], dz[h][r], acc[p][f][r]);
                if (i + kAhead < kAll) read(i + kAhead);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (next == 0) {
#pragma unroll
                for (int p = 0; p < KP; ++p) {
                    const int k = k0 + p * 32 + group * 8, left = a.k - k;
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = acc[p][j / 4][r][j % 4];
                        if (m0 + r * 16 >= a.m) continue;
                        if (part) {
                            float *const to = part + ((int64_t)slice * a.m + m0 + r * 16) * a.k + k;
                            if (left >= 8) {
                                store_loose(to, f32x4{v[0], v[1], v[2], v[3]});
                                store_loose(to + 4, f32x4{v[4], v[5], v[6], v[7]});
                            } else {
#pragma unroll
                                for (int j = 0; j < 8; ++j)
                                    if (j < left) to[j] = v[j];
                            }
                        } else {
                            put_piece((T *)a.dx + (m0 + r * 16) * a.dxs + k, left, pack8<T>(v));
                        }
                    }
                }
                m0 += walkers * 256;
            }
            if constexpr (!kLate) {
                derive(next);
                load();
            }
            chunk = next;
        }
    };
    if (wave & 2) walk(std::true_type{});
    else walk(std::false_type{});
}

// dx of few rows: the slices' sums, in order.
template <typename T>
__global__ __launch_bounds__(256) void dx_join_kernel(const GatedGradArgs a, const float *part, int slices) {
    const int64_t values = a.m * a.k, step = (int64_t)gridDim.x * 256;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < values; i += step) {
        float t = part[i];
#pragma unroll 8
        for (int s = 1; s < slices; ++s) t += part[(int64_t)s * values + i];
        ((T *)a.dx)[i / a.k * a.dxs + i % a.k] = (T)t;
    }
}

// Four values of dW, slots k .. k + 3 of slot n of a tile's 2 U (gate, then up),
// rounded once.
template <typename T, int U>
__device__ __forceinline__ void put_gate_dw(const GatedGradArgs &a, int n0, int n, int k, f32x4 t) {
    const bool up = n >= U;
    const int row = column_of(n0 + n - (up ? U : 0), a.n);
    if (row < 0) return;
    auto into = [&](auto *w) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = column_of(k + j, a.k);
            if (c >= 0) w[c] = (std::remove_reference_t<decltype(*w)>)(a.accumulate ? (float)w[c] + t[j] : t[j]);
        }
    };
    void *const to = up ? a.dwu : a.dwg;
    const int64_t stride = up ? a.dus : a.dgs;
    if (a.dw_f32) into((float *)to + (int64_t)row * stride);
    else into((T *)to + (int64_t)row * stride);
}
template <int U>
__device__ __forceinline__ void put_gate_db(const GatedGradArgs &a, int n0, int n, float t) {
    const bool up = n >= U;
    const int c = column_of(n0 + n - (up ? U : 0), a.n);
    float *const to = up ? a.dbu : a.dbg;
    if (c >= 0) to[c] = a.accumulate ? to[c] + t : t;
}

// dW of U hidden units (2 U rows of gate and up) by KT inputs, and the biases'
// gradients, over a share of the rows, 64 or 32 a step.  Each thread turns the pieces of
// dh, g and u that it loaded a step ahead into dg and du, adds its columns up for
// the biases, and lays them and x into LDS tiles, one of two sets; then each wave
// adds the step's product to its part of dW, which stays in registers to the end
// (4 x 2 waves over 2 U x KT).  Both operands are read transposed.  Between two
// barriers half of the waves multiply this step first and prepare the next one then,
// the others the other way around.  dW and db leave as one partial per workgroup, joined
// in a fixed order by gated_join_kernel; a workgroup alone with its tile writes them
// itself.
//
// kDx: the tile holds all units and inputs, and dx is made here too, so that dh, g and
// u are read once.  Both weights lie in LDS, their columns dealt as in gated_dx_kernel; a
// wave has 16 of a step's rows and half of the inputs, and adds up in that kernel's
// order, so that dx is the same with and without the weights' gradients.  A step's dx is
// stored after the next step's loads have come and before those of the one after are
// asked for: a wait for loads never waits for young stores.
// (2^18 rows, 64 -> 128: 57 us and the join 6, 123 in two passes; 128 -> 128 87 and 154;
// 65537 rows, 35 -> 93 f16 28 + 5, 48.)
//
// 2^18 rows, 256 -> 512 bf16 228 us without dx, and the join 17; its bytes at the copy's
// rate take 179: bound by memory and, in part, by the slopes (VALU 52 %, matrix units 26 %).
template <typename T, int U, int KT, bool kShort, bool kDx>
__global__ __launch_bounds__(kGateThreads) void gated_dw_kernel(const GatedGradArgs a, float *part) {
    constexpr int R = gate_rows(U, KT), NT = 2 * U, FN = NT / 64, FK = KT / 32;  // fragments of a wave
    constexpr int PN = U / 8, PK = KT / 8;                               // pieces of a row
    constexpr int LN = R * PN / kGateThreads, LK = R * PK / kGateThreads;  // pieces of a thread
    constexpr int kBuffer = R * (NT + KT) * 2;
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wn = wave >> 1, wk = wave & 1;
    const int n0 = blockIdx.y * U, k0 = blockIdx.z * KT;
    f32x4 acc[FN][FK];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FK; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    float dbg[8] = {}, dbu[8] = {};
    RawGate raw[LN];
    u32x4 nx[LK];
    const int64_t steps = (a.m + R - 1) / R, by = gridDim.x;
    const int rn = threadIdx.x / PN, rk = threadIdx.x / PK;  // this thread's first rows in a step
    const Columns cn = columns_of(n0 + threadIdx.x % PN * 8, a.n), ck = columns_of(k0 + threadIdx.x % PK * 8, a.k);
    // Bytes of this thread's pieces from a step's first row (row strides are below 2^22).
    uint32_t at_dh[LN], at_g[LN], at_u[LN], at_x[LK];
    auto rows_of = [&](int last) __attribute__((always_inline)) {  // rows past the end read the last one
#pragma unroll
        for (int i = 0; i < LN; ++i) {
            const int at = rn + i * (kGateThreads / PN), r = at < last ? at : last;
            at_dh[i] = ((uint32_t)r * (uint32_t)a.dhs + cn.at) * 2u, at_g[i] = ((uint32_t)r * (uint32_t)a.ps + cn.at) * 2u,
            at_u[i] = ((uint32_t)r * (uint32_t)a.qs + cn.at) * 2u;
        }
#pragma unroll
        for (int i = 0; i < LK; ++i) {
            const int at = rk + i * (kGateThreads / PK), r = at < last ? at : last;
            at_x[i] = ((uint32_t)r * (uint32_t)a.xs + ck.at) * 2u;
        }
    };
    rows_of(R - 1);
    auto fetch = [&](int64_t step) __attribute__((always_inline)) {  // past the last step it is read again
        const int64_t m = (step < steps ? step : steps - 1) * R;
        if (a.m - m < R) rows_of((int)(a.m - m) - 1);
        const char *const dh = (const char *)a.dh + m * a.dhs * 2, *const g = (const char *)a.gate + m * a.ps * 2,
                   *const u = (const char *)a.up + m * a.qs * 2, *const x = (const char *)a.x + m * a.xs * 2;
#pragma unroll
        for (int i = 0; i < LN; ++i)
            raw[i] = {load_columns<kShort>((const T *)(dh + at_dh[i]), cn, a.n), load_columns<kShort>((const T *)(g + at_g[i]), cn, a.n),
                      load_columns<kShort>((const T *)(u + at_u[i]), cn, a.n)};
        if (a.dwg)
#pragma unroll
            for (int i = 0; i < LK; ++i) nx[i] = load_columns<kShort>((const T *)(x + at_x[i]), ck, a.k);
    };
    const int to_dz = tile_at<NT>(rn, threadIdx.x % PN), to_x = R * NT * 2 + tile_at<KT>(rk, threadIdx.x % PK);  // (rows 16 apart lie alike)
    auto prepare = [&](int64_t step, char *tiles) __attribute__((always_inline)) {
        const bool whole = (step + 1) * R <= a.m;
        if (a.dwg) {
            if (a.k % 8)  // pieces that the rows' end cuts: the slots of the piece before
#pragma unroll
                for (int i = 0; i < LK; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) nx[i][j] &= 2 * j >= ck.drop ? ~0u : 2 * j + 1 >= ck.drop ? 0xFFFF0000u : 0u;
            if (!whole)
#pragma unroll
                for (int i = 0; i < LK; ++i)
                    if (step * R + rk + i * (kGateThreads / PK) >= a.m) nx[i] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < LK; ++i) *(u32x4 *)(tiles + to_x + i * (kGateThreads / PK) * (KT * 2)) = nx[i];
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < LN; ++i) {
            float dg[8], du[8];
            gate_of<T>(raw[i], a.act, dg, du);
            if (!whole || a.n % 8 || n0 + U > a.n) {
                const int drop = step * R + rn + i * (kGateThreads / PN) < a.m ? cn.drop : 8;
#pragma unroll
                for (int j = 0; j < 8; ++j) dg[j] = j < drop ? 0.f : dg[j], du[j] = j < drop ? 0.f : du[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) dbg[j] += dg[j], dbu[j] += du[j];
            *(u32x4 *)(tiles + to_dz + i * (kGateThreads / PN) * (NT * 2)) = pack8<T>(dg);
            *(u32x4 *)(tiles + (to_dz ^ (PN << 4)) + i * (kGateThreads / PN) * (NT * 2)) = pack8<T>(du);
            __builtin_amdgcn_sched_barrier(0);  // one piece's values at a time: the registers hold no more
        }
    };
    // dx of a step's rows.
    constexpr int P = kDx ? KT / 64 : 1;  // pairs of input fragments of a wave
    static_assert(!kDx || R == 64);
    char *const weights = lds + 2 * kBuffer;
    const int columns_w = columns_base<KT>(lane);
    u32x4 dx[P];
    if constexpr (kDx)
        for (int i = threadIdx.x; i < NT * PK; i += kGateThreads) {
            const int slot = i / PK, w_piece = i % PK, unit = slot < U ? slot : slot - U, row = unit < a.n ? unit : 0;
            const T *const w = slot < U ? (const T *)a.wg + row * a.gs : (const T *)a.wu + row * a.us;
            const Columns c = columns_of(w_piece * 8, a.k);
            u32x4 v = shifted(load_columns<kShort>(w + c.at, c, a.k), c.drop & 7);
            if (unit >= a.n) v = u32x4{0, 0, 0, 0};
            const int to = tile_at<KT>(slot, (w_piece >> 2) * 4 + ((w_piece & 3) >> 1)) + (w_piece & 1) * 8;
            *(u32x2 *)(weights + to) = u32x2{v[0], v[1]};
            *(u32x2 *)(weights + (to ^ 32)) = u32x2{v[2], v[3]};
        }
    auto spread = [&](int turn) __attribute__((always_inline)) {
        if constexpr (!kDx) return;
        f32x4 d[P][2];
#pragma unroll
        for (int p = 0; p < P; ++p) d[p][0] = d[p][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        const int z_at = turn * kBuffer + tile_at<NT>((wave & 3) * 16 + (lane & 15), lane >> 4);
#pragma unroll
        for (int s = 0; s < NT / 32; ++s) {  // 32 units of gate, then of up
            const int slot = s / 2 * 32 + s % 2 * U;
            u32x4 z = *(const u32x4 *)(lds + (z_at ^ (slot << 1)));
            if (a.n % 8 && s / 2 * 32 + 32 > a.n) z = shifted(z, columns_of(s / 2 * 32 + (lane >> 4) * 8, a.n).drop & 7);  // (zeros past the units)
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int f = 0; f < 2; ++f)
                    d[p][f] = mma<T>(columns_at<KT>(weights, columns_w, slot, ((wave >> 2) * P + p) * 2 + f), z, d[p][f]);
        }
#pragma unroll
        for (int p = 0; p < P; ++p) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = d[p][j / 4][j % 4];
            dx[p] = pack8<T>(v);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    auto flush = [&](int64_t step) __attribute__((always_inline)) {
        if constexpr (!kDx) return;
        const int64_t m = step * R + (wave & 3) * 16 + (lane & 15);
        if (m >= a.m) return;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int k = ((wave >> 2) * P + p) * 32 + (lane >> 4) * 8;
            put_piece((T *)a.dx + m * a.dxs + k, a.k - k, dx[p]);
        }
    };
    const int columns_n = columns_base<NT>(lane) ^ (2 * wn * FN << 4), columns_k = columns_base<KT>(lane) ^ (2 * wk * FK << 4);
    auto multiply = [&](int turn) __attribute__((always_inline)) {
        if (!a.dwg) return;
        const int at_n = columns_n + turn * kBuffer, at_k = columns_k + turn * kBuffer;
#pragma unroll
        for (int m = 0; m < R; m += 32) {
            u32x4 dzf[FN];
#pragma unroll
            for (int i = 0; i < FN; ++i) dzf[i] = columns_at<NT>(lds, at_n, m, i);
#pragma unroll
            for (int j = 0; j < FK; ++j) {
                const u32x4 xf = columns_at<KT>(lds + R * NT * 2, at_k, m, j);
#pragma unroll
                for (int i = 0; i < FN; ++i) acc[i][j] = mma<T>(xf, dzf[i], acc[i][j]);
            }
            // x's fragments are read (two reads each) two before their products
            __builtin_amdgcn_sched_group_barrier(0x100, 2 * FN + 4, 0);
#pragma unroll
            for (int j = 0; j < FK - 2; ++j) {
                __builtin_amdgcn_sched_group_barrier(0x008, FN, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x008, 2 * FN, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto walk = [&](auto late) __attribute__((always_inline)) {
        fetch(blockIdx.x);
        prepare(blockIdx.x, lds);
        fetch(blockIdx.x + by);
        int turn = 0;
        int64_t last = blockIdx.x;
        for (int64_t step = blockIdx.x; step < steps; step += by, turn ^= 1) {
            step_barrier();  // this step's tiles are whole, and the last step's are done with
            if constexpr (!decltype(late)::value) multiply(turn), spread(turn);
            prepare(step + by, lds + (turn ^ 1) * kBuffer);
            if constexpr (!decltype(late)::value) flush(step);
            else if (step != blockIdx.x) flush(step - by);
            fetch(step + 2 * by);
            if constexpr (decltype(late)::value) multiply(turn), spread(turn);
            last = step;
        }
        if constexpr (decltype(late)::value) flush(last);
    };
    if (wave & 2) walk(std::true_type{});
    else walk(std::false_type{});

    // Partials: dW as fragments, [tile][workgroup][NT x KT], then db, [unit tile][workgroup][NT].
    const int tile = blockIdx.y * gridDim.z + blockIdx.z;
    const bool alone = gridDim.x == 1;
    if (a.dwg) {
        float *p = part + ((int64_t)tile * gridDim.x + blockIdx.x) * (NT * KT);
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FK; ++j) {
                const int fn = wn * FN + i, fk = wk * FK + j;
                if (alone) put_gate_dw<T, U>(a, n0, fn * 16 + (lane & 15), k0 + fk * 16 + (lane >> 4) * 4, acc[i][j]);
                else *(f32x4 *)(p + (fn * (KT / 16) + fk) * 256 + lane * 4) = acc[i][j];
            }
    }
    if (a.dbg && blockIdx.z == 0) {
        float *const sums = (float *)lds;  // [512 / PN][U], for the gate and then for up
        float *p = part + (a.dwg ? (int64_t)gridDim.y * gridDim.z * gridDim.x * (NT * KT) : 0) +
                   ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * NT;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            __syncthreads();
#pragma unroll
            for (int j = 0; j < 8; ++j) sums[threadIdx.x * 8 + j] = half ? dbu[j] : dbg[j];
            __syncthreads();
            for (int n = threadIdx.x; n < U; n += kGateThreads) {
                float t = 0.f;
                for (int r = 0; r < kGateThreads / PN; ++r) t += sums[r * U + n];
                if (alone) put_gate_db<U>(a, n0, half * U + n, t);
                else p[half * U + n] = t;
            }
        }
    }
}

// Four joined values, quad `local` of the tiles' dW or of the db, to their places.
template <typename T, int U>
__device__ __forceinline__ void gated_join_put(const GatedGradArgs &a, f32x4 t, int64_t local, int64_t per, bool weights, int kt, int nz) {
    const int tile = (int)(local / per), e = (int)(local % per);
    if (weights) {
        const int frag = e / 64, l = e % 64;
        put_gate_dw<T, U>(a, tile / nz * U, frag / (kt / 16) * 16 + (l & 15), tile % nz * kt + frag % (kt / 16) * 16 + (l >> 4) * 4, t);
    } else {
        for (int j = 0; j < 4; ++j) put_gate_db<U>(a, tile * U, e * 4 + j, t[j]);
    }
}

// dW = (dW +) the partials' sum, rounded once; db alike.  A workgroup takes 16
// groups of four values; 32 threads share the partials of each, and their sums
// are added in order, eight and then four.
template <typename T, int U>
__global__ __launch_bounds__(512) void gated_join_kernel(const float *part, int parts, int kt, int ny, int nz, GatedGradArgs a) {
    __shared__ f32x4 lds[32][16];
    constexpr int NT = 2 * U;
    const int slot = threadIdx.x & 15, share = threadIdx.x >> 4;
    const int64_t quads = a.dwg ? (int64_t)ny * nz * NT * kt / 4 : 0, all = quads + (a.dbg ? ny * NT / 4 : 0);
    const int64_t q = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 16 + slot;
    const int64_t per = q < quads ? NT * kt / 4 : NT / 4;      // quads of a partial
    const int64_t local = q < quads ? q : q - quads;
    const float *p = part + (q < quads ? 0 : quads * 4 * parts) + (local / per * per * parts + local % per) * 4;
    f32x4 t = {0.f, 0.f, 0.f, 0.f};
    if (q < all)
#pragma unroll 8
        for (int i = share; i < parts; i += 32) t += *(const f32x4 *)(p + i * per * 4);
    lds[share][slot] = t;
    __syncthreads();
    if (share < 4) {
        t = lds[share * 8][slot];
#pragma unroll
        for (int i = 1; i < 8; ++i) t += lds[share * 8 + i][slot];
    }
    __syncthreads();
    if (share < 4) lds[share][slot] = t;
    __syncthreads();
    if (share || q >= all) return;
    for (int i = 1; i < 4; ++i) t += lds[i][slot];
    gated_join_put<T, U>(a, t, local, per, q < quads, kt, nz);
}
// The same of few partials, a thread a group of four values (24 partials of 256 -> 512,
// 4096 rows: 58.6 us with dW and dx, 63.8 with the other join; 256 of 64 -> 128, 2^18 rows: 69
// and 62).
constexpr int kFewParts = 64;
template <typename T, int U>
__global__ __launch_bounds__(256) void gated_join_few_kernel(const float *part, int parts, int kt, int ny, int nz, GatedGradArgs a) {
    constexpr int NT = 2 * U;
    const int64_t quads = a.dwg ? (int64_t)ny * nz * NT * kt / 4 : 0, all = quads + (a.dbg ? ny * NT / 4 : 0);
    const int64_t q = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    if (q >= all) return;
    const int64_t per = q < quads ? NT * kt / 4 : NT / 4, local = q < quads ? q : q - quads;
    const float *p = part + (q < quads ? 0 : quads * 4 * parts) + (local / per * per * parts + local % per) * 4;
    f32x4 t = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int i = 0; i < parts; ++i) t += *(const f32x4 *)(p + i * per * 4);
    gated_join_put<T, U>(a, t, local, per, q < quads, kt, nz);
}

template <typename T, int KP, bool kShort = false>
hipError_t gated_dx_launch(const GatedGradArgs &a, const GatedGradPlan &p, float *part, hipStream_t stream) {
    const auto kernel = gated_dx_kernel<T, KP, kShort>;
    const int bytes = 2 * 2 * 32 * (KP * 32 * 2 + 32), tiles_k = (int)div_up(a.k, KP * 32);
    if (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    const int64_t tiles_m = div_up(a.m, 256), most = kCus * (KP == 2 ? 2 : 1) / (tiles_k * p.slices);  // (registers of one or two workgroups a CU)
    int64_t walkers = most < tiles_m ? most : tiles_m;
    walkers = div_up(walkers < 1 ? 1 : walkers, 8) * 8;  // whole rounds over the XCDs
    part = p.slices > 1 ? part : nullptr;
    kernel<<<dim3((unsigned)(walkers * tiles_k * p.slices)), kGateThreads, bytes, stream>>>(a, tiles_k, tiles_m, p.slices, p.per, part);
    if (part) {
        const int64_t groups = div_up(a.m * a.k, 256);
        dx_join_kernel<T><<<dim3((unsigned)(groups < kCus * 8 ? groups : kCus * 8)), 256, 0, stream>>>(a, part, p.slices);
    }
    return hipGetLastError();
}

template <typename T, int U, int KT, bool kShort = false>
hipError_t gated_dw_launch(const GatedGradArgs &a, const GatedGradPlan &p, float *part, hipStream_t stream) {
    auto kernel = gated_dw_kernel<T, U, KT, kShort, false>;
    int bytes = 2 * gate_rows(U, KT) * (2 * U + KT) * 2;
    if constexpr (U * KT <= 128 * 128)
        if (p.together) kernel = gated_dw_kernel<T, U, KT, kShort, true>, bytes += 2 * U * KT * 2;
    if (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    kernel<<<dim3((unsigned)p.parts, (unsigned)p.ny, (unsigned)p.nz), kGateThreads, bytes, stream>>>(a, part);
    return hipGetLastError();
}

template <typename T>
hipError_t gated_grad_run(const GatedGradArgs &a, const GatedGradPlan &p, float *part, hipStream_t stream) {
    hipError_t e = hipSuccess;
    if (a.m > 0 && (a.dwg || a.dbg)) {
        if (a.n < 8 || a.k < 8) e = gated_dw_launch<T, 64, 64, true>(a, p, part, stream);
        else if (p.units == 128) e = p.kt == 64 ? gated_dw_launch<T, 128, 64>(a, p, part, stream)
                              : p.kt == 128 ? gated_dw_launch<T, 128, 128>(a, p, part, stream)
                                            : gated_dw_launch<T, 128, 256>(a, p, part, stream);
        else e = p.kt == 64 ? gated_dw_launch<T, 64, 64>(a, p, part, stream)
               : p.kt == 128 ? gated_dw_launch<T, 64, 128>(a, p, part, stream)
                             : gated_dw_launch<T, 64, 256>(a, p, part, stream);
        if (e != hipSuccess) return e;
    }
    if ((a.dwg || a.dbg) && !(a.m > 0 && p.parts == 1)) {
        const int64_t quads = (a.dwg ? (int64_t)p.ny * p.nz * 2 * p.units * p.kt : 0) / 4 + (a.dbg ? p.ny * p.units / 2 : 0);
        const int parts = a.m > 0 ? p.parts : 0;
        if (parts <= kFewParts) {
            if (p.units == 128) gated_join_few_kernel<T, 128><<<grid_of(div_up(quads, 256)), 256, 0, stream>>>(part, parts, p.kt, p.ny, p.nz, a);
            else gated_join_few_kernel<T, 64><<<grid_of(div_up(quads, 256)), 256, 0, stream>>>(part, parts, p.kt, p.ny, p.nz, a);
        } else if (p.units == 128) gated_join_kernel<T, 128><<<grid_of(div_up(quads, 16)), 512, 0, stream>>>(part, parts, p.kt, p.ny, p.nz, a);
        else gated_join_kernel<T, 64><<<grid_of(div_up(quads, 16)), 512, 0, stream>>>(part, parts, p.kt, p.ny, p.nz, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (!a.dx || a.m == 0 || p.together) return hipSuccess;
    float *const dx_part = (float *)((char *)part + p.dx_at);
    if (a.n < 8 || a.k < 8) return gated_dx_launch<T, 2, true>(a, p, dx_part, stream);
    return p.kp == 2 ? gated_dx_launch<T, 2>(a, p, dx_part, stream)
           : p.kp == 4 ? gated_dx_launch<T, 4>(a, p, dx_part, stream)
                       : gated_dx_launch<T, 8>(a, p, dx_part, stream);
}

}  // namespace
}  // namespace res
}  // namespace hg
