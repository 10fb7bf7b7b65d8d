// Backward of y = act(x W^T + b) + r on the matrix cores; the sources that
// include this instantiate one operand type each.
//
//   dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum over rows of dz
//
// dz is rounded to the operands' type where it enters a product, as products of
// 16-bit operands need; db sums it unrounded.
#pragma once

#include "linear_grad.h"

namespace hg {
namespace res {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kGradThreads = 512;

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

// Pieces of dz and x are cut as Columns has it, slots that do not count zeroed
// where a piece is used; the join knows which column a slot stands for.
// The piece at p; kShort: rows may be shorter than a piece (the narrowest tiles').
template <bool kShort, typename T>
__device__ __forceinline__ u32x4 load_columns(const T *p, Columns c, int width) {
    if (!kShort || width >= 8) return load_loose<u32x4>(p);
    return c.drop ? u32x4{0, 0, 0, 0} : load_short(p, width);
}

// One piece of dz: 8 values from dy and z.
template <typename T, typename D>
struct RawDz {
    u32x4 dy[sizeof(D) == 4 ? 2 : 1], pre;
};
// dy and pre: this piece's row and column in each.
template <bool kShort, typename T, typename D>
__device__ __forceinline__ RawDz<T, D> load_dz(const GradArgs &a, const D *dy, const T *pre, Columns c) {
    RawDz<T, D> v;
    if constexpr (sizeof(D) == 4) {
        if (!kShort || a.n >= 8) {
            v.dy[0] = load_loose<u32x4>(dy), v.dy[1] = load_loose<u32x4>(dy + 4);
        } else {
            uint32_t t[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) t[j] = __float_as_uint(dy[j < a.n ? j : a.n - 1]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v.dy[j / 4][j % 4] = c.drop == 0 && j < a.n ? t[j] : 0u;
        }
    } else {
        v.dy[0] = load_columns<kShort>(dy, c, a.n);
    }
    v.pre = u32x4{0, 0, 0, 0};
    if (a.act != HG_ACT_NONE) v.pre = load_columns<kShort>(pre, c, a.n);
    return v;
}
template <typename T, typename D>
__device__ __forceinline__ void dz_of(const RawDz<T, D> &v, int act, int drop, float (&dz)[8]) {
    typedef T T8 __attribute__((ext_vector_type(8)));
    const T8 z = __builtin_bit_cast(T8, v.pre);
    if constexpr (sizeof(D) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) dz[j] = __uint_as_float(v.dy[j / 4][j % 4]);
    } else {
        const T8 d = __builtin_bit_cast(T8, v.dy[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dz[j] = (float)d[j];
    }
    auto times = [&](auto kind) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = slope((float)z[j], decltype(kind)::value);
            dz[j] = decltype(kind)::value == HG_ACT_RELU && s == 0.f ? 0.f : dz[j] * s;
        }
    };
    if (act == HG_ACT_RELU) times(std::integral_constant<int, HG_ACT_RELU>{});
    else if (act == HG_ACT_SILU) times(std::integral_constant<int, HG_ACT_SILU>{});
    else if (act == HG_ACT_GELU_TANH) times(std::integral_constant<int, HG_ACT_GELU_TANH>{});
    if (drop > 0)
#pragma unroll
        for (int j = 0; j < 8; ++j) dz[j] = j < drop ? 0.f : dz[j];
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

// W^T of rows n < NT, columns k < KT in LDS as fragments for dx: block
// (pair s of 16-column fragments, fragment f, step u of 32 rows n), lane (i, g):
// column 32 s + (i / 4) 8 + 4 f + i % 4, rows 32 u + 8 g .. + 7.  A thread turns
// 8 x 8 values: eight pieces of eight rows, two rows' halves merged at a time.
template <typename T, int NT, int KT>
__device__ __forceinline__ void stage_wt(const GradArgs &a, u32x4 *wt) {
    for (int b = threadIdx.x; b < NT / 8 * (KT / 8); b += kGradThreads) {
        const int k8 = b % (KT / 8), n8 = b / (KT / 8);
        u32x4 row[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int n = column_of(n8 * 8 + r, a.n);
            const T *const w = (const T *)a.w + (int64_t)(n < 0 ? 0 : n) * a.ws;
            const Columns c = columns_of(k8 * 8, a.k);
            row[r] = a.k < 8 ? load_short(w, a.k) : shifted(load_loose<u32x4>(w + c.at), c.drop);
            if (n < 0 || c.drop >= 8) row[r] = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            u32x4 v;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const uint32_t lo = row[2 * h][j / 2], hi = row[2 * h + 1][j / 2];
                v[h] = j & 1 ? (lo >> 16) | (hi & 0xFFFF0000u) : (lo & 0xFFFFu) | (hi << 16);
            }
            const int i = (k8 & 3) * 4 + (j & 3), f = j >> 2, s = k8 >> 2, u = n8 >> 2, g = n8 & 3;
            wt[((s * 2 + f) * (NT / 32) + u) * 64 + g * 16 + i] = v;
        }
    }
}

// Four values of dW, slots k .. k + 3 of slot n, rounded once.
template <typename T>
__device__ __forceinline__ void put_dw(const GradArgs &a, int n, int k, f32x4 t) {
    const int row = column_of(n, a.n);
    if (row < 0) return;
    auto into = [&](auto *w) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = column_of(k + j, a.k);
            if (c >= 0) w[c] = (std::remove_reference_t<decltype(*w)>)(a.accumulate ? (float)w[c] + t[j] : t[j]);
        }
    };
    if (a.dw_f32) into((float *)a.dw + (int64_t)row * a.dws);
    else into((T *)a.dw + (int64_t)row * a.dws);
}
__device__ __forceinline__ void put_db(const GradArgs &a, int n, float t) {
    const int c = column_of(n, a.n);
    if (c >= 0) a.db[c] = a.accumulate ? a.db[c] + t : t;
}

// The whole backward of up to NT outputs by KT inputs in one pass over the rows:
// dy, z and x are read once, dz lives in LDS only.  A workgroup a CU walks steps
// of R rows.  In a step each thread turns the pieces it loaded a step ahead into
// dz (adding its columns up for db) and lays dz and x into LDS; then each wave
// adds the step's product to its part of dW, which stays in registers to the
// end (4 x 2 waves over NT x KT), and makes one 32 x 32 block of dx from dz and
// the W^T fragments held in LDS.  dW and db leave as one partial per workgroup,
// joined in a fixed order by grad_join_kernel; a workgroup alone with its tile
// (few rows) writes them itself.
// Wider layers: tiles of NT x KT (blockIdx.y over outputs, .z over inputs)
// make dW and db alone, and the first column of tiles writes dz for dx's sake;
// each column of tiles reads dy and z and works out the slopes again.
// 2^18 x 256 x 256 bf16 with SiLU: 150 us with its join, 3.6 TB/s: W^T, dz and x fill
// the LDS and the products' sums the registers, so one step's loads are all that
// is on its way, and a step's products and its slope's arithmetic are not hidden
// in full.  2^18 x 128 x 128: 62 us, 4.3 TB/s.
template <typename T, typename D, int NT, int KT, bool kDx>
__global__ __launch_bounds__(kGradThreads) void grad_kernel(const GradArgs a, float *part, T *dz_out) {
    constexpr int R = grad_rows(NT, KT), FN = NT / 64, FK = KT / 32;  // fragments of a wave: FN outputs x FK inputs
    constexpr int PN = NT / 8, PK = KT / 8;                       // pieces of a row
    constexpr int LN = R * PN / kGradThreads, LK = R * PK / kGradThreads;  // pieces of a thread
    extern __shared__ __attribute__((aligned(16))) char lds[];
    char *const dzt = lds, *const xt = lds + R * NT * 2;
    u32x4 *const wt = (u32x4 *)(lds + R * (NT + KT) * 2);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wn = wave >> 1, wk = wave & 1;

    const int n0 = blockIdx.y * NT, k0 = blockIdx.z * KT;
    const bool store_dz = !kDx && dz_out && blockIdx.z == 0;
    // Where this thread's pieces lie is worked out anew in every step: held, it
    // would cost registers that the widest tile does not have, and a spill's
    // reload waits for every store and load before it.
    auto thread = [] {
        int t = threadIdx.x;
        asm volatile("" : "+v"(t));
        return t;
    };
    if constexpr (kDx) stage_wt<T, NT, KT>(a, wt);

    f32x4 acc[FN][FK];
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FK; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    float db[8] = {};

    RawDz<T, D> nz[LN];
    u32x4 nx[LK];
    // Addresses: a uniform base for the step and i, and this thread's 32-bit offset
    // of its row and column in a step (row strides are below 2^22).
    auto fetch = [&](int64_t step) {
        const int t = thread(), rn = t / PN, rk = t / PK;
        const Columns cn = columns_of(n0 + t % PN * 8, a.n), ck = columns_of(k0 + t % PK * 8, a.k);
        const int64_t m = step * R;
        const int last = a.m - m < R ? (int)(a.m - m) - 1 : R - 1;  // rows past the end read the last one
#pragma unroll
        for (int i = 0; i < LN; ++i) {
            const int skip = i * (kGradThreads / PN), room = last - skip < 0 ? 0 : last - skip;  // (a base stays inside)
            const int64_t base = m + (last - skip < 0 ? last : skip);
            const int r = rn < room ? rn : room;
            nz[i] = load_dz<NT == 64, T, D>(a, (const D *)a.dy + base * a.dys + (uint32_t)(r * (int)a.dys + cn.at),
                                  (const T *)a.pre + base * a.ps + (uint32_t)(r * (int)a.ps + cn.at), cn);
        }
        if (a.dw)
#pragma unroll
            for (int i = 0; i < LK; ++i) {
                const int skip = i * (kGradThreads / PK), room = last - skip < 0 ? 0 : last - skip;
                const int64_t base = m + (last - skip < 0 ? last : skip);
                const int r = rk < room ? rk : room;
                nx[i] = load_columns<KT == 64>((const T *)a.x + base * a.xs + (uint32_t)(r * (int)a.xs + ck.at), ck, a.k);
            }
    };

    // dx of a step is stored in the next one, between the use of the loads that
    // were made a step ahead and the next such loads: a wait for those loads then
    // has no younger stores to wait for.
    constexpr int kBlocks = KT / 32 * (R / 32) / 8;  // 32 x 32 blocks of dx a wave makes
    u32x4 late[kBlocks][2];
    auto store_late = [&](int64_t step) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
            const int block = wave + b * 8, k = block % (KT / 32) * 32 + (lane >> 4) * 8, left = a.k - k;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = block / (KT / 32) * 32 + r * 16 + (lane & 15);
                T *const p = (T *)a.dx + step * R * a.dxs + (uint32_t)(row * (int)a.dxs + k);
                if (step * R + row < a.m) {
                    if (left >= 8) store_loose<u32x4>(p, late[b][r]);
                    else
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j < left) p[j] = __builtin_bit_cast(T, (uint16_t)(late[b][r][j / 2] >> (16 * (j & 1))));
                }
            }
        }
    };

    const int64_t steps = (a.m + R - 1) / R;
    if (blockIdx.x < steps) fetch(blockIdx.x);
    for (int64_t step = blockIdx.x; step < steps; step += gridDim.x) {
        const bool whole = (step + 1) * R <= a.m;
        const int t = thread();
        const Columns cn = columns_of(n0 + t % PN * 8, a.n), ck = columns_of(k0 + t % PK * 8, a.k);
        __syncthreads();  // the last step's reads of the tiles are done
#pragma unroll
        for (int i = 0; i < LN; ++i) {
            const int r = t / PN + i * (kGradThreads / PN);
            float dz[8];
            dz_of<T, D>(nz[i], a.act, whole || step * R + r < a.m ? cn.drop : 8, dz);
#pragma unroll
            for (int j = 0; j < 8; ++j) db[j] += dz[j];
            *(u32x4 *)(dzt + tile_at<NT>(r, t % PN)) = pack8<T>(dz);
            if (store_dz && step * R + r < a.m) {
                T *const p = dz_out + (step * R + r) * a.n + cn.at;
                const int have = a.n < 8 ? a.n : 8;
                if (cn.drop == 0) put(p, have, rounded<8, T>(dz));
                else
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (j >= cn.drop) p[j] = (T)dz[j];
            }
        }
        if (a.dw)
#pragma unroll
            for (int i = 0; i < LK; ++i) {
                const int r = t / PK + i * (kGradThreads / PK);
                u32x4 v = nx[i];
                if (ck.drop > 0)
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[j] &= 2 * j >= ck.drop ? ~0u : 2 * j + 1 >= ck.drop ? 0xFFFF0000u : 0u;
                if (!whole && step * R + r >= a.m) v = u32x4{0, 0, 0, 0};
                *(u32x4 *)(xt + tile_at<KT>(r, t % PK)) = v;
            }
        if (kDx && step != blockIdx.x) store_late(step - gridDim.x);
        if (step + gridDim.x < steps) fetch(step + gridDim.x);
        __syncthreads();
        if (a.dw) {
#pragma unroll
            for (int m = 0; m < R; m += 32) {
                u32x4 dzf[FN];
#pragma unroll
                for (int i = 0; i < FN; ++i) dzf[i] = tile_columns<NT>(dzt, m, wn * FN + i, lane);
#pragma unroll
                for (int j = 0; j < FK; ++j) {
                    const u32x4 xf = tile_columns<KT>(xt, m, wk * FK + j, lane);
#pragma unroll
                    for (int i = 0; i < FN; ++i) acc[i][j] = mma<T>(xf, dzf[i], acc[i][j]);
                }
            }
        }
        if constexpr (kDx) {
            const int row = lane & 15, g = lane >> 4;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const int block = wave + b * 8, s = block % (KT / 32), m = block / (KT / 32) * 32;
                f32x4 d[2][2] = {};
#pragma unroll
                for (int u = 0; u < NT / 32; ++u) {
                    u32x4 z[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) z[r] = *(const u32x4 *)(dzt + tile_at<NT>(m + r * 16 + row, u * 4 + g));
#pragma unroll
                    for (int f = 0; f < 2; ++f) {
                        const u32x4 w = wt[((s * 2 + f) * (NT / 32) + u) * 64 + lane];
#pragma unroll
                        for (int r = 0; r < 2; ++r) d[f][r] = mma<T>(w, z[r], d[f][r]);
                    }
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float v[8] = {d[0][r][0], d[0][r][1], d[0][r][2], d[0][r][3],
                                        d[1][r][0], d[1][r][1], d[1][r][2], d[1][r][3]};
                    late[b][r] = pack8<T>(v);
                }
            }
        }
    }
    if (kDx && blockIdx.x < steps) store_late(blockIdx.x + (steps - 1 - blockIdx.x) / gridDim.x * gridDim.x);

    // Partials: dW as fragments, [tile][workgroup][NT x KT], then db, [output tile][workgroup][NT].
    const int tile = blockIdx.y * gridDim.z + blockIdx.z;
    const bool alone = gridDim.x == 1;
    if (a.dw) {
        float *p = part + ((int64_t)tile * gridDim.x + blockIdx.x) * (NT * KT);
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FK; ++j) {
                const int fn = wn * FN + i, fk = wk * FK + j;
                if (alone) put_dw<T>(a, n0 + fn * 16 + (lane & 15), k0 + fk * 16 + (lane >> 4) * 4, acc[i][j]);
                else *(f32x4 *)(p + (fn * (KT / 16) + fk) * 256 + lane * 4) = acc[i][j];
            }
    }
    if (a.db && blockIdx.z == 0) {
        float *const sums = (float *)lds;  // [512 / PN][NT]
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[threadIdx.x * 8 + j] = db[j];
        __syncthreads();
        float *p = part + (a.dw ? (int64_t)gridDim.y * gridDim.z * gridDim.x * (NT * KT) : 0) +
                   ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * NT;
        for (int n = threadIdx.x; n < NT; n += kGradThreads) {
            float t = 0.f;
            for (int r = 0; r < kGradThreads / PN; ++r) t += sums[r * NT + n];
            if (alone) put_db(a, n0 + n, t);
            else p[n] = t;
        }
    }
}

// dW = (dW +) the partials' sum, rounded once; db alike.  A workgroup takes 16
// groups of four values; 32 threads share the partials of each, and their sums
// are added in order, eight and then four.
template <typename T>
__global__ __launch_bounds__(512) void grad_join_kernel(const float *part, int parts, int nt, int kt, int ny, int nz, GradArgs a) {
    __shared__ f32x4 lds[32][16];
    const int slot = threadIdx.x & 15, share = threadIdx.x >> 4;
    const int64_t quads = a.dw ? (int64_t)ny * nz * nt * kt / 4 : 0, all = quads + (a.db ? ny * nt / 4 : 0);
    const int64_t q = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 16 + slot;
    const int64_t per = q < quads ? nt * kt / 4 : nt / 4;      // quads of a partial
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
    if (q < quads) {
        const int tile = (int)(local / per), e = (int)(local % per), frag = e / 64, l = e % 64;
        put_dw<T>(a, tile / nz * nt + frag / (kt / 16) * 16 + (l & 15), tile % nz * kt + frag % (kt / 16) * 16 + (l >> 4) * 4, t);
    } else {
        for (int j = 0; j < 4; ++j) put_db(a, (int)local * 4 + j, t[j]);
    }
}

// W^T [k][n] of W [n][k], for dx of wide layers through the forward's kernels.
template <typename T>
__global__ __launch_bounds__(256) void transpose_kernel(const T *w, int64_t ws, int n, int k, T *wt) {
    __shared__ T tile[32][33];
    const int c = threadIdx.x & 31, r0 = threadIdx.x >> 5;
    for (int r = r0; r < 32; r += 8) {
        const int i = blockIdx.y * 32 + r, j = blockIdx.x * 32 + c;
        if (i < n && j < k) tile[r][c] = w[(int64_t)i * ws + j];
    }
    __syncthreads();
    for (int r = r0; r < 32; r += 8) {
        const int j = blockIdx.x * 32 + r, i = blockIdx.y * 32 + c;
        if (i < n && j < k) wt[(int64_t)j * n + i] = tile[c][r];
    }
}

template <typename T, typename D, int NT, int KT, bool kDx>
hipError_t grad_launch(const GradArgs &a, const GradPlan &p, float *part, T *dz, hipStream_t stream) {
    const auto kernel = grad_kernel<T, D, NT, KT, kDx>;
    const int bytes = grad_rows(NT, KT) * (NT + KT) * 2 + (kDx ? NT * KT * 2 : 0);
    if (bytes > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void *)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != hipSuccess) return e;
    }
    kernel<<<dim3((unsigned)p.parts, (unsigned)p.ny, (unsigned)p.nz), kGradThreads, bytes, stream>>>(a, part, dz);
    return hipGetLastError();
}

template <typename T, typename D, bool kDx>
hipError_t grad_pick(const GradArgs &a, const GradPlan &p, float *part, T *dz, hipStream_t stream) {
#define HG_GRAD(NT, KT) \
    if (p.nt == NT && p.kt == KT) return grad_launch<T, D, NT, KT, kDx>(a, p, part, dz, stream);
    HG_GRAD(64, 64)
    HG_GRAD(64, 128)
    HG_GRAD(64, 256)
    HG_GRAD(128, 64)
    HG_GRAD(128, 128)
    HG_GRAD(128, 256)
    HG_GRAD(256, 64)
    HG_GRAD(256, 128)
    HG_GRAD(256, 256)
#undef HG_GRAD
    return hipErrorInvalidValue;
}

template <typename T, typename D>
hipError_t grad_run(const GradArgs &a, const GradPlan &p, char *workspace, hipStream_t stream,
                    hipError_t (*forward)(const FwdArgs &, int, hipStream_t), int dtype) {
    float *const part = (float *)workspace;
    T *const dz = (T *)(workspace + p.dz_at), *const wt = (T *)(workspace + p.wt_at);
    hipError_t e;
    if (a.m > 0) {
        e = p.fused ? grad_pick<T, D, true>(a, p, part, nullptr, stream)
                    : grad_pick<T, D, false>(a, p, part, a.dx ? dz : nullptr, stream);
        if (e != hipSuccess) return e;
    }
    if ((a.dw || a.db) && !(a.m > 0 && p.parts == 1)) {
        const int64_t quads = (a.dw ? (int64_t)p.ny * p.nz * p.nt * p.kt : 0) / 4 + (a.db ? p.ny * p.nt / 4 : 0);
        const int parts = a.m > 0 ? p.parts : 0;
        grad_join_kernel<T><<<grid_of(div_up(quads, 16)), 512, 0, stream>>>(part, parts, p.nt, p.kt, p.ny, p.nz, a);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    if (a.dx && a.m > 0 && !p.fused) {
        transpose_kernel<T><<<dim3((unsigned)div_up(a.k, 32), (unsigned)div_up(a.n, 32)), 256, 0, stream>>>((const T *)a.w, a.ws, a.n,
                                                                                                       a.k, wt);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        FwdArgs f{};
        f.m = a.m, f.xs = a.n, f.ws = a.n, f.ys = a.dxs, f.k = a.n, f.n = a.k, f.act = HG_ACT_NONE;
        f.x = dz, f.w = wt, f.y = a.dx;
        return forward(f, dtype, stream);
    }
    return hipSuccess;
}

}  // namespace
}  // namespace res
}  // namespace hg
