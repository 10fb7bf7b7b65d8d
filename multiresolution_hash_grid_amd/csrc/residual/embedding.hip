// Rows of a table by their numbers, and the table's gradient (gfx950).
//
//   y[p] = scale table[ids[p]],   dtable[v] = scale sum over p with ids[p] = v of dy[p]
//
// The gradient sorts the ids and then sums dy's rows in sorted order, so that no two
// workgroups add to one row and no sum depends on scheduling:
//
//   1. ids as keys (rows for those that name no row) sorted with their places by a
//      stable radix sort of up to 9 bits a pass: a histogram of each tile of keys, then
//      each key's place from the histograms of all tiles;
//   2. the sorted places are cut into equal stretches, whatever the segments of equal
//      keys: a group of lanes sums a stretch row by row in registers; segments that
//      begin and end in it go straight to the table, the ends that cross into other
//      stretches through LDS, and those that cross workgroups through the workspace;
//   3. a segment that crosses workgroups is joined by the workgroup it begins in.
//
// A frequent id so costs its rows' reads and no more: its sum is spread over the card.
// A sort of small keys is bound by its launches and their latencies, one after another: the
// gradient of 2^18 x 64 bf16 to 200 rows takes 30 us (count 4, move 11, sum 11, join 4; its
// bytes 6.6), that of 2^15 x 512 to 50304 rows, two passes, 44 (its bytes 16).
#include <type_traits>

#include "device_types.h"

namespace hg {
namespace res {
namespace {

// ------------------------------------------------------------------ lookup

constexpr int kLookupThreads = 256;
constexpr int kLookupRows = 4;  // rows a group of lanes has in flight

struct LookupArgs {
    int64_t m, ts, ys;
    int rows, c;
    float scale;
    const void *ids, *table;
    void *y;
};

// A piece of a row of 16-bit values, past the caches.
template <typename Y>
__device__ __forceinline__ void stream8(Y *row, Columns c, const float (&v)[8]) {
    if (c.drop >= 8) return;
    typedef Y Y8 __attribute__((ext_vector_type(8)));
    Y8 a;
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = (Y)v[j];
    if constexpr (sizeof(Y) == 2) {
        store_stream(row + c.at, __builtin_bit_cast(u32x4, a));
    } else {
        store_stream(row + c.at, f32x4{a[0], a[1], a[2], a[3]});
        store_stream(row + c.at + 4, f32x4{a[4], a[5], a[6], a[7]});
    }
}

// G lanes a row, 8 columns a lane at a time.  kStream: y is larger than the caches, and
// stores pass them by (2^20 x 64 fp32 to bf16: 30 us, 4.6 TB/s, nearly all of it writes; 56
// through the caches).
template <typename T, typename Y, typename Id, int G, bool kStream>
__global__ __launch_bounds__(kLookupThreads) void lookup_kernel(const LookupArgs a) {
    constexpr int kGroups = kLookupThreads / G;
    const int lane = threadIdx.x % G, pieces = (a.c + 7) / 8;
    const int64_t step = (int64_t)gridDim.x * kGroups * kLookupRows;
    for (int64_t r0 = (int64_t)blockIdx.x * kGroups * kLookupRows + threadIdx.x / G; r0 < a.m; r0 += step) {
        int64_t at[kLookupRows];
        bool known[kLookupRows];
#pragma unroll
        for (int u = 0; u < kLookupRows; ++u) {
            const int64_t r = r0 + u * kGroups < a.m ? r0 + u * kGroups : a.m - 1;
            const int64_t id = ((const Id *)a.ids)[r];
            known[u] = (uint64_t)id < (uint64_t)a.rows;
            at[u] = known[u] ? id * a.ts : 0;
        }
        for (int p = lane; p < pieces; p += G) {
            const Columns col = columns_of(p * 8, a.c);
            float v[kLookupRows][8] = {};
            if (a.rows > 0)
#pragma unroll
                for (int u = 0; u < kLookupRows; ++u) load8<G == 1>((const T *)a.table + at[u], col, a.c, v[u]);
#pragma unroll
            for (int u = 0; u < kLookupRows; ++u) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[u][j] = known[u] ? v[u][j] * a.scale : 0.f;
                if (r0 + u * kGroups < a.m) {
                    Y *const row = (Y *)a.y + (r0 + u * kGroups) * a.ys;
                    if constexpr (kStream) stream8(row, col, v[u]);
                    else store8<G == 1>(row, col, a.c, v[u]);
                }
            }
        }
    }
}

template <typename T, typename Y, typename Id>
hipError_t lookup_pick(const LookupArgs &a, hipStream_t stream) {
    const int pieces = (a.c + 7) / 8;
    auto run = [&](auto g) {
        constexpr int G = decltype(g)::value;
        const int64_t need = div_up(a.m, (int64_t)kLookupThreads / G * kLookupRows), most = kCus * 16;
        const dim3 grid((unsigned)(need < most ? need : most));
        if (a.c >= 8 && a.m * a.c * (int64_t)sizeof(Y) > kStreamBytes) lookup_kernel<T, Y, Id, G, true><<<grid, kLookupThreads, 0, stream>>>(a);
        else lookup_kernel<T, Y, Id, G, false><<<grid, kLookupThreads, 0, stream>>>(a);
    };
    if (pieces <= 1) run(std::integral_constant<int, 1>{});
    else if (pieces <= 2) run(std::integral_constant<int, 2>{});
    else if (pieces <= 4) run(std::integral_constant<int, 4>{});
    else if (pieces <= 8) run(std::integral_constant<int, 8>{});
    else if (pieces <= 16) run(std::integral_constant<int, 16>{});
    else if (pieces <= 32) run(std::integral_constant<int, 32>{});
    else run(std::integral_constant<int, 64>{});
    return hipGetLastError();
}

template <typename T, typename Y>
hipError_t lookup_ids(const LookupArgs &a, int ids_bits, hipStream_t stream) {
    return ids_bits == 64 ? lookup_pick<T, Y, int64_t>(a, stream) : lookup_pick<T, Y, int32_t>(a, stream);
}

// ------------------------------------------------------------------ sort

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kDigitBits = 9;                  // most of a pass
constexpr int kBins = 1 << kDigitBits;
// A tile that is the only one needs no histograms of others: up to 4096 keys (14.4 us; four
// tiles of 1024 18.0).  One among others has 1024 at least (2^15 keys of 16 bits: 44 us, with
// 2048 46, with 4096 54).
constexpr int kTileKeys = 4096, kLeastKeys = 1024;
constexpr int kMaxTiles = 128;                 // each tile reads the histograms of all
constexpr uint32_t kNoKey = 0xFFFFFFFFu;       // no key is as large

// Rows of zeros, by any number of threads together.
struct Fill {
    char *p;               // NULL: nothing to fill
    int64_t rows, bytes, stride;  // of a row, in bytes
    int groups;            // workgroups that fill
};
__device__ __forceinline__ void fill_rows(const Fill &f, int group) {
    const u32x4 zero = {0, 0, 0, 0};
    const bool one = f.stride == f.bytes;
    const int64_t rows = one ? 1 : f.rows, bytes = one ? f.rows * f.bytes : f.bytes;
    // a contiguous table is one long row shared by all threads, others are dealt to the waves
    const int64_t first = one ? 0 : (int64_t)group * kSortWaves + threadIdx.x / 64, step = one ? 1 : (int64_t)f.groups * kSortWaves;
    const int64_t at = one ? (int64_t)group * kSortThreads + threadIdx.x : threadIdx.x % 64;
    const int64_t lanes = one ? (int64_t)f.groups * kSortThreads : 64;
    for (int64_t r = first; r < rows; r += step) {
        char *const row = f.p + r * f.stride;
        for (int64_t i = at * 16; i + 16 <= bytes; i += lanes * 16) store_loose<u32x4>(row + i, zero);
        for (int64_t i = bytes / 16 * 16 + at * 2; i < bytes; i += lanes * 2) store_loose<uint16_t>(row + i, 0);
    }
}

struct SortArgs {
    const void *ids;       // of the first pass
    const uint32_t *keys, *places;  // of the others
    uint32_t *keys_out, *places_out;
    uint32_t *counts;      // [tiles][kBins]
    int m, tile, tiles, rows, shift, bits;
    Fill fill;
};

// The key of entry i: the ids themselves in the first pass.
template <typename Id>
__device__ __forceinline__ uint32_t key_of(const SortArgs &a, int i) {
    if constexpr (__is_same(Id, uint32_t)) {
        return a.keys[i];
    } else {
        const int64_t id = ((const Id *)a.ids)[i];
        return (uint64_t)id < (uint64_t)a.rows ? (uint32_t)id : (uint32_t)a.rows;
    }
}

// The lanes of the wave, of those in `lanes`, whose digit is this lane's.
__device__ __forceinline__ uint64_t peers_of(uint32_t digit, int bits, uint64_t lanes) {
    for (int bit = 0; bit < bits; ++bit) {
        const uint64_t set = __ballot((digit >> bit) & 1);
        lanes &= (digit >> bit) & 1 ? set : ~set;
    }
    return lanes;
}

// Workgroup t < tiles: histogram of tile t's digits, equal ones of a wave added by one
// lane (ids often come in runs).  The others fill.
template <typename Id>
__global__ __launch_bounds__(kSortThreads) void count_kernel(const SortArgs a) {
    __shared__ uint32_t bins[kBins];
    if ((int)blockIdx.x >= a.tiles) {
        fill_rows(a.fill, blockIdx.x - a.tiles);
        return;
    }
    const int digits = 1 << a.bits;
    for (int i = threadIdx.x; i < digits; i += kSortThreads) bins[i] = 0;
    __syncthreads();
    const int end = a.m - blockIdx.x * a.tile < a.tile ? a.m : (blockIdx.x + 1) * a.tile;
    for (int i0 = blockIdx.x * a.tile + (int)(threadIdx.x & ~63u); i0 < end; i0 += kSortThreads) {
        const int i = i0 + (int)(threadIdx.x & 63);
        const uint32_t d = (key_of<Id>(a, i < end ? i : end - 1) >> a.shift) & (digits - 1);
        const uint64_t peers = peers_of(d, a.bits, __ballot(i < end));
        if (i < end && (peers & ((1ull << (threadIdx.x & 63)) - 1)) == 0) atomicAdd(&bins[d], (uint32_t)__popcll(peers));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < digits; i += kSortThreads) a.counts[blockIdx.x * kBins + i] = bins[i];
}

// Moves tile t's keys and places to where they belong.  A wave takes a stretch of
// the tile and goes through it 64 keys at a time: a key's rank among the equal
// digits of its 64 comes from one ballot a bit, and a counter for each wave and
// digit in LDS carries on from there, so equal keys keep their order.  A tile that
// is the only one needs no histograms of others.  Stretches of up to 512 keys stay in
// registers between their histogram and their move.
constexpr int kHeldKeys = 8;
template <typename Id>
__global__ __launch_bounds__(kSortThreads) void scatter_kernel(const SortArgs a) {
    __shared__ uint32_t at[kSortWaves][kBins], before[kSortThreads], total[kSortThreads], wave_sum[kSortWaves];
    if ((int)blockIdx.x >= a.tiles) {
        fill_rows(a.fill, blockIdx.x - a.tiles);
        return;
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = blockIdx.x;
    const int digits = 1 << a.bits, mask = digits - 1;
    for (int i = threadIdx.x; i < kSortWaves * kBins; i += kSortThreads) at[i / kBins][i % kBins] = 0;
    __syncthreads();
    // this wave's stretch [begin, end)
    const int have = a.m - t * a.tile < a.tile ? a.m - t * a.tile : a.tile;
    const int per = (have + kSortWaves * 64 - 1) / (kSortWaves * 64) * 64;
    const int begin = t * a.tile + (wave * per < have ? wave * per : have), end = t * a.tile + ((wave + 1) * per < have ? (wave + 1) * per : have);
    const bool hold = per <= kHeldKeys * 64;
    const uint64_t below = (1ull << lane) - 1;
    uint32_t held[kHeldKeys], held_place[kHeldKeys], rank[kHeldKeys], equal[kHeldKeys];  // equal: of the first lane of its digit, else 0
    if (hold) {
#pragma unroll
        for (int j = 0; j < kHeldKeys; ++j) {
            if (begin + j * 64 >= end) break;
            const int i = begin + j * 64 + lane, e = i < end ? i : t * a.tile;
            held[j] = key_of<Id>(a, e);
            if constexpr (__is_same(Id, uint32_t)) held_place[j] = a.places[e];
            else held_place[j] = i;
        }
#pragma unroll
        for (int j = 0; j < kHeldKeys; ++j) {
            if (begin + j * 64 >= end) break;
            const bool is = begin + j * 64 + lane < end;
            const uint32_t d = (held[j] >> a.shift) & mask;
            const uint64_t peers = peers_of(d, a.bits, __ballot(is));
            rank[j] = __popcll(peers & below);
            equal[j] = is && rank[j] == 0 ? __popcll(peers) : 0;
            if (equal[j]) atomicAdd(&at[wave][d], equal[j]);
        }
    } else {
        for (int i = begin + lane; i < end; i += 64) atomicAdd(&at[wave][(key_of<Id>(a, i) >> a.shift) & mask], 1u);
    }
    __syncthreads();
    // of each digit: its entries in earlier tiles, and in all
    const int shares = kSortThreads / digits, digit = threadIdx.x & mask, share = threadIdx.x >> a.bits;
    uint32_t b = 0, all = 0;
    if (a.tiles == 1) {
        if (share == 0)
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) all += at[w][digit];
    } else {
#pragma unroll 16
        for (int i = share; i < a.tiles; i += shares) {
            const uint32_t n = a.counts[i * kBins + digit];
            b += i < t ? n : 0;
            all += n;
        }
    }
    before[threadIdx.x] = b, total[threadIdx.x] = all;
    __syncthreads();
    b = all = 0;
    if ((int)threadIdx.x < digits)
        for (int i = 0; i < shares; ++i) b += before[i * digits + threadIdx.x], all += total[i * digits + threadIdx.x];
    // exclusive sum over the digits: within waves, then of the waves' totals
    uint32_t sum = all;
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t v = __shfl_up(sum, o, 64);
        if (lane >= o) sum += v;
    }
    if (lane == 63) wave_sum[wave] = sum;
    __syncthreads();
    if ((int)threadIdx.x < digits) {
        uint32_t base = sum - all + b;
        for (int w = 0; w < wave; ++w) base += wave_sum[w];
        uint32_t n[kSortWaves];  // counts of a wave's stretch become its counters' start
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) n[w] = at[w][threadIdx.x];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            at[w][threadIdx.x] = base;
            base += n[w];
        }
    }
    __syncthreads();
    // A key to its place: its digit's counter and its rank; the first lane of the digit counts on.
    auto move = [&](bool mine, uint32_t key, uint32_t place, uint32_t rank, uint32_t equal) __attribute__((always_inline)) {
        const uint32_t d = (key >> a.shift) & mask, to = at[wave][d] + rank;
        wave_exchange();
        if (equal) at[wave][d] = to + equal;
        wave_exchange();
        if (mine) {
            a.keys_out[to] = key;
            a.places_out[to] = place;
        }
    };
    if (hold) {
#pragma unroll
        for (int j = 0; j < kHeldKeys; ++j) {
            if (begin + j * 64 >= end) break;
            move(begin + j * 64 + lane < end, held[j], held_place[j], rank[j], equal[j]);
        }
    } else {
        for (int i0 = begin; i0 < end; i0 += 64) {
            const bool is = i0 + lane < end;
            const int i = is ? i0 + lane : end - 1;
            const uint32_t key = key_of<Id>(a, i);
            uint32_t place = i;
            if constexpr (__is_same(Id, uint32_t)) place = a.places[i];
            const uint64_t peers = peers_of((key >> a.shift) & mask, a.bits, __ballot(is));
            const uint32_t r = __popcll(peers & below);
            move(is, key, place, r, is && r == 0 ? (uint32_t)__popcll(peers) : 0u);
        }
    }
}

// ------------------------------------------------------------------ sums of segments

constexpr int kSumThreads = 256;
constexpr int kSumRows = 8;       // rows a group of lanes has in flight; a stretch is a multiple of it
constexpr int kSumColumns = 512;  // of a workgroup: 64 lanes of 8

struct SumArgs {
    const uint32_t *keys, *places;
    const void *dy;
    void *dtable;
    float *heads, *tails;  // [workgroups][c]: sums of segments that began before a workgroup, and that go on after it
    int64_t dys, ts;
    int m, c, rows, stretch, accumulate;
    float scale;
};

template <typename D>
__device__ __forceinline__ void put_one(const SumArgs &a, uint32_t row, int col, float sum) {
    D *const p = (D *)a.dtable + (int64_t)row * a.ts + col;
    const float v = sum * a.scale;
    *p = (D)(a.accumulate ? (float)*p + v : v);
}

// Workgroup (w, y): entries w * kSlots * stretch .., columns from 512 y.  Slot s is
// a group of G lanes with entries s * stretch .. of those.  What a slot leaves:
// first: the sum of the segment that reaches into it from before, if one does, and
// through: it goes on after the slot too; last: that of a segment which begins in it
// and goes on.
template <typename T, typename D, int G>
__global__ __launch_bounds__(kSumThreads) void sum_kernel(const SumArgs a) {
    constexpr int kSlots = kSumThreads / G;
    __shared__ float first[kSlots][G * 8], last[kSlots][G * 8];
    __shared__ uint32_t first_key[kSlots], last_key[kSlots];  // kNoKey: there is none
    __shared__ int through[kSlots];
    const int lane = threadIdx.x % G, slot = threadIdx.x / G;
    const int c0 = blockIdx.y * kSumColumns, nominal = c0 + lane * 8;
    const Columns col = columns_of(nominal, a.c);
    const int64_t e0 = (int64_t)blockIdx.x * kSlots * a.stretch;
    const int64_t i0 = e0 + (int64_t)slot * a.stretch, i1 = i0 + a.stretch < a.m ? i0 + a.stretch : a.m;
    if (lane == 0) first_key[slot] = last_key[slot] = kNoKey, through[slot] = 0;

    // a sum of 8 columns to the table; slots that the piece before holds too are its
    auto put8 = [&](uint32_t row, const float (&sum)[8]) {
        if (row >= (uint32_t)a.rows || col.drop >= 8) return;
        D *const p = (D *)a.dtable + (int64_t)row * a.ts;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = sum[j] * a.scale;
        if (col.drop == 0 && !a.accumulate) {
            store8<G == 1>(p, col, a.c, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j >= col.drop && col.at + j < a.c) p[col.at + j] = (D)(a.accumulate ? (float)p[col.at + j] + v[j] : v[j]);
        }
    };
    float acc[8] = {};
    bool whole = false;
    uint32_t whole_key = kNoKey;
    if (i0 < i1) {
        uint32_t key[kSumRows], place[kSumRows];
        auto entries = [&](int64_t i) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < kSumRows; ++u) {
                const int64_t e = i + u < i1 ? i + u : i1 - 1;
                key[u] = a.keys[e], place[u] = a.places[e];
            }
        };
        entries(i0);
        const uint32_t next = i1 < a.m ? a.keys[i1] : kNoKey, prev = i0 > 0 ? a.keys[i0 - 1] : kNoKey;
        uint32_t now = key[0];
        bool open = prev == now;  // the segment began before this slot
        for (int64_t i = i0; i < i1 && now < (uint32_t)a.rows; i += kSumRows) {
            uint32_t k[kSumRows];
            float v[kSumRows][8];
#pragma unroll
            for (int u = 0; u < kSumRows; ++u) {
                k[u] = key[u];
                load8<G == 1>((const T *)a.dy + (int64_t)place[u] * a.dys, col, a.c, v[u]);
            }
            if (i + kSumRows < i1) entries(i + kSumRows);  // the next rows' while these are on their way
#pragma unroll
            for (int u = 0; u < kSumRows; ++u) {
                if (i + u >= i1) break;
                if (k[u] != now) {
                    if (open) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) first[slot][lane * 8 + j] = acc[j];
                        if (lane == 0) first_key[slot] = now;
                        open = false;
                    } else {
                        put8(now, acc);
                    }
                    now = k[u];
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[j] = 0.f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] += v[u][j];
            }
        }
        whole = open && next == now && now < (uint32_t)a.rows;
        if (now < (uint32_t)a.rows && !whole) {
            if (open) {
#pragma unroll
                for (int j = 0; j < 8; ++j) first[slot][lane * 8 + j] = acc[j];
                if (lane == 0) first_key[slot] = now;
            } else if (next == now) {
#pragma unroll
                for (int j = 0; j < 8; ++j) last[slot][lane * 8 + j] = acc[j];
                if (lane == 0) last_key[slot] = now;
            } else {
                put8(now, acc);
            }
        }
        whole_key = now;
    }
    // Slots that lie within one segment: where all of a wave's do, they are one.
    const bool together = G < 64 && __ballot(whole) == ~0ull;
    if (together)
#pragma unroll
        for (int o = G; o < 64; o <<= 1)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += __shfl_xor(acc[j], o, 64);
    if (whole && (!together || slot % (64 / G) == 0)) {
#pragma unroll
        for (int j = 0; j < 8; ++j) first[slot][lane * 8 + j] = acc[j];
        if (lane == 0) first_key[slot] = whole_key, through[slot] = 1;
    }
    __syncthreads();
    // The slots' ends, in order, one column a thread: only the slots that have some.
    // Bit s % 64 of word s / 64: slot s has a first sum, it goes through, it has a last one.
    constexpr int kWords = (kSlots + 63) / 64;
    uint64_t some[kWords], passes[kWords], starts[kWords];
    {
        const int l = threadIdx.x & 63;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
            const int s = w * 64 + l < kSlots ? w * 64 + l : kSlots - 1;
            const bool is = w * 64 + l < kSlots;
            some[w] = __ballot(is && first_key[s] != kNoKey);
            passes[w] = __ballot(is && through[s]);
            starts[w] = __ballot(is && last_key[s] != kNoKey);
        }
    }
    for (int k = threadIdx.x; k < G * 8; k += kSumThreads) {
        const int column = column_of(c0 + k, a.c);
        if (column < 0) continue;
        bool before = (some[0] & 1) != 0;   // the open segment began before this workgroup
        float carry = 0.f;
        bool open = false;
#pragma unroll
        for (int w = 0; w < kWords; ++w)
            for (uint64_t left = some[w] | starts[w]; left; left &= left - 1) {
                const int bit = __builtin_ctzll(left), s = w * 64 + bit;
                if (some[w] >> bit & 1) {
                    carry += first[s][k];
                    open = true;
                    if (passes[w] >> bit & 1) continue;
                    if (before) a.heads[(int64_t)blockIdx.x * a.c + column] = carry;
                    else put_one<D>(a, first_key[s], column, carry);
                    before = open = false;
                }
                if (starts[w] >> bit & 1) open = true, before = false, carry = last[s][k];
                else carry = 0.f;
            }
        if (open) (before ? a.heads : a.tails)[(int64_t)blockIdx.x * a.c + column] = carry;
    }
}

// Workgroup w joins the segment that begins in stretch w of `per` entries and goes
// on into the next ones: its own tail, and the heads of those it reaches into.
template <typename D, int G>
__global__ __launch_bounds__(kSumThreads) void segment_join_kernel(const SumArgs a, int per, int groups) {
    constexpr int kSlots = kSumThreads / G;
    __shared__ float sums[kSlots][G * 8];
    const int w = blockIdx.x;
    const int64_t end = (int64_t)(w + 1) * per;
    if (end >= a.m) return;
    const uint32_t key = a.keys[end];
    if (key >= (uint32_t)a.rows || a.keys[end - 1] != key || (w > 0 && a.keys[end - per - 1] == key)) return;
    int lo = w;  // the last workgroup whose first entry has this key
    for (int n = kSumThreads; n == kSumThreads; lo += n) {
        const int z = lo + 1 + (int)threadIdx.x;
        n = __syncthreads_count(z < groups && a.keys[(int64_t)z * per] == key);
    }
    const int lane = threadIdx.x % G, slot = threadIdx.x / G, c0 = blockIdx.y * kSumColumns;
    const Columns col = columns_of(c0 + lane * 8, a.c);
    float acc[8] = {};
#pragma unroll 4
    for (int z = w + 1 + slot; z <= lo; z += kSlots) {
        float v[8];
        load8<G == 1>(a.heads + (int64_t)z * a.c, col, a.c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += v[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[slot][lane * 8 + j] = acc[j];
    __syncthreads();
    for (int k = threadIdx.x; k < G * 8; k += kSumThreads) {
        const int column = column_of(c0 + k, a.c);
        if (column < 0) continue;
        float t = a.tails[(int64_t)w * a.c + column];
        for (int s = 0; s < kSlots; ++s) t += sums[s][k];
        put_one<D>(a, key, column, t);
    }
}

// ------------------------------------------------------------------ plan

struct Plan {
    int lanes, stretch, per, groups;  // lanes of a row; entries of a slot and of a workgroup; workgroups over the entries
    int tile, tiles, passes;
    size_t counts_at, keys_at, places_at, heads_at, tails_at, bytes;
};

Plan plan_of(const hg_embedding_grad &op) {
    Plan p{};
    if (op.m == 0 || op.rows == 0) return p;
    const int pieces = (op.c + 7) / 8, columns = (int)div_up(pieces, 64);
    p.lanes = 1;
    while (p.lanes < 64 && p.lanes < pieces) p.lanes *= 2;
    // Stretches as short as one load's rows where they fill the card (2048 workgroups), longer
    // ones where there are more: fewer ends to join.
    const int64_t slots = kSumThreads / p.lanes;
    const int64_t want = div_up(op.m * columns, slots * 2048);
    p.stretch = (int)div_up(want, kSumRows) * kSumRows;
    p.per = (int)(slots * p.stretch);
    p.groups = (int)div_up(op.m, p.per);
    const int bits = 32 - __builtin_clz((unsigned)op.rows);
    p.passes = (int)div_up(bits, kDigitBits);
    p.tile = op.m <= kTileKeys ? (int)op.m : (int)(div_up(div_up(op.m, kMaxTiles), kSortThreads) * kSortThreads);
    if (op.m > kTileKeys && p.tile < kLeastKeys) p.tile = kLeastKeys;
    p.tiles = (int)div_up(op.m, p.tile);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t was = at;
        at += (bytes + 255) / 256 * 256;
        return was;
    };
    const int buffers = p.passes > 1 ? 2 : 1;
    p.counts_at = take(p.tiles > 1 ? (size_t)p.tiles * kBins * 4 : 0);
    p.keys_at = take((size_t)op.m * 4 * buffers);
    p.places_at = take((size_t)op.m * 4 * buffers);
    p.heads_at = take(p.groups > 1 ? (size_t)p.groups * op.c * 4 : 0);
    p.tails_at = take(p.groups > 1 ? (size_t)p.groups * op.c * 4 : 0);
    p.bytes = at;
    return p;
}

template <typename T, typename D>
hipError_t sum_run(const SumArgs &a, const Plan &p, hipStream_t stream) {
    const dim3 grid((unsigned)p.groups, (unsigned)div_up(a.c, kSumColumns));
    auto run = [&](auto g) {
        constexpr int G = decltype(g)::value;
        sum_kernel<T, D, G><<<grid, kSumThreads, 0, stream>>>(a);
        if (p.groups > 1) segment_join_kernel<D, G><<<grid, kSumThreads, 0, stream>>>(a, p.per, p.groups);
    };
    switch (p.lanes) {
    case 1: run(std::integral_constant<int, 1>{}); break;
    case 2: run(std::integral_constant<int, 2>{}); break;
    case 4: run(std::integral_constant<int, 4>{}); break;
    case 8: run(std::integral_constant<int, 8>{}); break;
    case 16: run(std::integral_constant<int, 16>{}); break;
    case 32: run(std::integral_constant<int, 32>{}); break;
    default: run(std::integral_constant<int, 64>{});
    }
    return hipGetLastError();
}

int bytes_of(int dtype) { return dtype == HG_F32 ? 4 : 2; }

}  // namespace

hipError_t launch_embedding_forward(const hg_embedding &op, hipStream_t stream) {
    const LookupArgs a{op.m, op.table_stride, op.y_stride, op.rows, op.c, op.scale, op.ids, op.table, op.y};
    if (op.table_dtype == HG_F16) return lookup_ids<f16, f16>(a, op.ids_bits, stream);
    if (op.table_dtype == HG_BF16) return lookup_ids<bf16, bf16>(a, op.ids_bits, stream);
    if (op.y_dtype == HG_F16) return lookup_ids<float, f16>(a, op.ids_bits, stream);
    if (op.y_dtype == HG_BF16) return lookup_ids<float, bf16>(a, op.ids_bits, stream);
    return lookup_ids<float, float>(a, op.ids_bits, stream);
}

size_t embedding_backward_bytes(const hg_embedding_grad &op) { return plan_of(op).bytes; }

hipError_t launch_embedding_backward(const hg_embedding_grad &op, void *workspace, hipStream_t stream) {
    if (op.rows == 0) return hipSuccess;
    const Plan p = plan_of(op);
    char *const ws = (char *)workspace;
    SortArgs s{};
    if (!op.accumulate) {
        const int64_t e = bytes_of(op.dtable_dtype), bytes = (int64_t)op.rows * op.c * e;
        const int64_t groups = div_up(bytes, 65536);
        // (one row has no stride)
        s.fill = Fill{(char *)op.dtable, op.rows, op.c * e, op.rows > 1 ? op.dtable_stride * e : op.c * e, (int)(groups < 1024 ? groups : 1024)};
    }
    const Fill whole = s.fill;
    if (op.m == 0) {
        if (op.accumulate) return hipSuccess;
        count_kernel<int32_t><<<dim3((unsigned)s.fill.groups), kSortThreads, 0, stream>>>(s);
        return hipGetLastError();
    }
    uint32_t *const keys[2] = {(uint32_t *)(ws + p.keys_at), (uint32_t *)(ws + p.keys_at) + op.m};
    uint32_t *const places[2] = {(uint32_t *)(ws + p.places_at), (uint32_t *)(ws + p.places_at) + op.m};
    s.ids = op.ids, s.counts = (uint32_t *)(ws + p.counts_at);
    s.m = (int)op.m, s.tile = p.tile, s.tiles = p.tiles, s.rows = op.rows;
    const int bits = 32 - __builtin_clz((unsigned)op.rows);
    s.bits = (int)div_up(bits, p.passes);
    int share = 0;
    for (int pass = 0; pass < p.passes; ++pass) {
        s.shift = pass * s.bits;
        s.keys_out = keys[pass & 1], s.places_out = places[pass & 1];
        s.keys = keys[~pass & 1], s.places = places[~pass & 1];
        // each launch of the sort fills its share of the table beside its tiles (2^17 x 256: 61 us, all in the first 64)
        const int launches = p.passes * (p.tiles > 1 ? 2 : 1);
        auto next = [&] {
            if (whole.groups == 0) return dim3((unsigned)p.tiles);
            const int64_t from = whole.rows * share / launches, to = whole.rows * (share + 1) / launches;
            ++share;
            s.fill.p = whole.p + from * whole.stride, s.fill.rows = to - from;
            return dim3((unsigned)(p.tiles + s.fill.groups));
        };
        auto run = [&](auto id) {
            typedef decltype(id) Id;
            dim3 grid;
            if (p.tiles > 1) grid = next(), count_kernel<Id><<<grid, kSortThreads, 0, stream>>>(s);
            grid = next(), scatter_kernel<Id><<<grid, kSortThreads, 0, stream>>>(s);
        };
        if (pass > 0) run(uint32_t{});
        else if (op.ids_bits == 64) run(int64_t{});
        else run(int32_t{});
    }
    const int out = (p.passes - 1) & 1;
    const SumArgs a{keys[out], places[out], op.dy, op.dtable, (float *)(ws + p.heads_at), (float *)(ws + p.tails_at), op.dy_stride,
                    op.dtable_stride, (int)op.m, op.c, op.rows, p.stretch, op.accumulate, op.scale};
    const bool wide = op.dtable_dtype == HG_F32;
    if (op.dy_dtype == HG_F16) return wide ? sum_run<f16, float>(a, p, stream) : sum_run<f16, f16>(a, p, stream);
    if (op.dy_dtype == HG_BF16) return wide ? sum_run<bf16, float>(a, p, stream) : sum_run<bf16, bf16>(a, p, stream);
    return sum_run<float, float>(a, p, stream);
}

}  // namespace res
}  // namespace hg
