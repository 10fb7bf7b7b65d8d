// AdamW over many tensors in one launch (gfx950).
//
//   m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2          (g scaled first)
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Adam as published (Kingma and Ba 2015) with the decay taken out of the
// gradient (Loshchilov and Hutter 2019).  Rates, decays and types are each
// tensor's own, so the hash tables (no decay, a higher rate) and the head's
// weights go in one step.
//
// 8-bit moments.  256 consecutive values share a power of two 2^(e - 127),
// the byte e, picked so that the block's largest value lies in the top binade
// but one of the code below it: scaling is exact and costs no precision,
// because the codes are floats themselves.
//   m: sign, 4 exponent bits (bias 7), 3 mantissa bits; |m| in [2^7, 2^8) at most
//   v: no sign, 5 exponent bits (bias 15), 3 mantissa bits; v in [2^15, 2^16) at most
// v keeps a factor of 2^33 between a block's largest and smallest value (m 2^17):
// the gradients of hash entries that share a block differ by orders of
// magnitude, and v is their square.  Both are rounded stochastically: with
// b2 = 0.99 a moment moves by 1 % a step and its codes are 12 % apart, so
// rounding to nearest would hold every code where it is for good.  A nonzero
// v keeps a code of at least 1: a v of zero under a live m would divide by eps.
// Placing the value's binary exponent so that the code's smallest normal
// becomes fp32's smallest normal makes the truncation of fp32 bits the
// truncation of the code, gradual underflow included: noise is added below
// the last bit kept and the word is shifted.
// Bound by memory: 28 + 2 bytes a value with fp32 state and a 16-bit copy, 16 + 2
// with 8-bit state; 2^24 values of the one go in 105 us (4.8 TB/s), 2^25 of the
// other in 119 (5.1 TB/s).
// The state's arithmetic is one IEEE operation at a time (no contraction), so
// that the codes do not depend on how a compiler pairs operations.
#include "device_types.h"

namespace hg {
namespace res {
namespace {

struct Tensor {
    float *p;
    void *g, *m, *v, *copy;
    uint8_t *me, *ve;
    int64_t count;
    float step_size;   // lr / (1 - b1^t); with clocks lr
    float keep;        // 1 - lr wd
    uint32_t key;      // of the rounding noise
    int32_t first;     // first workgroup
    int32_t place;     // in the caller's list
    int8_t grad_type, copy_type, vec, pad;
};
struct Args {
    Tensor t[kAdamwTensors];
    int32_t n;
    int32_t flags;
    float beta1, beta2, omb1, omb2, root, eps;  // root = 1 / sqrt(1 - b2^t)
    uint32_t seed;
    const float *grad_scale;
    hg_adamw_clock *clocks;
};
static_assert(sizeof(Args) <= 4096, "kernel arguments");

constexpr int kThreads = 256;
constexpr int kPer = 4;                        // consecutive values of a thread: a wave has one 256-value block
// One block a wave: with 2, 4, 8 blocks 2^24 values of fp32 state take 6, 10, 16 % longer and
// 2^25 of 8-bit state 6, 13, 21 (a wave's stores hold back its next loads).
constexpr int kChunk = kThreads * kPer;
constexpr int64_t kMaxGroups = 1023 * kGridX;  // of a launch, in whole rows of the grid: their numbers are 32-bit

// A 32-bit finalizer of multiplications and shifts (MurmurHash3's, public domain).
__host__ __device__ __forceinline__ uint32_t mix(uint32_t h) {
    h ^= h >> 16;
    h *= 0x85EBCA6Bu;
    h ^= h >> 13;
    h *= 0xC2B2AE35u;
    return h ^ (h >> 16);
}

__host__ __device__ __forceinline__ uint32_t noise_key(uint32_t seed, int place) {
    return mix(seed + 0x9E3779B9u * (uint32_t)(place + 1));
}

// What depends on t, of one tensor.
struct Rates {
    float step_size, root;
    uint32_t key;
};

__device__ __forceinline__ bool skipped(const Args &a) {
    return a.grad_scale && !(fabsf(*a.grad_scale) <= 3.402823466e38f);
}

// Counts the step for each tensor of the launch that follows, unless it is
// skipped, and leaves there what the host works out where it knows t.
__global__ __launch_bounds__(64) void adamw_clock_kernel(const Args a) {
    const int i = threadIdx.x;
    if (i >= a.n || skipped(a)) return;
    hg_adamw_clock *const c = a.clocks + a.t[i].place;
    const int32_t t = c->step + 1;
    c->step = t;
    c->step_size = (float)((double)a.t[i].step_size / (1.0 - pow((double)a.beta1, (double)t)));
    c->root = (float)(1.0 / sqrt(1.0 - pow((double)a.beta2, (double)t)));
    c->key = noise_key(a.seed + (uint32_t)t, a.t[i].place);
}

template <bool kVec>
__device__ __forceinline__ void load4(const void *base, int type, int64_t i, int left, float (&v)[4]) {
    if (type == HG_F32) {
        const float *p = (const float *)base + i;
        if (kVec) {
            const f32x4 a = *(const f32x4 *)p;
            for (int j = 0; j < 4; ++j) v[j] = a[j];
        } else {
            for (int j = 0; j < 4; ++j) v[j] = j < left ? p[j] : 0.f;
        }
        return;
    }
    const uint16_t *p = (const uint16_t *)base + i;
    uint16_t h[4];
    if (kVec) {
        const u32x2 a = *(const u32x2 *)p;
        h[0] = a.x & 0xFFFF, h[1] = a.x >> 16, h[2] = a.y & 0xFFFF, h[3] = a.y >> 16;
    } else {
        for (int j = 0; j < 4; ++j) h[j] = j < left ? p[j] : (uint16_t)0;
    }
    for (int j = 0; j < 4; ++j)
        v[j] = type == HG_F16 ? (float)__builtin_bit_cast(f16, h[j]) : __uint_as_float((uint32_t)h[j] << 16);
}

template <bool kVec>
__device__ __forceinline__ void store4(void *base, int type, int64_t i, int left, const float (&v)[4]) {
    if (type == HG_F32) {
        float *p = (float *)base + i;
        if (kVec) *(f32x4 *)p = f32x4{v[0], v[1], v[2], v[3]};
        else
            for (int j = 0; j < 4; ++j)
                if (j < left) p[j] = v[j];
        return;
    }
    uint16_t h[4];
    for (int j = 0; j < 4; ++j)
        h[j] = type == HG_F16 ? __builtin_bit_cast(uint16_t, (f16)v[j]) : __builtin_bit_cast(uint16_t, (bf16)v[j]);
    uint16_t *p = (uint16_t *)base + i;
    if (kVec) *(u32x2 *)p = u32x2{h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16};
    else
        for (int j = 0; j < 4; ++j)
            if (j < left) p[j] = h[j];
}

template <bool kVec>
__device__ __forceinline__ uint32_t load_codes(const void *base, int64_t i, int left) {
    const uint8_t *p = (const uint8_t *)base + i;
    if (kVec) return *(const uint32_t *)p;
    uint32_t c = 0;
    for (int j = 0; j < 4; ++j)
        if (j < left) c |= (uint32_t)p[j] << (8 * j);
    return c;
}
template <bool kVec>
__device__ __forceinline__ void store_codes(void *base, int64_t i, int left, uint32_t c) {
    uint8_t *p = (uint8_t *)base + i;
    if (kVec) *(uint32_t *)p = c;
    else
        for (int j = 0; j < 4; ++j)
            if (j < left) p[j] = (uint8_t)(c >> (8 * j));
}

// Block exponent of a block whose largest magnitude has these bits; 255 marks
// a block that holds a value that is not finite (it reads back as NaN).
__device__ __forceinline__ uint32_t block_exponent(uint32_t bits, int top) {
    const int e = (int)(bits >> 23);
    if (e == 255) return 255;
    const int k = e - top;
    return bits == 0 || k < 1 ? 1 : (uint32_t)k;
}

template <bool kVec>
__device__ __forceinline__ void clear4(const Tensor &t, int64_t i, int left) {
    const float z[4] = {0.f, 0.f, 0.f, 0.f};
    store4<kVec>(t.g, t.grad_type, i, left, z);
}

template <int kBits, bool kVec>
__device__ __forceinline__ void update4(const Tensor &t, const Args &a, const Rates &rates, int64_t i, int left, float scale) {
#pragma clang fp contract(off)
    float p[4], g[4], m[4], v[4];
    load4<kVec>(t.p, HG_F32, i, left, p);
    load4<kVec>(t.g, t.grad_type, i, left, g);
    if (kBits == 32) {
        load4<kVec>(t.m, HG_F32, i, left, m);
        load4<kVec>(t.v, HG_F32, i, left, v);
    } else {
        const uint32_t mc = load_codes<kVec>(t.m, i, left), vc = load_codes<kVec>(t.v, i, left);
        const int64_t b = i / 256;
        const int me = left > 0 ? t.me[b] : 1, ve = left > 0 ? t.ve[b] : 1;
        const float mn = me == 255 ? __builtin_nanf("") : 1.f, vn = ve == 255 ? __builtin_nanf("") : 1.f;
        for (int j = 0; j < 4; ++j) {
            const uint32_t c = (mc >> (8 * j)) & 255u, d = (vc >> (8 * j)) & 255u;
            const float x = ldexpf(__uint_as_float((c & 127u) << 20), me - 7);  // 2^(127 - 7) 2^(me - 127)
            m[j] = (c & 128u ? -x : x) * mn;
            v[j] = ldexpf(__uint_as_float(d << 20), ve - 15) * vn;
        }
    }
    float pn[4];
    for (int j = 0; j < 4; ++j) {
        const float gj = a.grad_scale ? g[j] * scale : g[j];
        m[j] = m[j] * a.beta1 + gj * a.omb1;
        v[j] = v[j] * a.beta2 + (gj * gj) * a.omb2;
        pn[j] = p[j] * t.keep - rates.step_size * m[j] / (sqrtf(v[j]) * rates.root + a.eps);
    }
    if (kBits == 32) {
        store4<kVec>(t.m, HG_F32, i, left, m);
        store4<kVec>(t.v, HG_F32, i, left, v);
    } else {
        uint32_t mb = 0, vb = 0;
        for (int j = 0; j < 4; ++j)
            if (j < left) {
                const uint32_t x = __float_as_uint(m[j]) & 0x7FFFFFFFu, y = __float_as_uint(v[j]) & 0x7FFFFFFFu;
                mb = x > mb ? x : mb, vb = y > vb ? y : vb;
            }
        const uint32_t me = block_exponent(wave_max_u32(mb), 7), ve = block_exponent(wave_max_u32(vb), 15);
        uint32_t mc = 0, vc = 0;
        for (int j = 0; j < 4; ++j) {
            const uint32_t h = mix((uint32_t)(i + j) ^ rates.key);
            const uint32_t mt = __float_as_uint(ldexpf(fabsf(m[j]), 7 - (int)me));
            const uint32_t vt = __float_as_uint(ldexpf(v[j], 15 - (int)ve));
            uint32_t c = ((mt + ((h & 0xFFFFu) << 4)) >> 20) & 127u;
            uint32_t d = ((vt + ((h >> 16) << 4)) >> 20) & 255u;
            if (m[j] < 0.f && c) c |= 128u;
            if (d == 0 && v[j] > 0.f) d = 1;
            mc |= c << (8 * j), vc |= d << (8 * j);
        }
        store_codes<kVec>(t.m, i, left, mc);
        store_codes<kVec>(t.v, i, left, vc);
        if ((threadIdx.x & 63) == 0 && left > 0) {
            t.me[i / 256] = (uint8_t)me;
            t.ve[i / 256] = (uint8_t)ve;
        }
    }
    store4<kVec>(t.p, HG_F32, i, left, pn);
    if (t.copy) store4<kVec>(t.copy, t.copy_type, i, left, pn);
    if (a.flags & HG_ADAM_ZERO_GRAD) clear4<kVec>(t, i, left);
}

template <int kBits>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const Args a) {
    const bool skip = skipped(a);  // the step does nothing, or clears the gradients
    if (skip && !(a.flags & HG_ADAM_ZERO_SKIPPED)) return;
    const float scale = a.grad_scale ? *a.grad_scale : 1.f;
    const int block = (int)(blockIdx.y * kGridX + blockIdx.x);
    // The tensor of this workgroup: first[] is ascending.
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.t[mid].first <= block) lo = mid;
        else hi = mid - 1;
    }
    const Tensor &t = a.t[lo];
    Rates rates{t.step_size, a.root, t.key};
    if (a.clocks) {
        const hg_adamw_clock &c = a.clocks[t.place];
        rates = {c.step_size, c.root, c.key};
    }
    const int64_t i = (int64_t)(block - t.first) * kChunk + threadIdx.x * kPer;
    const int64_t left = t.count - i;
    // Whole waves decide together: a block is a wave's 256 values.
    const int64_t wave_left = t.count - (i - (threadIdx.x & 63) * kPer);
    if (wave_left <= 0) return;
    const int mine = left > 4 ? 4 : left < 0 ? 0 : (int)left;
    if (skip) clear4<false>(t, i, mine);
    else if (wave_left >= 256 && t.vec) update4<kBits, true>(t, a, rates, i, 4, scale);
    else update4<kBits, false>(t, a, rates, i, mine, scale);
}

}  // namespace

hipError_t launch_adamw(const hg_adamw &opt, const hg_adamw_tensor *tensors, int32_t n, const float *grad_scale,
                        int32_t flags, hipStream_t stream) {
    const bool clock = (flags & HG_ADAM_CLOCK) != 0;
    const double t0 = clock ? 1.0 : (double)opt.step;
    const double bc1 = clock ? 1.0 : 1.0 - pow((double)opt.beta1, t0), bc2 = 1.0 - pow((double)opt.beta2, t0);
    auto al = [](const void *p, uintptr_t k) { return ((uintptr_t)p % k) == 0; };
    for (const int bits : {32, 8}) {
        int32_t at = 0;
        while (at < n) {
            Args a;
            a.n = 0;
            a.flags = flags;
            a.beta1 = opt.beta1, a.beta2 = opt.beta2;
            a.omb1 = (float)(1.0 - (double)opt.beta1), a.omb2 = (float)(1.0 - (double)opt.beta2);
            a.root = (float)(1.0 / sqrt(bc2));
            a.eps = opt.eps;
            a.seed = opt.seed;
            a.grad_scale = grad_scale;
            a.clocks = clock ? opt.clocks : nullptr;
            int64_t groups = 0;
            for (; at < n && a.n < kAdamwTensors; ++at) {
                const hg_adamw_tensor &s = tensors[at];
                if (s.count == 0 || s.state_bits != bits) continue;
                const int64_t more = div_up(s.count, kChunk);
                if (groups + more > kMaxGroups) break;
                Tensor &t = a.t[a.n++];
                t.p = s.param, t.g = s.grad, t.m = s.m, t.v = s.v, t.copy = s.copy;
                t.me = s.m_exp, t.ve = s.v_exp;
                t.count = s.count;
                t.step_size = (float)((double)s.lr / bc1);
                t.keep = (float)(1.0 - (double)s.lr * (double)s.weight_decay);
                t.key = noise_key(opt.seed, at);
                t.place = at;
                t.first = (int32_t)groups;
                t.grad_type = (int8_t)s.grad_dtype, t.copy_type = (int8_t)s.copy_dtype;
                const uintptr_t sa = bits == 8 ? 4 : 16;
                t.vec = al(s.param, 16) && al(s.grad, s.grad_dtype == HG_F32 ? 16 : 8) && al(s.m, sa) && al(s.v, sa) &&
                        (!s.copy || al(s.copy, s.copy_dtype == HG_F32 ? 16 : 8));
                groups += more;
            }
            if (a.n == 0) continue;
            if (clock) adamw_clock_kernel<<<1, 64, 0, stream>>>(a);
            if (bits == 32) adamw_kernel<32><<<grid_of(groups), kThreads, 0, stream>>>(a);
            else adamw_kernel<8><<<grid_of(groups), kThreads, 0, stream>>>(a);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

}  // namespace res
}  // namespace hg
