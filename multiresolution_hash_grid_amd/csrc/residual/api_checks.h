// Argument checks that the residual head's C entry points share.
#pragma once

#include <cmath>

#include "residual_internal.h"

namespace hg {
namespace res {

constexpr int64_t kMaxRows = (int64_t)1 << 40;
constexpr int kMaxWidth = 65536;
constexpr int kMaxColumns = 1 << 20;
constexpr int64_t kMaxGradStride = (int64_t)1 << 22;  // of a backward's rows: a step's offsets are 32-bit

inline int size_of(int dtype) {
    switch (dtype) {
    case HG_F32: return 4;
    case HG_F16:
    case HG_BF16: return 2;
    case HG_F8: return 1;
    }
    return 0;
}

// A matrix [m][cols]: pointer there (or allowed to be NULL), aligned to its
// elements, rows that do not overlap and whose last byte has a 63-bit offset.
inline int check_rows(const char *name, const void *p, int64_t stride, int64_t m, int64_t cols, int dtype, bool needed) {
    if (!p) return needed ? abi_fail(HG_EINVAL, "%s is NULL", name) : HG_OK;
    if ((uintptr_t)p % size_of(dtype)) return abi_fail(HG_EINVAL, "%s is not aligned to its elements", name);
    if (m > 1 && stride < cols)
        return abi_fail(HG_EINVAL, "%s: row stride %lld < %lld columns", name, (long long)stride, (long long)cols);
    if (stride > (int64_t)1 << 20 && m > ((int64_t)1 << 60) / stride)
        return abi_fail(HG_EINVAL, "%s: rows and stride too large", name);
    return HG_OK;
}

// An output in place of an input: rows of the same stride, or they would meet others.
inline int check_in_place(const char *out, const void *p, int64_t stride, const char *in, const void *q, int64_t q_stride, int64_t m) {
    if (!p || p != q || m < 2 || stride == q_stride) return HG_OK;
    return abi_fail(HG_EINVAL, "%s in place of %s needs its row stride (%lld, not %lld)", out, in, (long long)q_stride, (long long)stride);
}

inline int check_vector(const char *name, const float *p, bool needed) {
    if (!p) return needed ? abi_fail(HG_EINVAL, "%s is NULL", name) : HG_OK;
    if ((uintptr_t)p % 4) return abi_fail(HG_EINVAL, "%s is not 4-byte aligned", name);
    return HG_OK;
}

inline int check_sizes(int64_t m, int32_t k, int32_t n, int32_t act) {
    if (m < 0 || m > kMaxRows) return abi_fail(HG_EINVAL, "m = %lld outside 0..2^40", (long long)m);
    if (k < 1 || k > kMaxWidth || n < 1 || n > kMaxWidth)
        return abi_fail(HG_EINVAL, "k = %d or n = %d outside 1..%d", k, n, kMaxWidth);
    if (act < HG_ACT_NONE || act > HG_ACT_GELU_TANH) return abi_fail(HG_EINVAL, "unknown activation %d", act);
    return HG_OK;
}

inline int launched(hipError_t e, const char *what) {
    if (e != hipSuccess) return abi_fail(HG_EHIP, "%s: %s", what, hipGetErrorString(e));
    return abi_ok();
}

inline int check_workspace(const void *workspace, size_t have, size_t need) {
    if (need == 0) return HG_OK;
    if (!workspace || have < need) return abi_fail(HG_EINVAL, "workspace of %zu bytes, %zu needed", workspace ? have : 0, need);
    if ((uintptr_t)workspace % 256) return abi_fail(HG_EINVAL, "workspace is not 256-byte aligned");
    return HG_OK;
}

inline int check_norm_sizes(int64_t m, int32_t c, int dtype) {
    if (m < 0 || m > kMaxRows) return abi_fail(HG_EINVAL, "m = %lld outside 0..2^40", (long long)m);
    if (c < 1 || c > kMaxColumns) return abi_fail(HG_EINVAL, "c = %d outside 1..%d", c, kMaxColumns);
    if (dtype != HG_F32 && dtype != HG_F16 && dtype != HG_BF16)
        return abi_fail(HG_EUNSUPPORTED, "dtype %d is not HG_F32, HG_F16 or HG_BF16", dtype);
    return HG_OK;
}

}  // namespace res
}  // namespace hg
