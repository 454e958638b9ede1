// Argument checks and launch helpers shared by the layer operators' hosts.
#pragma once

#include <hip/hip_runtime_api.h>

#include <initializer_list>

#include "internal.h"

namespace zs {
namespace {

inline bool aligned(const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
inline bool vec16(const void *p, int64_t ld, int es) { return aligned(p, 16) && ld * es % 16 == 0; }

inline bool known_dtype(int32_t d) { return d == ZERO_BF16 || d == ZERO_FP32; }
inline int bytes_of(int32_t d) { return d == ZERO_BF16 ? 2 : 4; }

// Whether p is one of `others`; NULL is nothing.  What a call writes must not
// be an address that it uses for something else: only equal addresses are
// looked for, since matrices with leading dimensions may share a range.
inline bool is_one_of(const void *p, std::initializer_list<const void *> others)
{
    for (const void *o : others)
        if (p && p == o)
            return true;
    return false;
}

// The exponent bytes of a kept matrix that has them.
inline const void *scales_of(const zero_saved *s)
{
    return s && s->format == ZERO_SAVED_E4M3 ? s->scales : nullptr;
}
inline const void *data_of(const zero_saved *s) { return s ? s->data : nullptr; }

inline zero_status launched(const char *what)
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return fail(ZERO_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
    return ZERO_OK;
}

// A matrix argument: pointer, leading dimension and alignment.
inline zero_status check_matrix(const char *what, const void *p, int64_t ld, int64_t cols, int32_t dtype)
{
    if (!known_dtype(dtype))
        return fail(ZERO_ERR_INVALID_ARG, "%s: unknown dtype %d", what, dtype);
    if (!p)
        return fail(ZERO_ERR_INVALID_ARG, "%s is required", what);
    if (ld < cols)
        return fail(ZERO_ERR_INVALID_ARG, "%s: leading dimension %lld below %lld columns", what, (long long)ld,
                    (long long)cols);
    if (!aligned(p, bytes_of(dtype)))
        return fail(ZERO_ERR_ALIGNMENT, "%s is misaligned", what);
    return ZERO_OK;
}

// The most rows, columns and leading dimension of the elementwise calls: all
// products of two of them, and byte offsets, then fit 63 bits.
constexpr int64_t kMaxDim = int64_t(1) << 40, kMaxElems = int64_t(1) << 60;

inline zero_status check_extent(int64_t rows, int64_t cols, int64_t ld)
{
    if (rows < 0 || cols < 0)
        return fail(ZERO_ERR_INVALID_ARG, "negative size");
    if (rows > kMaxDim || cols > kMaxDim || ld > kMaxDim || (ld > 0 && rows > kMaxElems / ld))
        return fail(ZERO_ERR_UNSUPPORTED, "matrix too large (%lld x %lld, leading dimension %lld)",
                    (long long)rows, (long long)cols, (long long)ld);
    return ZERO_OK;
}

}  // namespace

// A kept matrix of rows x cols (both formats).
zero_status saved_check(const char *what, const zero_saved *s, int64_t rows, int64_t cols);

}  // namespace zs
