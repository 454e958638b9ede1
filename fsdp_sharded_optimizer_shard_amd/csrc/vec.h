// Eight neighbouring values at a time, in bf16, fp32 or codes: one or two
// 16-byte (codes: 8-byte) accesses where the caller says that all are there, else one
// by one.  Device memory takes such an access at any element's address (a misaligned one
// touches one more line), LDS does not.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace zs {
namespace {

typedef uint32_t Words4 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t Words2 __attribute__((ext_vector_type(2), aligned(1)));

__device__ __forceinline__ uint4 load16(const void *q)
{
    const Words4 w = *static_cast<const Words4 *>(q);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store16(void *q, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    *static_cast<Words4 *>(q) = Words4{a, b, c, d};
}

// Two values to bf16, nearest even, the first in the low half: one
// v_cvt_pk_bf16_f32.  NaN stays NaN.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

// Eight bf16 to fp32.
__device__ __forceinline__ void widen8(uint4 w, float (&x)[8])
{
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[2 * k] = __uint_as_float(ww[k] << 16);
        x[2 * k + 1] = __uint_as_float(ww[k] & 0xffff0000u);
    }
}

// x[0 .. n) of 8 neighbouring values of dtype DT at element i; `vec`: n is 8, and the
// values are read at once.
__device__ __forceinline__ void load8(const void *p, bool bf16, int64_t i, bool vec, int n, float (&x)[8])
{
    if (bf16) {
        const uint16_t *q = static_cast<const uint16_t *>(p) + i;
        if (vec) {
            widen8(load16(q), x);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = k < n ? __uint_as_float((uint32_t)q[k] << 16) : 0.0f;
        }
    } else {
        const float *q = static_cast<const float *>(p) + i;
        if (vec) {
            const uint4 a = load16(q), b = load16(q + 4);
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = __uint_as_float(w[k]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = k < n ? q[k] : 0.0f;
        }
    }
}

__device__ __forceinline__ void store8(void *p, bool bf16, int64_t i, bool vec, int n, const float (&x)[8])
{
    if (bf16) {
        uint16_t *q = static_cast<uint16_t *>(p) + i;
        const uint32_t h[4] = {pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                               pack_bf16(x[6], x[7])};
        if (vec) {
            store16(q, h[0], h[1], h[2], h[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n)
                    q[k] = (uint16_t)(h[k >> 1] >> (16 * (k & 1)));
        }
    } else {
        float *q = static_cast<float *>(p) + i;
        if (vec) {
            store16(q, __float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
            store16(q + 4, __float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n)
                    q[k] = x[k];
        }
    }
}

__device__ __forceinline__ uint2 load_bytes8(const uint8_t *q, bool vec, int n)
{
    if (vec) {
        const Words2 w = *reinterpret_cast<const Words2 *>(q);
        return make_uint2(w[0], w[1]);
    }
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < n)
            w[k >> 2] |= (uint32_t)q[k] << (8 * (k & 3));
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store_bytes8(uint8_t *q, bool vec, int n, uint2 w)
{
    if (vec) {
        *reinterpret_cast<Words2 *>(q) = Words2{w.x, w.y};
        return;
    }
    const uint32_t ww[2] = {w.x, w.y};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < n)
            q[k] = (uint8_t)(ww[k >> 2] >> (8 * (k & 3)));
}

}  // namespace
}  // namespace zs
