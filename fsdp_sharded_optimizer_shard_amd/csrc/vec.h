// Eight neighbouring values at a time, in bf16, fp32 or codes: one or two
// 16-byte (codes: 8-byte) accesses where the address allows, else one by one.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace zs {
namespace {

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

// x[0 .. n) of 8 neighbouring values of dtype DT at element i; `vec`: the
// address is 16-byte aligned (and n is 8).
__device__ __forceinline__ void load8(const void *p, bool bf16, int64_t i, bool vec, int n, float (&x)[8])
{
    if (bf16) {
        const uint16_t *q = static_cast<const uint16_t *>(p) + i;
        if (vec) {
            widen8(*reinterpret_cast<const uint4 *>(q), x);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                x[k] = k < n ? __uint_as_float((uint32_t)q[k] << 16) : 0.0f;
        }
    } else {
        const float *q = static_cast<const float *>(p) + i;
        if (vec) {
            const float4 a = *reinterpret_cast<const float4 *>(q);
            const float4 b = *reinterpret_cast<const float4 *>(q + 4);
            x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
            x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
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
            *reinterpret_cast<uint4 *>(q) = make_uint4(h[0], h[1], h[2], h[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n)
                    q[k] = (uint16_t)(h[k >> 1] >> (16 * (k & 1)));
        }
    } else {
        float *q = static_cast<float *>(p) + i;
        if (vec) {
            *reinterpret_cast<float4 *>(q) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4 *>(q + 4) = make_float4(x[4], x[5], x[6], x[7]);
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
    if (vec)
        return *reinterpret_cast<const uint2 *>(q);
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
        *reinterpret_cast<uint2 *>(q) = w;
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
