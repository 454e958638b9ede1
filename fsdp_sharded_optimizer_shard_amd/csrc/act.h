// Activations, their slopes and the 8-bit code of the layer operators, in
// fp32 device code.
//
// The sigmoid family goes through E = exp(-|u|) <= 1 and r = 1 / (1 + E):
// sigmoid(u) = r for u >= 0, E r below, and its slope factor
// sigmoid (1 - sigmoid) = E r^2 on both sides, so nothing cancels and nothing
// overflows.  exp is v_exp_f32 of u log2(e) (1 ulp, plus the argument's
// rounding: |u| 2^-24 relative) and the reciprocal v_rcp_f32 (1 ulp).
//
// The normal distribution function is 1/2 erfc(-z / sqrt 2).  With
// a = |z| / sqrt 2 and t = 1 / (1 + 0.3 a), 1/2 erfc(a) e^(a^2) = t P(t), P the
// degree-8 polynomial of least relative error on a in [0, 10] (2e-8, fitted
// by reweighted least squares on Chebyshev points against 64-bit values).
// Writing the tail as a product keeps its relative precision, which
// 1 + erf(z / sqrt 2) loses for negative z; the slope z phi(z) shares its
// exponential.  Its fp32 evaluation is within 9e-7 of 64 bits (relative) for
// z > -4 and within 3e-6 down to -8, where the rounding of z^2 in the
// exponent decides.
//
// An exponential below fp32's normal numbers comes as 0, so values and slopes
// under 2^-117 may: silu past -87, gelu_tanh past -10, gelu past -13.
//
// Infinities: every activation takes its limit (gelu(-inf) = silu(-inf) = -0,
// slopes 0 and 1); NaN stays NaN.
#pragma once

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

#include "zero_shard.h"

namespace zs {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp_neg(float a)  // exp(-a), a >= 0
{
    return __builtin_amdgcn_exp2f(-a * kLog2e);
}

// sigmoid(u), and in q the factor sigmoid (1 - sigmoid).
__device__ __forceinline__ float sigmoid(float u, float &q)
{
    const float e = exp_neg(__builtin_fabsf(u));
    const float r = __builtin_amdgcn_rcpf(1.0f + e);
    const float er = e * r;
    q = er * r;
    return u < 0.0f ? er : r;
}

// Phi(z), and in g exp(-z^2 / 2).
__device__ __forceinline__ float normal_cdf(float z, float &g)
{
    const float a = __builtin_fabsf(z);
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(a, 0.21213203435596426f, 1.0f));
    g = __builtin_amdgcn_exp2f(a * a * (-0.5f * kLog2e));
    float p = -0.064761624f;
    p = __builtin_fmaf(p, t, 0.24278247f);
    p = __builtin_fmaf(p, t, -0.25614092f);
    p = __builtin_fmaf(p, t, 0.27386227f);
    p = __builtin_fmaf(p, t, -0.047327001f);
    p = __builtin_fmaf(p, t, 0.10746377f);
    p = __builtin_fmaf(p, t, 0.074169382f);
    p = __builtin_fmaf(p, t, 0.085357644f);
    p = __builtin_fmaf(p, t, 0.084594004f);
    const float q = p * t * g;
    return z < 0.0f ? q : 1.0f - q;
}

// -inf times a zero sigmoid would be NaN; the lowest finite value gives -0.
// (A NaN may come back as the bound: every caller multiplies it by a sigmoid
// that is NaN then.)
__device__ __forceinline__ float finite_low(float z)
{
    return __builtin_amdgcn_fmed3f(z, -FLT_MAX, __builtin_inff());
}
// Past +-128 every slope's second term is 0 -- silu's e^-|z|, the slowest to
// go, leaves fp32 at 104 -- and the bound keeps it from 0 * inf.
__device__ __forceinline__ float bound128(float z) { return __builtin_amdgcn_fmed3f(z, -128.0f, 128.0f); }

constexpr float kTanhK = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

template <int ACT>
__device__ __forceinline__ float act(float z)
{
    float q;
    if constexpr (ACT == ZERO_ACT_RELU)
        return z < 0.0f ? 0.0f : z;
    else if constexpr (ACT == ZERO_ACT_GELU)
        return finite_low(z) * normal_cdf(z, q);
    else if constexpr (ACT == ZERO_ACT_GELU_TANH)
        return finite_low(z) * sigmoid(kTanhK * z * __builtin_fmaf(0.044715f * z, z, 1.0f), q);
    else if constexpr (ACT == ZERO_ACT_SILU)
        return finite_low(z) * sigmoid(z, q);
    else
        return z;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float z)
{
    float q;
    if constexpr (ACT == ZERO_ACT_RELU) {
        return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
    } else if constexpr (ACT == ZERO_ACT_GELU) {
        const float c = normal_cdf(z, q);
        return __builtin_fmaf(bound128(z) * kInvSqrt2Pi, q, c);
    } else if constexpr (ACT == ZERO_ACT_GELU_TANH) {
        const float b = bound128(z);
        const float s = sigmoid(kTanhK * z * __builtin_fmaf(0.044715f * z, z, 1.0f), q);
        return __builtin_fmaf(b * q, kTanhK * __builtin_fmaf(3.0f * 0.044715f * b, b, 1.0f), s);
    } else if constexpr (ACT == ZERO_ACT_SILU) {
        const float s = sigmoid(z, q);
        return __builtin_fmaf(bound128(z), q, s);
    } else {
        return 1.0f;
    }
}

// f with the activation as a constant; on the device `a` is the same in every
// lane.
template <class F>
__host__ __device__ __forceinline__ void by_act(int a, F f)
{
    switch (a) {
    case ZERO_ACT_RELU: f(std::integral_constant<int, ZERO_ACT_RELU>{}); break;
    case ZERO_ACT_GELU: f(std::integral_constant<int, ZERO_ACT_GELU>{}); break;
    case ZERO_ACT_GELU_TANH: f(std::integral_constant<int, ZERO_ACT_GELU_TANH>{}); break;
    case ZERO_ACT_SILU: f(std::integral_constant<int, ZERO_ACT_SILU>{}); break;
    default: f(std::integral_constant<int, ZERO_ACT_NONE>{}); break;
    }
}

// ---- the 8-bit code: e4m3 values under one exponent per 32 rows of a column

constexpr uint32_t kInf = 0x7f800000u;

// The magnitude bits that count for a block's largest value: 0 for NaN and
// infinities, which become NaN codes whatever the exponent.
__device__ __forceinline__ uint32_t mag_bits(float x)
{
    const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
    return u < kInf ? u : 0u;
}

// e + 127 for the least e in [-117, 120] with max <= 448 * 2^e (448 = 1.75 * 2^8):
// the bits of max give its exponent and whether its mantissa is past 1.75.
// -117 is the least e at which the smallest code, 2^-9 2^e, is a normal bf16.
__device__ __forceinline__ uint32_t block_byte(uint32_t max_bits)
{
    const int e = (int)(max_bits >> 23) - 8 + ((max_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)(e < 10 ? 10 : e > 247 ? 247 : e);
}

// 2^-e for the byte e + 127 (2^-120 .. 2^117, normal).
__device__ __forceinline__ float inv_scale(uint32_t byte)
{
    return __uint_as_float((254u - byte) << 23);
}

// x as the coder takes it: NaN and infinities to NaN, |x| to at most
// 240 * 2^120, so that no code stands for more than bf16 holds.
__device__ __forceinline__ float coder_in(float x)
{
    const float lim = 0x1.ep127f;
    const bool fine = (__float_as_uint(x) & 0x7fffffffu) < kInf;
    const float c = x > lim ? lim : x < -lim ? -lim : x;
    return fine ? c : __builtin_nanf("");
}

// Four codes, lowest byte first.  v_cvt_pk_fp8_f32 rounds to nearest even;
// |x| 2^-e <= 448 always.
__device__ __forceinline__ uint32_t code4(float a, float b, float c, float d)
{
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, lo, true);
}

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Byte i of two code words under its column's exponent byte, exactly.
__device__ __forceinline__ void decode8(uint2 w, uint2 bytes, float (&x)[8])
{
    const uint32_t ww[2] = {w.x, w.y}, bb[2] = {bytes.x, bytes.y};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)ww[h], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)ww[h], true);
        const float v[4] = {lo[0], lo[1], hi[0], hi[1]};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[4 * h + i] = v[i] * __uint_as_float(((bb[h] >> (8 * i)) & 0xffu) << 23);
    }
}

}  // namespace
}  // namespace zs
