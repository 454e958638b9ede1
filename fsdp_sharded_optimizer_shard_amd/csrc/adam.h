// One element's Adam / AdamW update and its step scalars, shared by the shard
// step and the step over many tensors.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "zero_shard.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

// The step scalars; the same layout as zero_adam_table_entry, so a table of
// them in device memory can be read as is.
struct AdamScalars {
    float lr, b1, b2, eps, wd;
    float omb1, omb2, bias1, bias2, decay;
    int32_t has_wd, decoupled;
};
static_assert(sizeof(AdamScalars) == sizeof(zero_adam_table_entry), "table entry layout");
static_assert(offsetof(AdamScalars, omb1) == offsetof(zero_adam_table_entry, one_minus_beta1) &&
                  offsetof(AdamScalars, decay) == offsetof(zero_adam_table_entry, decay) &&
                  offsetof(AdamScalars, has_wd) == offsetof(zero_adam_table_entry, has_decay) &&
                  offsetof(AdamScalars, decoupled) == offsetof(zero_adam_table_entry, decoupled),
              "table entry layout");

__device__ __forceinline__ void adam1(const AdamScalars &s, float g, float &p, float &m, float &v)
{
    if (s.has_wd) {
        if (s.decoupled)
            p = p * s.decay;
        else
            g = g + s.wd * p;
    }
    m = s.b1 * m + s.omb1 * g;
    v = s.b2 * v + s.omb2 * (g * g);
    const float m_hat = m / s.bias1;
    const float v_hat = v / s.bias2;
    const float denom = sqrtf(v_hat) + s.eps;
    p = p - s.lr * (m_hat / denom);
}

}  // namespace
}  // namespace zs
