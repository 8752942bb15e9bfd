// The activations of the dense product and their slopes.
#pragma once

#include "moe_common.hpp"

namespace moe {

__device__ __forceinline__ f32x4 widen4(u32x2 v) { return f32x4{bf_lo(v[0]), bf_hi(v[0]), bf_lo(v[1]), bf_hi(v[1])}; }

// gelu(z) = z * P(N(0,1) <= z)
__device__ __forceinline__ float gelu_f(float z) { return 0.5f * z * (1.0f + erff(z * 0.70710678f)); }

// f = act(f); act is the same in every lane
__device__ __forceinline__ void activate(f32x4& f, int act) {
    if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = f[i] < 0.0f ? 0.0f : f[i];  // a NaN stays
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = silu_f(f[i]);
    } else if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = gelu_f(f[i]);
    }
}

// d act / dz
__device__ __forceinline__ float slope(float z, int act) {
    if (act == MOE_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if (act == MOE_ACT_SILU) {
        const float s = sigmoid_f(z);
        return s * (1.0f + z * (1.0f - s));
    }
    if (act == MOE_ACT_GELU)
        return 0.5f * (1.0f + erff(z * 0.70710678f)) + z * __expf(-0.5f * z * z) * 0.39894228f;
    return 1.0f;
}

}  // namespace moe
