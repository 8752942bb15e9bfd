// The activations of the dense product and their slopes.
#pragma once

#include "moe_common.hpp"

namespace moe {

__device__ __forceinline__ f32x4 widen4(u32x2 v) { return f32x4{bf_lo(v[0]), bf_hi(v[0]), bf_lo(v[1]), bf_hi(v[1])}; }

// P(N(0,1) <= z), and e = exp(-z^2 / 2).  With a = |z| and t = 1 / (1 + 0.2644 a) the lower tail P(N(0,1) <= -a) is
// e * t * (a polynomial of degree 6 in t), fitted over 0 <= a <= 14 to the smallest greatest relative error (6e-7; 9e-7 in
// fp32, and the square's rounding in the exponent, z^2 * 2^-24, from there on).  A library's error function is three times as
// many instructions, and the 256 copies of it in the epilogue of a 256 x 256 tile do not fit the instruction cache.
__device__ __forceinline__ float normal_cdf(float z, float& e) {
    const float t = __builtin_amdgcn_rcpf(fmaf(0.26442201f, fabsf(z), 1.0f));
    e = __builtin_amdgcn_exp2f(-0.72134752f * z * z);
    float s = fmaf(-0.0686337128f, t, 0.199908718f);
    s = fmaf(s, t, -0.0719699413f);
    s = fmaf(s, t, 0.145972669f);
    s = fmaf(s, t, 0.0815478042f);
    s = fmaf(s, t, 0.107820027f);
    s = fmaf(s, t, 0.105354145f);
    const float q = s * t * e;
    return z > 0.0f ? 1.0f - q : q;
}

// gelu(z) = z * P(N(0,1) <= z)
__device__ __forceinline__ float gelu_f(float z) {
    float e;
    return z * normal_cdf(z, e);
}

// f = act(f)
template <int ACT>
__device__ __forceinline__ void activate(f32x4& f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (ACT == MOE_ACT_RELU) f[i] = f[i] < 0.0f ? 0.0f : f[i];  // a NaN stays
        if (ACT == MOE_ACT_SILU) f[i] = silu_f(f[i]);
        if (ACT == MOE_ACT_GELU) f[i] = gelu_f(f[i]);
    }
}
// the same with an activation that is known at run time, the same in every lane
__device__ __forceinline__ void activate(f32x4& f, int act) {
    if (act == MOE_ACT_RELU) activate<MOE_ACT_RELU>(f);
    else if (act == MOE_ACT_SILU) activate<MOE_ACT_SILU>(f);
    else if (act == MOE_ACT_GELU) activate<MOE_ACT_GELU>(f);
}

// d act / dz
__device__ __forceinline__ float slope(float z, int act) {
    if (act == MOE_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if (act == MOE_ACT_SILU) {
        const float s = sigmoid_f(z);
        return s * (1.0f + z * (1.0f - s));
    }
    if (act == MOE_ACT_GELU) {
        float e;
        const float c = normal_cdf(z, e);
        return fmaf(z * 0.39894228f, e, c);
    }
    return 1.0f;
}

}  // namespace moe
