// Block-scaled storage: 32 values share one power-of-two scale byte s (the OCP
// microscaling element types int8 and E2M1), device helpers.
//
// 8 bits (rows of saved activations, blocks along the row): with m the largest
// magnitude of the block,
//   s = max(biased exponent of m, 7),  q = clamp(rint(x * 2^(133-s)), -127, 127),
//   value = q * 2^(s-133).
// m * 2^(133-s) is below 128 (at most 127.5 for a bf16 m, so the clamp costs
// no more than the half step of the rounding), and |value - x| <= 2^(s-134),
// which is at most m / 128 while s is m's own exponent (m >= 2^-120).  The
// products with the powers of two are exact, and the value has at most 7
// significant bits, so it is a bf16.  s >= 7 keeps the step 2^(s-133) a normal
// number; below it the error is up to 2^-127, which may be all of x.  A block
// with a NaN or an infinity gets s = 255 and q = 0 and stands for NaN.
//
// 4 bits (weights, blocks along the contraction): s = max(biased exponent of m - 2, 2),
// value = c * 2^(s-127) with c one of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}, rounded to
// nearest even and saturated at 6 by the chip's conversion; s = 255 as above.
// s << 23 is the scale as a float; for 255 that is an infinity, with which the
// chip's conversion back gives NaN for every code.
#pragma once

#include "moe_common.hpp"

namespace moe {

typedef __attribute__((ext_vector_type(2))) uint16_t u16x2;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;

// Larger of two packed pairs of bf16 magnitudes, taken as 16-bit integers
// (the order of the magnitudes; NaN and infinity above everything).
__device__ __forceinline__ uint32_t max_mag2(uint32_t a, uint32_t b) {
    const u16x2 r = __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b));
    return __builtin_bit_cast(uint32_t, r);
}

// Scale byte of an 8-bit block whose largest bf16 magnitude has the bits m.
__device__ __forceinline__ uint32_t scale8_of(uint32_t m) { return max(m >> 7, 7u); }

// 2^(133-s), the factor before rounding (s = 7..254).
__device__ __forceinline__ float inv_step8(uint32_t s) { return __uint_as_float((260u - s) << 23); }

// 2^(s-133), the value of one step; NaN for s = 255 (and for s < 7, which no
// block has, the smallest step).
__device__ __forceinline__ float step8(uint32_t s) {
    return __uint_as_float(s == 255u ? 0x7fc00000u : (max(s, 7u) - 6u) << 23);
}

// Four values to four signed bytes.  After the clamp, adding 1.5 * 2^23 leaves
// the nearest-even integer in the low bits of the sum.
__device__ __forceinline__ uint32_t quant8x4(float x0, float x1, float x2, float x3, float inv) {
    auto one = [&](float x) {
        return __float_as_uint(__builtin_amdgcn_fmed3f(x * inv, -127.0f, 127.0f) + 12582912.0f);
    };
    const uint32_t lo = __builtin_amdgcn_perm(one(x1), one(x0), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(one(x3), one(x2), 0x04000c0cu);
    return lo | hi;
}

// 8 bf16 of a block that four neighbouring lanes hold (lanes 4i .. 4i+3) to
// their bytes; s is the block's scale byte, the same in the four lanes.
__device__ __forceinline__ u32x2 pack8_lane(u32x4 v, uint32_t& s) {
    uint32_t m = max_mag2(max_mag2(v[0] & 0x7fff7fffu, v[1] & 0x7fff7fffu),
                          max_mag2(v[2] & 0x7fff7fffu, v[3] & 0x7fff7fffu));
    m = max(m & 0xffffu, m >> 16);
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xb1, 0xf, 0xf, true));  // lane ^ 1
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4e, 0xf, 0xf, true));  // lane ^ 2
    s = scale8_of(m);
    const float inv = inv_step8(s);
    u32x2 o = {quant8x4(bf_lo(v[0]), bf_hi(v[0]), bf_lo(v[1]), bf_hi(v[1]), inv),
               quant8x4(bf_lo(v[2]), bf_hi(v[2]), bf_lo(v[3]), bf_hi(v[3]), inv)};
    if (s == 255u) o = u32x2{0u, 0u};
    return o;
}

// Signed byte i of w as a float.
template <int I>
__device__ __forceinline__ float byte_f32(uint32_t w) {
    return (float)((int32_t)(w << (24 - 8 * I)) >> 24);
}

// Two exact bf16 values held as floats, packed by their upper halves.
__device__ __forceinline__ uint32_t pack_hi2(float lo, float hi) {
    return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

// Four signed bytes times the step, as two packed bf16 pairs (exact).
__device__ __forceinline__ u32x2 dequant8x4(uint32_t w, float step) {
    return u32x2{pack_hi2(byte_f32<0>(w) * step, byte_f32<1>(w) * step),
                 pack_hi2(byte_f32<2>(w) * step, byte_f32<3>(w) * step)};
}

}  // namespace moe
