// Selection of a token's top-k experts by one wave (route.hip has the rule).
#pragma once

#include "moe_common.hpp"

namespace moe {

__device__ __forceinline__ uint32_t score_key(float s) {
    // -0 and +0 compare equal: s + 0 is +0 for both (and s for every other s)
    const uint32_t u = __float_as_uint(s + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);  // negative: ~u; else u | sign; > 0 unless NaN
}

__device__ __forceinline__ float key_score(uint32_t u) {
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}

// max / min over the 64 lanes: butterflies within each row of 16 (quad
// permutes, half-row and row mirrors), then row broadcasts bring every row
// into lane 63.  Lanes without a DPP source take the identity.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, false));   // quad [1,0,3,2]
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, false));   // quad [2,3,0,1]
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, false));  // row_half_mirror
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, false));  // row_mirror
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));  // row_bcast:15
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));  // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ uint32_t wave_min_u32(uint32_t v) {
    const int id = -1;  // all ones: the identity of an unsigned min
    v = min(v, (uint32_t)__builtin_amdgcn_update_dpp(id, (int)v, 0xB1, 0xf, 0xf, false));
    v = min(v, (uint32_t)__builtin_amdgcn_update_dpp(id, (int)v, 0x4E, 0xf, 0xf, false));
    v = min(v, (uint32_t)__builtin_amdgcn_update_dpp(id, (int)v, 0x141, 0xf, 0xf, false));
    v = min(v, (uint32_t)__builtin_amdgcn_update_dpp(id, (int)v, 0x140, 0xf, 0xf, false));
    v = min(v, (uint32_t)__builtin_amdgcn_update_dpp(id, (int)v, 0x142, 0xa, 0xf, false));
    v = min(v, (uint32_t)__builtin_amdgcn_update_dpp(id, (int)v, 0x143, 0xc, 0xf, false));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// The K rounds of a wave maximum, for one token whose lane l holds the keys of experts
// l, l + 64, ... (0: absent or taken).  On return lane k < K holds choice k
// (its expert id and score); s_max is the best score.
template <int EPL>
__device__ __forceinline__ void select_rounds(uint32_t (&key)[EPL], int K, int lane, int& my_idx, float& my_score,
                                              float& s_max) {
    my_idx = 0;
    my_score = 0.0f;
    s_max = 0.0f;
    for (int k = 0; k < K; ++k) {
        // the lane's best remaining key; strict > keeps the lowest slot on a tie
        uint32_t best = key[0];
        int bj = 0;
#pragma unroll
        for (int i = 1; i < EPL; ++i)
            if (key[i] > best) {
                best = key[i];
                bj = i;
            }
        const uint32_t m = wave_max_u32(best);
        const uint64_t tied = __ballot(best == m);
        int e_win;
        if (__popcll(tied) == 1) {
            const int wl = __builtin_ctzll(tied);
            e_win = __builtin_amdgcn_readlane(bj, wl) * 64 + wl;
        } else {
            // several lanes hold this score: the lowest expert id among them
            e_win = (int)wave_min_u32(best == m ? (uint32_t)(bj * 64 + lane) : 0xffffffffu);
        }
        e_win = __builtin_amdgcn_readfirstlane(e_win);
        if (lane == (e_win & 63)) {
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (i == (e_win >> 6)) key[i] = 0u;
        }
        const float sc = key_score(m);
        if (k == 0) s_max = sc;
        if (lane == k) {
            my_idx = e_win;
            my_score = sc;
        }
    }
}

}  // namespace moe
