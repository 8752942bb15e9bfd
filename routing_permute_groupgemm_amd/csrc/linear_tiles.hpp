// The dense product on the GroupGEMM's kernel for one activation, each compiled in a translation unit of its own
// (linear_none.hip, linear_relu.hip, linear_silu.hip, linear_gelu.hip).
#pragma once

#include "gemm_kernel.hpp"

namespace moe {

enum : int { TILES_SMALL = 1, TILES_MID = 2, TILES_BIG = 3 };  // 128 x 128, 128 x 256, 256 x 256

template <int EPI>
static int launch_linear_epi(const GemmParams& p, int tiles, hipStream_t s) {
    // eight waves, two a SIMD, run the two smaller tiles 5 to 20% faster than four
    if (tiles == TILES_SMALL) return launch_cfg<128, 128, 32, 2, 4, LAY_MN, EPI, SCHED_ROWS, kDeepBudget>(p, s);
    if (tiles == TILES_MID) return launch_cfg<128, 256, 32, 2, 4, LAY_MN, EPI, SCHED_ROWS, kLdsBudget>(p, s);
    return launch_cfg<256, 256, 32, 2, 2, LAY_MN, EPI, SCHED_ROWS, kLdsBudget>(p, s);
}

template <int ACT>
static int launch_linear_act(const GemmParams& p, int tiles, hipStream_t s) {
    if (p.res) {
        if (p.c2) return launch_linear_epi<EPI_LINEAR + ACT + 12>(p, tiles, s);
        return launch_linear_epi<EPI_LINEAR + ACT + 4>(p, tiles, s);
    }
    if (p.c2) return launch_linear_epi<EPI_LINEAR + ACT + 8>(p, tiles, s);
    return launch_linear_epi<EPI_LINEAR + ACT>(p, tiles, s);
}

int launch_linear_none(const GemmParams& p, int tiles, hipStream_t s);
int launch_linear_relu(const GemmParams& p, int tiles, hipStream_t s);
int launch_linear_silu(const GemmParams& p, int tiles, hipStream_t s);
int launch_linear_gelu(const GemmParams& p, int tiles, hipStream_t s);

}  // namespace moe
