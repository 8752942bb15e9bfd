// Entry points of the gate/up GroupGEMM that saves (a, b) in 8-bit blocks, on
// the permuted rows and zero-copy; the kernel template is in gemm_kernel.hpp.
#include "gemm_kernel.hpp"

using moe_host::misaligned;

namespace moe {

// Tiles of 64 rows x 64 columns of h while the chip holds them all: 8 experts of
// 64 rows, H = 128, F = 256 (32 tiles) 7.4 us against 14.3 with the large ones; 32 of
// 64, H = 1024, F = 512 (256) 24 against 32; 32 of 34, H = 7168, F = 2048 (1024) 350
// against 296.
template <bool GATHER>
static int launch_save8(const GemmParams& p, hipStream_t s) {
    if (fits_chip(p, 64, 64))
        return launch_cfg<64, 128, 32, 2, 2, LAY_MN, EPI_SWIGLU8, SCHED_ROWS, kLdsBudget, 0, GATHER>(p, s);
    return launch<LAY_MN, EPI_SWIGLU8, SCHED_ROWS, GATHER>(p, s);
}

}  // namespace moe

extern "C" int moe_grouped_gemm_swiglu_save8(const moe_bf16* x_perm, const moe_bf16* w_gate, const moe_bf16* w_up,
                                             const int32_t* offsets, int e_local, int H, int F, int cap_rows,
                                             moe_bf16* h, int8_t* ab8, uint8_t* ab8_scale, moe_stream stream) {
    using namespace moe;
    if (e_local < 0 || e_local > kMaxGroups || H <= 0 || F < 0 || cap_rows < 0) return MOE_EINVAL;
    if (H % 64 || F % 64) return MOE_ESHAPE;
    if (!offsets) return MOE_EINVAL;
    if (e_local == 0 || cap_rows == 0 || F == 0) return MOE_OK;
    if (!x_perm || !w_gate || !w_up || !h || !ab8 || !ab8_scale) return MOE_EINVAL;
    if (misaligned(x_perm) || misaligned(w_gate) || misaligned(w_up) || misaligned(offsets) || misaligned(h) ||
        misaligned(ab8) || misaligned(ab8_scale))
        return MOE_EALIGN;
    // 32-bit load offsets below 2^31 (see moe_grouped_gemm_swiglu)
    if ((int64_t)256 * H * 2 >= (1ll << 31) || (int64_t)H * F * 2 >= (1ll << 31)) return MOE_EINVAL;
    GemmParams p{};
    p.a = x_perm;
    p.lda = H;
    p.w0 = w_gate;
    p.w1 = w_up;
    p.w_stride = (int64_t)H * F;
    p.ldw = F;
    p.offsets = offsets;
    p.e_local = e_local;
    p.cap = cap_rows;
    p.N = F;
    p.Kd = H;
    p.c = h;
    p.ldc = F;
    p.q8 = ab8;
    p.s8 = ab8_scale;
    return launch_save8<false>(p, (hipStream_t)stream);
}

extern "C" int moe_grouped_gemm_swiglu_gather_save8(const moe_bf16* x, int T, const int32_t* src, int K,
                                                    const moe_bf16* w_gate, const moe_bf16* w_up,
                                                    const int32_t* offsets, int e_local, int H, int F, int cap_rows,
                                                    moe_bf16* h, int8_t* ab8, uint8_t* ab8_scale,
                                                    moe_stream stream) {
    using namespace moe;
    if (e_local < 0 || e_local > kMaxGroups || H <= 0 || F < 0 || cap_rows < 0 || T < 0 || K < 1 || K > 16)
        return MOE_EINVAL;
    if (H % 64 || F % 64) return MOE_ESHAPE;
    // as moe_grouped_gemm_swiglu_gather: load offsets below the one that masks rows
    if ((int64_t)T * H * 2 > (int64_t)kOOB_GATHER || (int64_t)H * F * 2 >= (1ll << 31)) return MOE_EINVAL;
    if ((int64_t)cap_rows > (int64_t)T * K) return MOE_EINVAL;
    if (!offsets) return MOE_EINVAL;
    if (e_local == 0 || cap_rows == 0 || F == 0) return MOE_OK;
    if (!x || !src || !w_gate || !w_up || !h || !ab8 || !ab8_scale) return MOE_EINVAL;
    if (misaligned(x) || misaligned(src) || misaligned(w_gate) || misaligned(w_up) || misaligned(offsets) ||
        misaligned(h) || misaligned(ab8) || misaligned(ab8_scale))
        return MOE_EALIGN;
    GemmParams p{};
    p.a = x;
    p.lda = H;
    p.src = src;
    p.topk = K;
    p.topk_rcp = 0xffffffffu / (uint32_t)K;
    p.a_rows = T;
    p.w0 = w_gate;
    p.w1 = w_up;
    p.w_stride = (int64_t)H * F;
    p.ldw = F;
    p.offsets = offsets;
    p.e_local = e_local;
    p.cap = cap_rows;
    p.N = F;
    p.Kd = H;
    p.c = h;
    p.ldc = F;
    p.q8 = ab8;
    p.s8 = ab8_scale;
    return launch_save8<true>(p, (hipStream_t)stream);
}
