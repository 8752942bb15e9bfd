// Entry point of the down dgrad with the SwiGLU backward from (a, b) saved in
// 8-bit blocks; the kernel template is in gemm_kernel.hpp.
#include "gemm_kernel.hpp"

using moe_host::misaligned;

extern "C" int moe_grouped_gemm_swiglu_bwd8(const moe_bf16* dy_perm, const moe_bf16* w_down, const int32_t* offsets,
                                            int e_local, int H, int F, int cap_rows, const int8_t* ab8,
                                            const uint8_t* ab8_scale, moe_bf16* dab, moe_bf16* h,
                                            moe_stream stream) {
    using namespace moe;
    if (e_local < 0 || e_local > kMaxGroups || H <= 0 || F < 0 || cap_rows < 0) return MOE_EINVAL;
    if (H % 64 || F % 64) return MOE_ESHAPE;
    if (!offsets) return MOE_EINVAL;
    if (e_local == 0 || cap_rows == 0 || F == 0) return MOE_OK;
    if (!dy_perm || !w_down || !ab8 || !ab8_scale || !dab) return MOE_EINVAL;
    if (misaligned(dy_perm) || misaligned(w_down) || misaligned(offsets) || misaligned(ab8) ||
        misaligned(ab8_scale) || misaligned(dab) || misaligned(h))
        return MOE_EALIGN;
    // 32-bit load offsets below 2^31 (see moe_grouped_gemm_swiglu)
    if ((int64_t)256 * H * 2 >= (1ll << 31) || (int64_t)H * F * 2 >= (1ll << 31)) return MOE_EINVAL;
    GemmParams p{};
    p.a = dy_perm;
    p.lda = H;
    p.w0 = w_down;
    p.w_stride = (int64_t)H * F;
    p.ldw = H;
    p.offsets = offsets;
    p.e_local = e_local;
    p.cap = cap_rows;
    p.N = F;
    p.Kd = H;
    p.c = dab;
    p.ldc = 2 * F;
    p.c2 = h;
    p.q8 = const_cast<int8_t*>(ab8);
    p.s8 = const_cast<uint8_t*>(ab8_scale);
    // The smallest tiles that the chip holds all at once, whatever the contraction.  us for 64 x 64, 128 x 128 and
    // the large ones, routed rows (Poisson about the mean) on full buffers: 8 experts of 64 rows, H = 128, F = 256 (32
    // tiles) 7.4, 13.9, 24; 8 of 64, F = 2048 (256) at H = 1024 20, 25, 39, at 4096 46, 51, 76, at 7168 93, 102, 140;
    // 32 of 32, F = 1024 (512) 19, 27, 30, then 65, 90, 82, then 122, 168, 161; 32 of 100, F = 512 (512) 21, 28, 41,
    // then 45, 56, 81, then 101, 120, 165.  They lose where the mean fills its tiles and the chip, so that the spread
    // needs a second round: 8 of 128, F = 2048 (512) 34, 30, 52, then 81, 58, 93, then 162, 112, 160 (with buffers of
    // twice the rows, which the sizes do not tell from these: 32 of 64, F = 512 20, 26, 40, then 46, 52, 77, then 111,
    // 105, 144).  128 x 128 against the large ones: 32 of 256, F = 768 (384 of 128 rows) at H = 2048 63 against 73, at
    // 4096 122 against 128, at 7168 205 against 194; 16 of 1024 (768, so the large ones), H = 2048 115 against 77.
    if (fits_chip(p, 64, 64))
        return launch_cfg<64, 64, 32, 2, 2, LAY_KC, EPI_SWIGLU_BWD8, SCHED_ROWS, kLdsBudget>(p, (hipStream_t)stream);
    if (fits_chip(p, 128, 128))
        return launch_cfg<128, 128, 32, 2, 2, LAY_KC, EPI_SWIGLU_BWD8, SCHED_ROWS, kLdsBudget>(p, (hipStream_t)stream);
    return launch<LAY_KC, EPI_SWIGLU_BWD8, SCHED_ROWS>(p, (hipStream_t)stream);
}
