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
    // The smallest tiles that the chip holds all at once.  64 x 64: 8 experts of 64
    // rows, H = 128, F = 256 (32 tiles) 7.4 us against 13.9 with 128 x 128 and 24 with the
    // large ones; 32 of 64, H = 1024, F = 512 (256) 20 against 24 and 38.  128 x 128: 32
    // of 256, H = 2048, F = 768 (384) 62 against 72; 16 of 1024 (768) 115 against 77.
    if (fits_chip(p, 64, 64))
        return launch_cfg<64, 64, 32, 2, 2, LAY_KC, EPI_SWIGLU_BWD8, SCHED_ROWS, kLdsBudget>(p, (hipStream_t)stream);
    if (fits_chip(p, 128, 128))
        return launch_cfg<128, 128, 32, 2, 2, LAY_KC, EPI_SWIGLU_BWD8, SCHED_ROWS, kLdsBudget>(p, (hipStream_t)stream);
    return launch<LAY_KC, EPI_SWIGLU_BWD8, SCHED_ROWS>(p, (hipStream_t)stream);
}
