// Entry points of the gate/up GroupGEMM that saves (a, b) in 8-bit blocks, on
// the permuted rows and zero-copy; the kernel template is in gemm_kernel.hpp.
#include "gemm_kernel.hpp"

using moe_host::misaligned;

namespace moe {

// Whether tiles of 64 rows x 64 columns of h are the faster ones: where the chip holds them all and their weights
// are few or short.  A panel is one expert's 64 columns of both matrices.  Its rows are 128 bytes, half a large
// tile's, and what several tiles read of it comes from the L2, so the small tiles' advantage, more CUs at work,
// goes with the panels and with the contraction.  Small against large tiles, us, routed rows (Poisson about the
// mean) on full buffers unless said otherwise:
//   H = 128:  8 experts of 64 rows, F = 256 (32 panels) 7.4 against 14.3
//   H = 512:  32 of 64, F = 1024 (512 panels) 26 against 26; 32 of 32 20 against 23
//   H = 1024: 32 of 64, F = 512 (256) 24 against 33, F = 1024 (512) 42 against 37
//   H = 2048: the same 37 against 53 and 98 against 61; 8 of 64, F = 1024 (128) 24 against 46; 8 of 256, F = 1024
//             (128, 512 tiles) 55 against 48; 8 of 48, F = 2048 (256) 54 against 48
//   H = 2560: 32 of 64, F = 512 (256) 54 against 65, of 100 45 against 70; 8 of 256, F = 1024 (128) 70 against 56
//   H = 3584: 8 of 64, F = 2048 (256) 66 against 79; 32 of 32, F = 512 (256) 84 against 72
//   H = 4096: 32 of 64, F = 512 (256) 99 against 96, F = 1024 (512) 200 against 105; 8 of 128, F = 1024 (128) 59
//             against 92, of 256 96 against 76; 8 of 64, F = 1536 (192) 63 against 85, of 48 101 against 81
//   H = 7168: 32 of 64, F = 512 (256) 177 against 155, F = 1024 (512) 322 against 175; 8 of 128, F = 1024 (128) 99
//             against 148, of 256 (512 tiles) 175 against 127; 8 of 64, F = 1536 (192) 173 against 140
// Buffers of twice the rows (a share of the experts) are not told from full ones by the sizes: 8 of 128, F = 1024,
// H = 4096 61 against 93 with them, H = 7168 109 against 149, which the rule gives to the large tiles.
static bool small_save8(const GemmParams& p) {
    if (!fits_chip(p, 64, 64)) return false;
    const int64_t cus = moe_host::num_cus(), panels = (int64_t)p.e_local * (p.N / 64);
    if (panels > cus) return p.Kd <= 512;
    if (p.Kd <= 3584) return true;
    if (p.Kd <= 4096) return panels <= 3 * cus / 4;
    return panels <= cus / 2 && fits_chip(p, 64, 64, 1);
}

template <bool GATHER>
static int launch_save8(const GemmParams& p, hipStream_t s) {
    if (small_save8(p))
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
