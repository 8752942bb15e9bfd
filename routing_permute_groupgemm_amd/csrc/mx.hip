// Packing and unpacking of block-scaled storage (formats in mx.hpp): rows of
// activations in 8 bits, expert weights in 4 bits.  All four passes are bound
// by the memory they stream; each value is read and written once.
#include "mx.hpp"

namespace moe {

// Rows to process: all, or the routed rows offsets[e_local] if fewer.
__device__ __forceinline__ int64_t live_rows(const int32_t* offsets, int e_local, int64_t rows) {
    if (!offsets) return rows;
    const int64_t r = offsets[e_local];
    return r < rows ? (r > 0 ? r : 0) : rows;
}

// 8 columns per lane (16 bytes in, 8 out), so 4 lanes hold a block of 32: its
// largest magnitude is a maximum over the lane's pairs and two lane exchanges.
// Two chunks of a lane are in flight together, and one workgroup takes 512: with
// as many short workgroups as there is work, 125808 x 4096 ran in 241 us (6.5 TB/s;
// unpack8 242), against 283 with 8 persistent ones per CU and 317 with a chunk at
// a time.  NT: non-temporal on both sides, for rows of 64 MiB or more (a quarter
// of the last-level cache, as in the combine), which no cache holds until the
// backward reads them; without it 274 us.
constexpr int kChunks = 2;
template <bool NT>
__global__ __launch_bounds__(256) void pack8_kernel(const u32x4* __restrict__ x, int64_t rows, int cols8,
                                                    const int32_t* __restrict__ offsets, int e_local,
                                                    u32x2* __restrict__ q, uint8_t* __restrict__ scale) {
    const int64_t n = live_rows(offsets, e_local, rows) * cols8;  // a multiple of 8: blocks are whole
    for (int64_t i0 = (int64_t)blockIdx.x * (256 * kChunks); i0 < n; i0 += (int64_t)gridDim.x * (256 * kChunks)) {
        u32x4 v[kChunks];
#pragma unroll
        for (int u = 0; u < kChunks; ++u) {
            const int64_t i = i0 + u * 256 + threadIdx.x;
            v[u] = u32x4{0u, 0u, 0u, 0u};
            if (i < n) v[u] = NT ? __builtin_nontemporal_load(x + i) : x[i];
        }
#pragma unroll
        for (int u = 0; u < kChunks; ++u) {
            const int64_t i = i0 + u * 256 + threadIdx.x;
            uint32_t s;
            const u32x2 o = pack8_lane(v[u], s);
            if (i < n) {
                if (NT) __builtin_nontemporal_store(o, q + i);
                else q[i] = o;
                if ((threadIdx.x & 3) == 0) scale[i >> 2] = (uint8_t)s;
            }
        }
    }
}

template <bool NT>
__global__ __launch_bounds__(256) void unpack8_kernel(const u32x2* __restrict__ q, const uint8_t* __restrict__ scale,
                                                      int64_t rows, int cols8, const int32_t* __restrict__ offsets,
                                                      int e_local, u32x4* __restrict__ x) {
    const int64_t n = live_rows(offsets, e_local, rows) * cols8;
    for (int64_t i0 = (int64_t)blockIdx.x * (256 * kChunks); i0 < n; i0 += (int64_t)gridDim.x * (256 * kChunks)) {
        u32x2 v[kChunks];
        uint32_t s[kChunks];
#pragma unroll
        for (int u = 0; u < kChunks; ++u) {
            const int64_t i = i0 + u * 256 + threadIdx.x;
            v[u] = u32x2{0u, 0u};
            s[u] = 127u;
            if (i < n) {
                v[u] = NT ? __builtin_nontemporal_load(q + i) : q[i];
                s[u] = scale[i >> 2];
            }
        }
#pragma unroll
        for (int u = 0; u < kChunks; ++u) {
            const int64_t i = i0 + u * 256 + threadIdx.x;
            const float step = step8(s[u]);
            const u32x2 a = dequant8x4(v[u][0], step), b = dequant8x4(v[u][1], step);
            const u32x4 o = {a[0], a[1], b[0], b[1]};
            if (i < n) {
                if (NT) __builtin_nontemporal_store(o, x + i);
                else x[i] = o;
            }
        }
    }
}

// A wave takes block g (its index in the workgroup) of a 128-long contraction
// tile for 128 columns, two columns per lane: 32 reads of whole 256-byte row
// pieces, then each lane holds two whole blocks.  The four waves write the
// four quarters of 8 tiles of 1 KiB.  The bf16 side, which a model's loading
// touches once, is non-temporal: 32 x 7168 x 2048 weights pack in 210 us (5.7
// TB/s; 232 without) and unpack in 168 (232).
__global__ __launch_bounds__(256) void pack4_kernel(const uint16_t* __restrict__ w, int Kd, int N, int KT,
                                                    u32x4* __restrict__ q4, uint8_t* __restrict__ s4) {
    const int lane = threadIdx.x & 63, g = threadIdx.x >> 6;
    const int n = blockIdx.x * 128 + 2 * lane, kt = blockIdx.y;
    const int64_t e = blockIdx.z;
    if (n >= N) return;
    const int k0 = kt * 128 + g * 32;
    uint32_t v[32], m = 0, s2 = 0x0202;
    u32x4 o[2] = {u32x4{0u, 0u, 0u, 0u}, u32x4{0u, 0u, 0u, 0u}};
    if (k0 < Kd) {
        const uint32_t* src = (const uint32_t*)(w + (e * Kd + k0) * (int64_t)N + n);
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = __builtin_nontemporal_load(src + (int64_t)k * (N >> 1));
#pragma unroll
        for (int k = 0; k < 32; ++k) m = max_mag2(m, v[k] & 0x7fff7fffu);
        uint32_t s[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t b = (c ? m >> 16 : m & 0xffffu) >> 7;  // biased exponent
            s[c] = b == 255u ? 255u : max(b, 4u) - 2u;
            const float f = __uint_as_float(s[c] << 23);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                uint32_t d = 0;
#define MOE_FP4(I)                                                                                                   \
    d = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(                                                                   \
        d, __builtin_bit_cast(bf16x2, __builtin_amdgcn_perm(v[8 * t + 2 * I + 1], v[8 * t + 2 * I],                  \
                                                            c ? 0x07060302u : 0x05040100u)),                         \
        f, I)
                MOE_FP4(0);
                MOE_FP4(1);
                MOE_FP4(2);
                MOE_FP4(3);
#undef MOE_FP4
                o[c][t] = s[c] == 255u ? 0u : d;
            }
        }
        s2 = s[0] | (s[1] << 8);
    }
    const int64_t tile = (e * (N >> 4) + (n >> 4)) * KT + kt;
    const int slot = 16 * g + (n & 15);
    q4[tile * 64 + slot] = o[0];
    q4[tile * 64 + slot + 1] = o[1];
    *(uint16_t*)(s4 + tile * 64 + slot) = (uint16_t)s2;
}

__global__ __launch_bounds__(256) void unpack4_kernel(const u32x4* __restrict__ q4, const uint8_t* __restrict__ s4,
                                                      int Kd, int N, int KT, uint16_t* __restrict__ w) {
    const int lane = threadIdx.x & 63, g = threadIdx.x >> 6;
    const int n = blockIdx.x * 128 + 2 * lane, kt = blockIdx.y;
    const int64_t e = blockIdx.z;
    const int k0 = kt * 128 + g * 32;
    if (n >= N || k0 >= Kd) return;
    const int64_t tile = (e * (N >> 4) + (n >> 4)) * KT + kt;
    const int slot = 16 * g + (n & 15);
    const u32x4 a = q4[tile * 64 + slot], b = q4[tile * 64 + slot + 1];
    const uint32_t s2 = *(const uint16_t*)(s4 + tile * 64 + slot);
    const float fa = __uint_as_float((s2 & 0xffu) << 23), fb = __uint_as_float((s2 >> 8) << 23);
    uint32_t* dst = (uint32_t*)(w + (e * Kd + k0) * (int64_t)N + n);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#define MOE_FP4(I)                                                                                                   \
    {                                                                                                                \
        const uint32_t pa = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(a[t], fa, I));    \
        const uint32_t pb = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(b[t], fb, I));    \
        __builtin_nontemporal_store(__builtin_amdgcn_perm(pb, pa, 0x05040100u),                                      \
                                    dst + (int64_t)(8 * t + 2 * I) * (N >> 1));                                      \
        __builtin_nontemporal_store(__builtin_amdgcn_perm(pb, pa, 0x07060302u),                                      \
                                    dst + (int64_t)(8 * t + 2 * I + 1) * (N >> 1));                                  \
    }
        MOE_FP4(0)
        MOE_FP4(1)
        MOE_FP4(2)
        MOE_FP4(3)
#undef MOE_FP4
    }
}

// A workgroup for every 512 chunks, as far as a launch may have threads (below 2^32: 2^36 values, which the
// loop then takes in several steps).
static int grid8(int64_t chunks) {
    return (int)std::min<int64_t>((chunks + 256 * kChunks - 1) / (256 * kChunks), (1 << 24) - 1);
}

static bool streams8(int64_t rows, int cols) { return rows * cols * 2 >= (64ll << 20); }

static int check8(int64_t rows, int cols, const int32_t* offsets, int e_local) {
    if (rows < 0 || cols < 0 || rows >= (1ll << 31)) return MOE_EINVAL;
    if (offsets && (e_local < 0 || e_local > 512)) return MOE_EINVAL;
    if (cols % 64) return MOE_ESHAPE;
    return MOE_OK;
}

static int check4(int E, int Kd, int N) {
    if (E < 0 || E > 512 || Kd < 0 || N < 0) return MOE_EINVAL;
    if (Kd % 64 || N % 64) return MOE_ESHAPE;
    if ((int64_t)Kd * N * 2 >= (1ll << 31) || Kd > 65535 * 128) return MOE_EINVAL;
    return MOE_OK;
}

}  // namespace moe

using moe_host::misaligned;

extern "C" int moe_pack8(const moe_bf16* x, int64_t rows, int cols, const int32_t* offsets, int e_local, int8_t* q,
                         uint8_t* scale, moe_stream stream) {
    using namespace moe;
    const int rc = check8(rows, cols, offsets, e_local);
    if (rc != MOE_OK) return rc;
    if (rows == 0 || cols == 0) return MOE_OK;
    if (!x || !q || !scale) return MOE_EINVAL;
    if (misaligned(x) || misaligned(q) || misaligned(scale) || misaligned(offsets)) return MOE_EALIGN;
    const auto kernel = streams8(rows, cols) ? pack8_kernel<true> : pack8_kernel<false>;
    kernel<<<grid8(rows * (cols / 8)), 256, 0, (hipStream_t)stream>>>((const u32x4*)x, rows, cols / 8, offsets, e_local,
                                                                      (u32x2*)q, scale);
    return moe_host::launch_status();
}

extern "C" int moe_unpack8(const int8_t* q, const uint8_t* scale, int64_t rows, int cols, const int32_t* offsets,
                           int e_local, moe_bf16* x, moe_stream stream) {
    using namespace moe;
    const int rc = check8(rows, cols, offsets, e_local);
    if (rc != MOE_OK) return rc;
    if (rows == 0 || cols == 0) return MOE_OK;
    if (!x || !q || !scale) return MOE_EINVAL;
    if (misaligned(x) || misaligned(q) || misaligned(scale) || misaligned(offsets)) return MOE_EALIGN;
    const auto kernel = streams8(rows, cols) ? unpack8_kernel<true> : unpack8_kernel<false>;
    kernel<<<grid8(rows * (cols / 8)), 256, 0, (hipStream_t)stream>>>((const u32x2*)q, scale, rows, cols / 8, offsets,
                                                                      e_local, (u32x4*)x);
    return moe_host::launch_status();
}

extern "C" int moe_pack4(const moe_bf16* w, int E, int Kd, int N, uint8_t* q4, uint8_t* s4, moe_stream stream) {
    using namespace moe;
    const int rc = check4(E, Kd, N);
    if (rc != MOE_OK) return rc;
    if (E == 0 || Kd == 0 || N == 0) return MOE_OK;
    if (!w || !q4 || !s4) return MOE_EINVAL;
    if (misaligned(w) || misaligned(q4) || misaligned(s4)) return MOE_EALIGN;
    const int KT = (Kd + 127) / 128;
    pack4_kernel<<<dim3((N + 127) / 128, KT, E), 256, 0, (hipStream_t)stream>>>(w, Kd, N, KT, (u32x4*)q4, s4);
    return moe_host::launch_status();
}

extern "C" int moe_unpack4(const uint8_t* q4, const uint8_t* s4, int E, int Kd, int N, moe_bf16* w,
                           moe_stream stream) {
    using namespace moe;
    const int rc = check4(E, Kd, N);
    if (rc != MOE_OK) return rc;
    if (E == 0 || Kd == 0 || N == 0) return MOE_OK;
    if (!w || !q4 || !s4) return MOE_EINVAL;
    if (misaligned(w) || misaligned(q4) || misaligned(s4)) return MOE_EALIGN;
    const int KT = (Kd + 127) / 128;
    unpack4_kernel<<<dim3((N + 127) / 128, KT, E), 256, 0, (hipStream_t)stream>>>((const u32x4*)q4, s4, Kd, N, KT, w);
    return moe_host::launch_status();
}
