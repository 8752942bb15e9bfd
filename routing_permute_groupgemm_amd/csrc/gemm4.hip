// Grouped products of few rows per expert with weights in 4-bit blocks (the
// serving form of the gate/up and down GroupGEMMs).
//
//   gate/up: h[r] = bf16(silu(x_r . Wg_j) * (x_r . Wu_j)),  down: c[r] = bf16(a_r . W_j)
// for the rows r of expert j, W the bf16 values of the packed weights (mx.hpp)
// and fp32 sums.  A token meets a handful of experts, so almost every byte
// moved is a weight, read once: the time is that of streaming 17/32 byte a
// weight, and the kernel's work is to keep enough of those bytes in flight.
//
// Packed tiles hold 16 output columns x 128 contraction values in 1 KiB, in
// the order of the matrix instruction's first operand: lane l of a wave owns
// the block of 32 contraction values 32*(l/16) .. +31 of column l%16, one
// 16-byte load, one scale byte and 16 conversions (each exact: a 4-bit value
// times a power of two is a bf16) for four v_mfma_f32_16x16x32_bf16.  The
// rows are the second operand: lane l holds the same 32 contraction values of
// row l%16, 64 contiguous bytes.  The four steps of a tile take 8 values from
// every lane group, so the contraction order inside a tile is a fixed
// permutation of the natural one.
//
// A workgroup computes 16*MT rows x 16*NT columns (of both matrices for
// gate/up); its W waves take the contraction tiles in turn and their fp32
// sums meet in LDS, added in wave order.  No LDS is used on the way in: a
// weight byte has one reader, and the rows are read once per workgroup.
#include "mx.hpp"

namespace moe {

struct Gemm4Params {
    const uint16_t* a;   // rows in expert order, or the tokens with src
    const int32_t* src;  // row r is a[src[r] / topk]; NULL: row r is a[r]
    int topk;
    uint32_t topk_rcp;   // floor((2^32 - 1) / topk)
    int64_t a_rows;
    const uint8_t* q[2];
    const uint8_t* s[2];
    const int32_t* offsets;
    int e_local;
    int64_t cap;
    int Kd, N, KT;
    uint16_t* c;         // [cap, N]
};

// Per-lane byte offset that is outside every resource (those of tokens may
// reach 3.75 GiB), also with any column offset of a row added.
constexpr uint32_t kNoRow = kOOB_GATHER;

template <int MATS, int MT, int NT, int W>
__global__ __launch_bounds__(64 * W) void gemm4_kernel(Gemm4Params p) {
    constexpr int ACC = MATS * NT * MT;
    __shared__ f32x4 part[W][ACC][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // ---- this workgroup's tile, from the device-resident row counts ----
    // Lane l counts the row tiles of experts l*per .. l*per+per-1.
    constexpr int BM = 16 * MT;
    const int per = (p.e_local + 63) >> 6;
    int mine = 0;
    for (int i = 0; i < per; ++i) {
        const int j = lane * per + i;
        if (j < p.e_local) {
            const int64_t lo = min((int64_t)p.offsets[j], p.cap), hi = min((int64_t)p.offsets[j + 1], p.cap);
            mine += (int)((hi - lo + BM - 1) / BM);
        }
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int t = __shfl_up(incl, o, 64);
        if (lane >= o) incl += t;
    }
    const int tiles = __builtin_amdgcn_readlane(incl, 63);
    const int slabs = (p.N / 16 + NT - 1) / NT;
    // workgroup b runs on XCD b % 8: each XCD takes a contiguous run, in which
    // an expert's row tiles of one slab (the same weights) are neighbours
    const int run = (tiles * slabs + 7) >> 3;
    const int at = (int)(blockIdx.x >> 3);
    const int id = (int)(blockIdx.x & 7) * run + at;
    if (at >= run || id >= tiles * slabs) return;
    const int slab = id / tiles;
    int rest = id - slab * tiles;
    const uint64_t has = __ballot(incl > rest);  // the first lane with more tiles up to it
    const int owner = __builtin_ctzll(has);
    rest -= __builtin_amdgcn_readlane(incl - mine, owner);
    int j = owner * per, row0 = 0, rows = 0;
    for (int i = 0; i < per; ++i) {
        const int jj = owner * per + i;
        const int64_t lo = min((int64_t)p.offsets[jj], p.cap), hi = min((int64_t)p.offsets[jj + 1], p.cap);
        const int n = (int)((hi - lo + BM - 1) / BM);
        if (rest < n) {
            j = jj;
            row0 = (int)lo + rest * BM;
            rows = min(BM, (int)(hi - row0));
            break;
        }
        rest -= n;
    }
    j = __builtin_amdgcn_readfirstlane(j);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    rows = __builtin_amdgcn_readfirstlane(rows);

    // ---- the rows: a byte offset per lane and 16-row block ----
    const int r16 = lane & 15, g = lane >> 4;
    const uint32_t ld = (uint32_t)p.Kd * 2u;
    const bool gather = p.src != nullptr;
    const uint16_t* base = gather ? p.a : p.a + (int64_t)row0 * p.Kd;
    const auto rs = make_rsrc(base, gather ? (uint32_t)(p.a_rows * p.Kd * 2) : (uint32_t)rows * ld);
    uint32_t off[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int r = 16 * m + r16;
        off[m] = kNoRow;
        if (r < rows) {
            uint32_t tok = (uint32_t)r;
            if (gather) {
                const uint32_t v = (uint32_t)p.src[row0 + r];
                tok = __umulhi(v, p.topk_rcp);  // the quotient, or one less
                if (v - tok * (uint32_t)p.topk >= (uint32_t)p.topk) ++tok;
            }
            if (!gather || tok < (uint64_t)p.a_rows) off[m] = tok * ld + 64u * g;
        }
    }

    // ---- contraction ----
    const int nt0 = slab * NT;
    const int64_t tile0 = ((int64_t)j * (p.N >> 4) + nt0) * p.KT;
    struct Stage {
        u32x4 w[MATS][NT];
        uint32_t s[MATS][NT];
        u32x4 x[MT][4];
    };
    auto load = [&](Stage& t, int kt) {
#pragma unroll
        for (int q = 0; q < MATS; ++q)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const bool in = NT == 1 || nt0 + i < (p.N >> 4);
                const int64_t tile = tile0 + (in ? (int64_t)i * p.KT : 0) + kt;
                t.w[q][i] = *(const u32x4*)(p.q[q] + tile * 1024 + lane * 16);
                t.s[q][i] = p.s[q][tile * 64 + lane];
            }
        // the last tile may end after two blocks: the others' values are 0
        const bool in = kt * 128 + 32 * g < p.Kd;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int st = 0; st < 4; ++st)
                t.x[m][st] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                               rs, (in ? off[m] : kNoRow) + (uint32_t)(kt * 256 + st * 16), 0, 0));
    };
    f32x4 acc[MATS][NT][MT];
#pragma unroll
    for (int q = 0; q < MATS; ++q)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[q][i][m] = f32x4{};
    auto multiply = [&](const Stage& t) {
#pragma unroll
        for (int q = 0; q < MATS; ++q)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const float f = __uint_as_float(t.s[q][i] << 23);
#pragma unroll
                for (int st = 0; st < 4; ++st) {
                    const uint32_t d = t.w[q][i][st];
                    const u32x4 v = {
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, f, 0)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, f, 1)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, f, 2)),
                        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, f, 3))};
                    const bf16x8 wv = __builtin_bit_cast(bf16x8, v);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        acc[q][i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            wv, __builtin_bit_cast(bf16x8, t.x[m][st]), acc[q][i][m], 0, 0, 0);
                }
            }
    };
    Stage s0, s1;
    int kt = wave;
    if (kt < p.KT) load(s0, kt);
    for (; kt < p.KT; kt += 2 * W) {
        if (kt + W < p.KT) load(s1, kt + W);
        multiply(s0);
        if (kt + W >= p.KT) break;
        if (kt + 2 * W < p.KT) load(s0, kt + 2 * W);
        multiply(s1);
    }

    // ---- the waves' sums, in wave order ----
#pragma unroll
    for (int q = 0; q < MATS; ++q)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int m = 0; m < MT; ++m) part[wave][(q * NT + i) * MT + m][lane] = acc[q][i][m];
    __syncthreads();
    for (int t = wave; t < NT * MT; t += W) {
        f32x4 v = part[0][t][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) v += part[w][t][lane];
        if (MATS == 2) {
            f32x4 u = part[0][ACC / 2 + t][lane];
#pragma unroll
            for (int w = 1; w < W; ++w) u += part[w][ACC / 2 + t][lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = v[i] * __builtin_amdgcn_rcpf(1.0f + __expf(-v[i])) * u[i];
        }
        // lane: row l%16, columns 4*(l/16) .. +3 of the 16 x 16 block
        const int r = 16 * (t % MT) + r16;
        const int n = 16 * (nt0 + t / MT) + 4 * g;
        if (r < rows && n < p.N)
            *(u32x2*)(p.c + (int64_t)(row0 + r) * p.N + n) = u32x2{pack_bf2x(v[0], v[1]), pack_bf2x(v[2], v[3])};
    }
}

template <int MATS, int MT, int NT, int W>
static int launch4(const Gemm4Params& p, hipStream_t s) {
    const int64_t bm = 16 * MT;
    const int64_t tiles = std::min<int64_t>(p.cap, p.cap / bm + p.e_local);
    const int64_t slabs = (p.N / 16 + NT - 1) / NT;
    const int64_t grid = (tiles * slabs + 7) / 8 * 8;
    if (grid >= (1ll << 31)) return MOE_EINVAL;
    gemm4_kernel<MATS, MT, NT, W><<<(unsigned)grid, 64 * W, 0, s>>>(p);
    return moe_host::launch_status();
}

template <int MATS>
static int launch4_rows(const Gemm4Params& p, hipStream_t s) {
    const int64_t avg = (p.cap + p.e_local - 1) / p.e_local;
    if (avg <= 16) return launch4<MATS, 1, 2, 8>(p, s);
    if (avg <= 32) return launch4<MATS, 2, 2, 4>(p, s);
    return launch4<MATS, 4, 2, 4>(p, s);
}

// Checks common to both products; MOE_OK with *nothing set: no work.
static int check_gemm4(int e_local, int Kd, int N, int cap_rows, const int32_t* offsets, bool* nothing) {
    *nothing = false;
    if (e_local < 0 || e_local > 512 || Kd <= 0 || N < 0 || cap_rows < 0) return MOE_EINVAL;
    if (Kd % 64 || N % 64) return MOE_ESHAPE;
    // the byte offset of a row's end, added to the out-of-range offset, stays below 2^32
    if (Kd > (1 << 26) || (int64_t)Kd * N * 2 >= (1ll << 31)) return MOE_EINVAL;
    if (!offsets) return MOE_EINVAL;
    *nothing = e_local == 0 || cap_rows == 0 || N == 0;
    return MOE_OK;
}

}  // namespace moe

using moe_host::misaligned;

extern "C" int moe_grouped_gemm4_swiglu(const moe_bf16* x, int T, const int32_t* src, int K, const uint8_t* gate_q4,
                                        const uint8_t* gate_s4, const uint8_t* up_q4, const uint8_t* up_s4,
                                        const int32_t* offsets, int e_local, int H, int F, int cap_rows, moe_bf16* h,
                                        moe_stream stream) {
    using namespace moe;
    bool nothing;
    const int rc = check_gemm4(e_local, H, F, cap_rows, offsets, &nothing);
    if (rc != MOE_OK) return rc;
    if (src) {
        if (T < 0 || K < 1 || K > 16 || (int64_t)T * K >= (1ll << 31) || cap_rows > (int64_t)T * K) return MOE_EINVAL;
        if ((int64_t)T * H * 2 > (int64_t)kOOB_GATHER) return MOE_EINVAL;
    }
    if (nothing) return MOE_OK;
    if (!x || !gate_q4 || !gate_s4 || !up_q4 || !up_s4 || !h) return MOE_EINVAL;
    if (misaligned(x) || misaligned(src) || misaligned(gate_q4) || misaligned(gate_s4) || misaligned(up_q4) ||
        misaligned(up_s4) || misaligned(offsets) || misaligned(h))
        return MOE_EALIGN;
    Gemm4Params p{};
    p.a = x;
    p.src = src;
    p.topk = src ? K : 1;
    p.topk_rcp = 0xffffffffu / (uint32_t)p.topk;
    p.a_rows = T;
    p.q[0] = gate_q4;
    p.q[1] = up_q4;
    p.s[0] = gate_s4;
    p.s[1] = up_s4;
    p.offsets = offsets;
    p.e_local = e_local;
    p.cap = cap_rows;
    p.Kd = H;
    p.N = F;
    p.KT = (H + 127) / 128;
    p.c = h;
    return launch4_rows<2>(p, (hipStream_t)stream);
}

extern "C" int moe_grouped_gemm4(const moe_bf16* a, const uint8_t* q4, const uint8_t* s4, const int32_t* offsets,
                                 int e_local, int Kd, int N, int cap_rows, moe_bf16* c, moe_stream stream) {
    using namespace moe;
    bool nothing;
    const int rc = check_gemm4(e_local, Kd, N, cap_rows, offsets, &nothing);
    if (rc != MOE_OK) return rc;
    if (nothing) return MOE_OK;
    if (!a || !q4 || !s4 || !c) return MOE_EINVAL;
    if (misaligned(a) || misaligned(q4) || misaligned(s4) || misaligned(offsets) || misaligned(c)) return MOE_EALIGN;
    Gemm4Params p{};
    p.a = a;
    p.topk = 1;
    p.topk_rcp = 0xffffffffu;
    p.a_rows = cap_rows;
    p.q[0] = q4;
    p.s[0] = s4;
    p.offsets = offsets;
    p.e_local = e_local;
    p.cap = cap_rows;
    p.Kd = Kd;
    p.N = N;
    p.KT = (Kd + 127) / 128;
    p.c = c;
    return launch4_rows<1>(p, (hipStream_t)stream);
}
