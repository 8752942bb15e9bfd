// Grouped products of few rows per expert with weights in 4-bit blocks (the
// serving form of the gate/up and down GroupGEMMs).
//
//   gate/up: h[r] = bf16(silu(x_r . Wg_j) * (x_r . Wu_j)),  down: c[r] = bf16(a_r . W_j)
// for the rows r of expert j, W the bf16 values of the packed weights (mx.hpp)
// and fp32 sums.  A token meets a handful of experts, so almost every byte
// moved is a weight, read once: the time is that of streaming 17/32 byte a
// weight, and the kernels' work is to keep enough of those bytes in flight.
//
// Packed tiles hold 16 output columns x 128 contraction values in 1 KiB, in
// the order of the matrix instruction's first operand: lane l of a wave owns
// the block of 32 contraction values 32*(l/16) .. +31 of column l%16, one
// 16-byte load, one scale byte and 16 conversions (each exact: a 4-bit value
// times a power of two is a bf16) for four v_mfma_f32_16x16x32_bf16.  The
// rows are the second operand: lane l needs the same 32 contraction values of
// row l%16.  The four steps of a tile take 8 values from every lane group, so
// the contraction order inside a tile is a fixed permutation of the natural
// one.
//
// Two kernels share this:
//   gemm4_split: the waves of a workgroup take the contraction tiles of the
//     same 16 rows x 16*NT columns in turn; their fp32 sums meet in LDS, added
//     in wave order.  For a few tokens, whose tiles are too few to give every SIMD
//     a wave of its own columns.
//   gemm4_wide: every wave has its own 16*NT columns and runs the whole
//     contraction; the rows, which the waves share, go through LDS.  Nothing is
//     reduced across waves, and a row byte is read once per workgroup.
// The rule between them is in launch4_rows.
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
    uint16_t* c;         // bf16 [cap, N], or NULL
    float* c32;          // fp32 [cap, N], or NULL
    bool stream;         // weights that one row tile reads carry the non-temporal hint (launch4_rows)
};

// Per-lane byte offset that is outside every resource (those of tokens may
// reach 3.75 GiB), also with any column offset of a row added.
constexpr uint32_t kNoRow = kOOB_GATHER;

// The tile of this workgroup, the same in every lane (j = -1: none), and the number
// of row tiles of its expert (`tiles`).  Lane l holds the row tiles of experts
// l*PER .. l*PER+PER-1.  Workgroup b runs on XCD b % 8, and each XCD takes a
// contiguous run of the order:
//   BY_EXPERT  an expert's slabs (blocks of columns) one after another, the row
//              tiles of a slab next to each other: they read the same weights, and
//              the slabs the same rows, through one L2 (256 tokens: down 51 against 52
//              us, gate/up 80 against 82);
//   otherwise  the row tiles of all experts, slab by slab: with one or two rows an
//              expert there is nothing to share, and a run over all experts was
//              faster (one token: gate/up 12.0 against 12.8 us).
template <int PER, int BM, bool BY_EXPERT>
__device__ __forceinline__ void find_tile(const Gemm4Params& p, int lane, int slabs, int& j, int& row0, int& rows,
                                          int& slab, int& tiles) {
    int at[PER + 1];
#pragma unroll
    for (int i = 0; i <= PER; ++i) at[i] = p.offsets[min(lane * PER + i, p.e_local)];
    int n[PER], mine = 0;
#pragma unroll
    for (int i = 0; i <= PER; ++i) at[i] = (int)min((int64_t)at[i], p.cap);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        n[i] = (at[i + 1] - at[i] + BM - 1) / BM;
        mine += n[i];
    }
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int t = __shfl_up(incl, o, 64);
        if (lane >= o) incl += t;
    }
    const int total = __builtin_amdgcn_readlane(incl, 63);
    const int run = (total * slabs + 7) >> 3;
    const int b = (int)(blockIdx.x >> 3);
    int id = (int)(blockIdx.x & 7) * run + b;
    if (b >= run || id >= total * slabs) return;
    const int per = BY_EXPERT ? slabs : 1;  // places of a row tile in the order searched here
    if (!BY_EXPERT) {
        slab = id / total;
        id -= slab * total;
    }
    const int owner = __builtin_ctzll(__ballot(incl * per > id));  // the first lane with more places up to it
    int rest = id - (incl - mine) * per, expert = 0, place = 0, count = 1, first = 0, end = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (rest >= 0 && rest < n[i] * per) {
            expert = lane * PER + i;
            place = rest;
            count = n[i];
            first = at[i];
            end = at[i + 1];
        }
        rest -= n[i] * per;
    }
    j = __builtin_amdgcn_readlane(expert, owner);
    place = __builtin_amdgcn_readlane(place, owner);
    tiles = __builtin_amdgcn_readlane(count, owner);
    if (BY_EXPERT) {
        slab = place;
        place = 0;
        if (tiles > 1) {
            place = slab % tiles;
            slab /= tiles;
        }
    }
    row0 = __builtin_amdgcn_readlane(first, owner) + place * BM;
    rows = min(BM, __builtin_amdgcn_readlane(end, owner) - row0);
}

template <int BM, bool BY_EXPERT>
__device__ __forceinline__ void find_tile_of(const Gemm4Params& p, int lane, int slabs, int& j, int& row0, int& rows,
                                             int& slab, int& tiles) {
    j = -1;
    if (p.e_local <= 64) find_tile<1, BM, BY_EXPERT>(p, lane, slabs, j, row0, rows, slab, tiles);
    else if (p.e_local <= 128) find_tile<2, BM, BY_EXPERT>(p, lane, slabs, j, row0, rows, slab, tiles);
    else if (p.e_local <= 256) find_tile<4, BM, BY_EXPERT>(p, lane, slabs, j, row0, rows, slab, tiles);
    else find_tile<8, BM, BY_EXPERT>(p, lane, slabs, j, row0, rows, slab, tiles);
}

// 4 x 4 transpose between register index and lane group of 16 (16 bytes each):
// v[t] of group g becomes what v[g] of group t was.
__device__ __forceinline__ void transpose4(u32x4 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const auto a = __builtin_amdgcn_permlane32_swap(v[0][i], v[2][i], false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(v[1][i], v[3][i], false, false);
        const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
        const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
        v[0][i] = c[0];
        v[1][i] = c[1];
        v[2][i] = d[0];
        v[3][i] = d[1];
    }
}

// The resource that a tile's rows are read through (rows past it read 0), and
// the byte offset in it of the tile's row r.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const Gemm4Params& p, int row0, int rows) {
    if (p.src) return make_rsrc(p.a, (uint32_t)(p.a_rows * p.Kd * 2));
    return make_rsrc(p.a + (int64_t)row0 * p.Kd, (uint32_t)rows * ((uint32_t)p.Kd * 2u));
}
__device__ __forceinline__ uint32_t row_offset(const Gemm4Params& p, int row0, int rows, int r) {
    if (r >= rows) return kNoRow;
    uint32_t tok = (uint32_t)r;
    if (p.src) {
        const uint32_t v = (uint32_t)p.src[row0 + r];
        tok = __umulhi(v, p.topk_rcp);  // the quotient, or one less
        if (v - tok * (uint32_t)p.topk >= (uint32_t)p.topk) ++tok;
        if (tok >= (uint64_t)p.a_rows) return kNoRow;
    }
    return tok * ((uint32_t)p.Kd * 2u);
}

// First packed tile of each of the NT column tiles from nt0 of expert j (column
// tiles past the last are taken as the last; their results are not stored).
template <int NT>
__device__ __forceinline__ void column_tiles(const Gemm4Params& p, int j, int nt0, int64_t (&at)[NT]) {
    const int n = p.N >> 4;
#pragma unroll
    for (int i = 0; i < NT; ++i) at[i] = ((int64_t)j * n + min(nt0 + i, n - 1)) * p.KT;
}

// Eight codes times their block's scale, as bf16.
__device__ __forceinline__ bf16x8 fp4_step(uint32_t d, float f) {
    const u32x4 v = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, f, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, f, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, f, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, f, 3))};
    return __builtin_bit_cast(bf16x8, v);
}

// One contraction tile of a wave's weights: NT column tiles of each matrix.
template <int MATS, int NT>
struct Weights4 {
    u32x4 w[MATS][NT];
    uint32_t s[MATS][NT];
    template <bool NTL>
    __device__ __forceinline__ void load(const Gemm4Params& p, const int64_t (&at)[NT], int kt, int lane) {
#pragma unroll
        for (int q = 0; q < MATS; ++q)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int64_t tile = at[i] + kt;
                const u32x4* src = (const u32x4*)(p.q[q] + tile * 1024) + lane;
                w[q][i] = NTL ? __builtin_nontemporal_load(src) : *src;
                s[q][i] = p.s[q][tile * 64 + lane];
            }
    }
    // Step st (8 of each lane's 32 contraction values) as bf16.
    __device__ __forceinline__ bf16x8 step(int q, int i, int st) const {
        return fp4_step(w[q][i][st], __uint_as_float(s[q][i] << 23));
    }
};

// Columns n .. n+3 of row r, from the sums v (and u for gate/up).
template <int MATS>
__device__ __forceinline__ void store4(const Gemm4Params& p, int64_t r, int n, f32x4 v, f32x4 u) {
    if (MATS == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = silu_f(v[i]) * u[i];
    }
    if (p.c) *(u32x2*)(p.c + r * p.N + n) = u32x2{pack_bf2x(v[0], v[1]), pack_bf2x(v[2], v[3])};
    if (MATS == 1 && p.c32) *(f32x4*)(p.c32 + r * p.N + n) = v;
}

// 16 rows x 16*NT columns of a workgroup, the contraction tiles over its W waves.
// Measured for one token (H = 4096, F = 1536, 8 experts): gate/up 11.7 us for
// 53 MB of weights, down 7.4 us for 27 MB.
template <int MATS, int NT, int W>
__global__ __launch_bounds__(64 * W) void gemm4_split(Gemm4Params p) {
    constexpr int ACC = MATS * NT;
    __shared__ f32x4 part[W][ACC][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slabs = (p.N / 16 + NT - 1) / NT;
    int j, row0, rows, slab, shared;
    find_tile_of<16, false>(p, lane, slabs, j, row0, rows, slab, shared);
    if (j < 0) return;
    const int nt0 = slab * NT, r16 = lane & 15, g = lane >> 4;

    int64_t tiles[NT];
    column_tiles(p, j, nt0, tiles);
    struct Stage {
        Weights4<MATS, NT> w;
        u32x4 x[4];
    } s0, s1;
    int kt = wave;
    // the first weights do not wait for the rows' indices
    if (kt < p.KT) s0.w.template load<false>(p, tiles, kt, lane);
    const auto rs = rows_rsrc(p, row0, rows);
    uint32_t off = row_offset(p, row0, rows, r16);
    if (off != kNoRow) off += 16u * g;
    // load i: block i of the tile, 64 contiguous bytes of a row over the 4 lane
    // groups (0 behind the contraction's end)
    auto load_x = [&](Stage& t, int k) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            t.x[i] = __builtin_bit_cast(
                u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                           rs, (k * 128 + 32 * i < p.Kd ? off : kNoRow) + (uint32_t)(k * 256 + i * 64), 0, 0));
    };
    auto load = [&](Stage& t, int k) {
        t.w.template load<false>(p, tiles, k, lane);
        load_x(t, k);
    };
    f32x4 acc[MATS][NT];
#pragma unroll
    for (int q = 0; q < MATS; ++q)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[q][i] = f32x4{};
    auto multiply = [&](Stage& t) {
        transpose4(t.x);
#pragma unroll
        for (int q = 0; q < MATS; ++q)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int st = 0; st < 4; ++st)
                    acc[q][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        t.w.step(q, i, st), __builtin_bit_cast(bf16x8, t.x[st]), acc[q][i], 0, 0, 0);
    };
    if (kt < p.KT) load_x(s0, kt);
    for (; kt < p.KT; kt += 2 * W) {
        if (kt + W < p.KT) load(s1, kt + W);
        multiply(s0);
        if (kt + W >= p.KT) break;
        if (kt + 2 * W < p.KT) load(s0, kt + 2 * W);
        multiply(s1);
    }

    // the waves' sums, in wave order
#pragma unroll
    for (int q = 0; q < MATS; ++q)
#pragma unroll
        for (int i = 0; i < NT; ++i) part[wave][q * NT + i][lane] = acc[q][i];
    __syncthreads();
    for (int t = wave; t < NT; t += W) {
        f32x4 v[MATS];
#pragma unroll
        for (int q = 0; q < MATS; ++q) {
            v[q] = part[0][q * NT + t][lane];
#pragma unroll
            for (int w = 1; w < W; ++w) v[q] += part[w][q * NT + t][lane];
        }
        // lane: row l%16, columns 4*(l/16) .. +3 of the 16 x 16 block
        const int n = 16 * (nt0 + t) + 4 * g;
        if (r16 < rows && n < p.N) store4<MATS>(p, (int64_t)row0 + r16, n, v[0], v[MATS - 1]);
    }
}

// 16*MT rows x 16*NT*W columns of a workgroup of W waves.  A contraction tile of
// the rows is [16*MT][128] bf16 in LDS, 256-byte rows with their 16-byte chunks
// XOR-swizzled by row; two such buffers and one barrier a tile (a wave that
// writes buffer b for tile k+2 has passed the barrier of tile k+1, which every
// wave reaches after its reads of tile k).  Rows and weights of the next
// tile are in flight while one is multiplied; deeper prefetch of the weights
// (3 and 4 tiles) cost registers, and with them waves, and ran slower.  Row blocks
// past the tile's rows are neither read nor multiplied.
// NTL: the weights carry the non-temporal hint.
template <int MATS, int MT, int NT, int W, bool NTL>
__device__ __forceinline__ void wide_tile(const Gemm4Params& p, uint8_t (*xs)[MT * 4096], int j, int row0, int rows,
                                          int slab) {
    // a thread's 16-byte loads of the rows per tile, and the rows that one of them covers
    constexpr int XL = MT * 4 / W, XR = 4 * W;
    static_assert(XL * W == MT * 4, "the rows' loads split evenly over the threads");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nt0 = (slab * W + wave) * NT, r16 = lane & 15, g = lane >> 4;

    int64_t tiles[NT];
    column_tiles(p, j, nt0, tiles);
    Weights4<MATS, NT> wb[2];
    wb[0].template load<NTL>(p, tiles, 0, lane);  // does not wait for the rows' indices
    const auto rs = rows_rsrc(p, row0, rows);
    const int xrow = tid >> 4, xch = tid & 15;  // this thread's 16-byte chunk of rows xrow + XR*m
    uint32_t off[XL];
#pragma unroll
    for (int m = 0; m < XL; ++m) {
        off[m] = row_offset(p, row0, rows, XR * m + xrow);
        if (off[m] != kNoRow) off[m] += 16u * xch;
    }
    u32x4 xr[2][XL];
    auto load_x = [&](u32x4 (&x)[XL], int kt) {
        const bool in = kt * 128 + 8 * xch < p.Kd;  // 0 behind the contraction's end
#pragma unroll
        for (int m = 0; m < XL; ++m)
            x[m] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                 rs, (in ? off[m] : kNoRow) + (uint32_t)(kt * 256), 0, 0));
    };
    auto put_x = [&](const u32x4 (&x)[XL], int slot) {
#pragma unroll
        for (int m = 0; m < XL; ++m)
            *(MOE_LDS u32x4*)(xs[slot] + (XR * m + xrow) * 256 + ((xch ^ (xrow & 15)) << 4)) = x[m];
    };
    f32x4 acc[MATS][NT][MT];
#pragma unroll
    for (int q = 0; q < MATS; ++q)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[q][i][m] = f32x4{};
    auto multiply = [&](const Weights4<MATS, NT>& w, int slot) {
#pragma unroll
        for (int st = 0; st < 4; ++st) {
            bf16x8 xf[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m)
                if (m == 0 || 16 * m < rows)
                    xf[m] = __builtin_bit_cast(bf16x8, *(const MOE_LDS u32x4*)(xs[slot] + (16 * m + r16) * 256 +
                                                                               (((4 * g + st) ^ r16) << 4)));
#pragma unroll
            for (int q = 0; q < MATS; ++q)
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const bf16x8 wv = w.step(q, i, st);
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        if (m == 0 || 16 * m < rows)
                            acc[q][i][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, xf[m], acc[q][i][m], 0, 0, 0);
                }
        }
    };
    load_x(xr[0], 0);
    for (int k0 = 0; k0 < p.KT; k0 += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int kt = k0 + u;
            if (kt >= p.KT) break;
            put_x(xr[u], u);
            if (kt + 1 < p.KT) {
                load_x(xr[u ^ 1], kt + 1);
                wb[u ^ 1].template load<NTL>(p, tiles, kt + 1, lane);
            }
            __syncthreads();
            multiply(wb[u], u);
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int r = 16 * m + r16, n = 16 * (nt0 + i) + 4 * g;
            if (r < rows && n < p.N)
                store4<MATS>(p, (int64_t)row0 + r, n, acc[0][i][m], acc[MATS - 1][i][m]);
        }
}

template <int MATS, int MT, int NT, int W>
__global__ __launch_bounds__(64 * W) void gemm4_wide(Gemm4Params p) {
    __shared__ __attribute__((aligned(16))) uint8_t xs[2][MT * 4096];
    const int slabs = (p.N / 16 + NT * W - 1) / (NT * W);
    int j, row0, rows, slab, tiles;
    find_tile_of<16 * MT, true>(p, threadIdx.x & 63, slabs, j, row0, rows, slab, tiles);
    if (j < 0) return;
    // An expert's weights that no other workgroup reads go past the cache; those of several row tiles stay in the L2
    // that these share.  Gate/up of 256 tokens on 32 experts (one tile each) 77 against 90 us; of 512 tokens on 128
    // experts (one to three) 170 against 189 with the hint on all and 175 on none.
    if (p.stream && tiles == 1) wide_tile<MATS, MT, NT, W, true>(p, xs, j, row0, rows, slab);
    else wide_tile<MATS, MT, NT, W, false>(p, xs, j, row0, rows, slab);
}

// Whether a launch may have this many workgroups of W waves: its threads stay below 2^32 (and the tile numbers
// below 2^31).
static bool too_many(int64_t grid, int W) { return grid * (64 * W) >= (1ll << 32); }

template <int MATS, int NT, int W>
static int launch_split(const Gemm4Params& p, hipStream_t s) {
    const int64_t tiles = std::min<int64_t>(p.cap, p.cap / 16 + p.e_local);
    const int64_t grid = (tiles * ((p.N / 16 + NT - 1) / NT) + 7) / 8 * 8;
    if (too_many(grid, W)) return MOE_EINVAL;
    gemm4_split<MATS, NT, W><<<(unsigned)grid, 64 * W, 0, s>>>(p);
    return moe_host::launch_status();
}

template <int MATS, int MT, int NT, int W>
static int launch_wide(const Gemm4Params& p, hipStream_t s) {
    const int64_t tiles = std::min<int64_t>(p.cap, p.cap / (16 * MT) + p.e_local);
    const int64_t grid = (tiles * ((p.N / 16 + NT * W - 1) / (NT * W)) + 7) / 8 * 8;
    if (too_many(grid, W)) return MOE_EINVAL;
    gemm4_wide<MATS, MT, NT, W><<<(unsigned)grid, 64 * W, 0, s>>>(p);
    return moe_host::launch_status();
}

// Which kernel, from the host's sizes alone: cap rows over e_local experts make at
// most `tiles` row tiles of 16.
//   split: gate/up below 6.25 waves a SIMD if every wave took 16 columns, down below 3.75.
//     Where every tile has rows (128 experts, H = 4096, F = 1536, these in us against
//     wide) gate/up is even from 3 waves on: one token (0.75) 12.7 against 22.1, four (3)
//     34.0 against 32.5, eight (6) 58 against 57 (H = 2048, F = 768: eight (3) 17.9 against
//     15.9, twelve (4.5) 21.0 against 19.9); down with its combine of one token (2) 10.5 against
//     12.4, two (4) 14.8 against 14.1, four (8) 23 against 20 (of three at the smaller sizes (3) 10.1
//     against 9.7).  On a share of the experts, with room for every pair, most tiles are
//     empty and wide leaves most waves idle: 32 of 256, H = 7168, F = 2048, gate/up of four
//     tokens (4) 19 against 41, of sixteen (5) 34 against 47; down of one (3.5) 6.0 against
//     9.0, four (14) 14.7 against 17.
//     Two column tiles a workgroup once those make two workgroups a CU (gate/up of two
//     tokens 19.8 against 22.2 us, of one 13.3 against 12.7).
//   wide, rows: tiles of 16 up to two rows an expert, of 32 beyond.  128 experts, gate/up
//     and down: 23 tokens 30 + 16 us with 16 rows, 33 + 18 with 32; 96 tokens (6 rows)
//     133 + 74 against 128 + 73; 256 tokens (16) 165 + 97 against 147 + 83; 64 rows were
//     slower at 512 tokens (182 to 218 us for gate/up).
//   wide, columns of 32-row tiles: 256 a workgroup, which reads the rows half as often,
//     once that leaves 4 workgroups a CU, else 128.  512 tokens on 128 experts, H = 4096,
//     F = 1536, a skewed router: gate/up 170 against 183 us, down 106 against 118; 64 tokens
//     on 8 experts of 4096 columns (0.75): 52 against 44; 256 tokens on 128 experts of 768
//     columns (2.3): 45 against 42.
//   non-temporal weights (stream): when the packed matrices that the rows can touch
//     fill half the last-level cache (128 MB) or more, so that they are not there the
//     next time, for the experts whose rows fit one tile (gemm4_wide).
//
// What bounds them is the stream of weights.  512 tokens: gate/up fetches 0.92 GB (of
// 0.89 that it must) and down 0.45 (0.44) at about 5.2 TB/s, near what a plain copy
// reaches without the non-temporal hint (5.4); with the conversions or the matrix
// instructions left out they took as long.  256 tokens, non-temporal: 6.5 TB/s.
template <int MATS>
static int launch4_rows(Gemm4Params p, hipStream_t s) {
    const int64_t cols = p.N / 16;
    const int64_t tiles = std::min<int64_t>(p.cap, p.cap / 16 + p.e_local);
    const int64_t cus = moe_host::num_cus();
    if (tiles * cols < (MATS == 2 ? 25 : 15) * cus) {
        if (tiles * cols >= 2 * 2 * cus) return launch_split<MATS, 2, 4>(p, s);
        return launch_split<MATS, 1, 4>(p, s);
    }
    const int64_t experts = std::min<int64_t>(p.cap, p.e_local);
    p.stream = experts * MATS * p.N * p.Kd * 17 / 32 >= (128ll << 20);
    if (p.cap <= 2ll * p.e_local) return launch_wide<MATS, 1, 2 / MATS, 4>(p, s);
    const int64_t wide = std::min<int64_t>(p.cap, p.cap / 32 + p.e_local) * ((p.N + 255) / 256);
    if (wide >= 4 * cus) return launch_wide<MATS, 2, 2, 8>(p, s);
    return launch_wide<MATS, 2, 1, 8>(p, s);
}

// out[t] = bf16(sum over k ascending of gate[t,k] * y[pos[t,k]]) from fp32 rows: moe_combine without the rounding
// of y, which left out 2.9e-3 off where it is 2.4e-3 off now (the bf16 of h and of out remain).  4 columns per
// thread; a token's rows and gates are the same in every lane of a wave.  Bound by the rows' bytes (512 tokens,
// H = 4096: 12 us for 71 MB), for a token or two by its latency (4 us).
__global__ __launch_bounds__(256) void combine32_kernel(const float* __restrict__ y, int64_t cap,
                                                        const int32_t* __restrict__ pos,
                                                        const float* __restrict__ gates, int T, int K, int N,
                                                        uint16_t* __restrict__ out) {
    const int n = (int)(blockIdx.x * 64 + (threadIdx.x & 63)) * 4;
    const int64_t t = (int64_t)blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (t >= T || n >= N) return;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < K; k0 += 8) {
        f32x4 v[8];
        float g[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int r = k0 + k < K ? pos[t * K + k0 + k] : -1;
            const bool in = r >= 0 && r < cap;
            v[k] = in ? *(const f32x4*)(y + (int64_t)r * N + n) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            g[k] = in ? gates[t * K + k0 + k] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) acc += g[k] * v[k];
    }
    *(u32x2*)(out + t * N + n) = u32x2{pack_bf2x(acc[0], acc[1]), pack_bf2x(acc[2], acc[3])};
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

extern "C" size_t moe_gemm4_combine_workspace_size(int cap_rows, int N) {
    return cap_rows > 0 && N > 0 ? (size_t)cap_rows * (size_t)N * 4 : 0;
}

extern "C" int moe_grouped_gemm4_combine(const moe_bf16* a, const uint8_t* q4, const uint8_t* s4,
                                         const int32_t* offsets, int e_local, int Kd, int N, int cap_rows,
                                         const int32_t* pos, const float* gates, int T, int K, moe_bf16* y,
                                         moe_bf16* out, void* ws, size_t ws_bytes, moe_stream stream) {
    using namespace moe;
    bool nothing;
    const int rc = check_gemm4(e_local, Kd, N, cap_rows, offsets, &nothing);
    if (rc != MOE_OK) return rc;
    if (T < 0 || K < 1 || K > 16 || (int64_t)T * K >= (1ll << 31)) return MOE_EINVAL;
    if (T > 4 * 65535) return MOE_EINVAL;
    // without tokens there is no sum, but the rows may still be asked for
    if (N == 0 || (T == 0 && (nothing || !y))) return MOE_OK;
    if (T > 0 && (!pos || !gates || !out)) return MOE_EINVAL;
    if (!nothing && (!a || !q4 || !s4)) return MOE_EINVAL;
    if (misaligned(a) || misaligned(q4) || misaligned(s4) || misaligned(offsets) || misaligned(pos) ||
        misaligned(gates) || misaligned(y) || misaligned(out) || misaligned(ws))
        return MOE_EALIGN;
    if (!nothing && (!ws || ws_bytes < moe_gemm4_combine_workspace_size(cap_rows, N))) return MOE_EWORKSPACE;
    hipStream_t s = (hipStream_t)stream;
    if (!nothing) {
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
        p.c = y;
        p.c32 = (float*)ws;
        const int st = launch4_rows<1>(p, s);
        if (st != MOE_OK) return st;
    }
    if (T == 0) return MOE_OK;
    // with no expert or no row here, every token's sum is empty: cap 0 takes no row
    combine32_kernel<<<dim3((N / 4 + 63) / 64, (T + 3) / 4), 256, 0, s>>>((const float*)ws, nothing ? 0 : cap_rows,
                                                                          pos, gates, T, K, N, out);
    return moe_host::launch_status();
}
